"""The longest sums and the widest strides around a mixer.  Inputs are -1, 0 and 1, so that every
sum is a whole number below 2^24: exact in fp32 in any order, rounded once in bf16."""

import threading

import pytest
import torch

from test_gpu_block import DT, TYPES, block, linear_case, norm_case  # noqa: F401

pytestmark = pytest.mark.gpu


def signs(gen, *shape, dtype):
    return torch.randint(-1, 2, shape, generator=gen, device="cuda", dtype=torch.int8).to(dtype)


def exact(x, w):
    """x w in blocks of k, in 64 bits."""
    return sum(x[:, k:k + (1 << 20)].double() @ w[k:k + (1 << 20)].double() for k in range(0, w.shape[0], 1 << 20))


@DT
@pytest.mark.parametrize("M", [3, 20])
@pytest.mark.parametrize("transposed", [False, True])
def test_sums_over_the_most_channels(block, M, transposed, dtype):  # noqa: F811
    K, N = 1 << 24, 8
    g = torch.Generator(device="cuda").manual_seed(M)
    x = signs(g, M, K, dtype=dtype)
    w = signs(g, N, K, dtype=dtype).t() if transposed else signs(g, K, N, dtype=dtype)
    y, _ = block.linear_fwd(x, w)
    assert torch.equal(y, exact(x, w).to(dtype))


@DT
def test_gradients_over_many_rows(block, dtype):  # noqa: F811
    M, K, N = (1 << 24) + 5, 8, 24
    g = torch.Generator(device="cuda").manual_seed(2)
    x, d, w = signs(g, M, K, dtype=dtype), signs(g, M, N, dtype=dtype), signs(g, K, N, dtype=dtype)
    got = block.linear_bwd(x, w, d)
    assert torch.equal(got["dweight"], exact(x.t(), d).to(dtype))
    assert torch.equal(got["dbias"], d.sum(0, dtype=torch.float64).to(dtype))
    assert torch.equal(got["dx"], (d.float() @ w.float().t()).to(dtype))


def apart(t, stride):
    """The rows of t, ``stride`` values apart."""
    far = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype, device="cuda").as_strided(t.shape, (stride, 1))
    return far.copy_(t)


@DT
@pytest.mark.parametrize("stride", [(1 << 31) + 8, (1 << 31) + 3])
def test_rows_of_the_product_far_apart(block, stride, dtype):  # noqa: F811
    c = linear_case(1, 3, 72, 40, dtype)
    want = block.linear_fwd(c["x"], c["w"], c["bias"], act="silu", residual=c["residual"])[0]
    assert torch.equal(block.linear_fwd(apart(c["x"], stride), c["w"], c["bias"], act="silu",
                                        residual=apart(c["residual"], stride))[0], want)
    assert torch.equal(block.linear_bwd(apart(c["x"], stride), c["w"], c["d_y"])["dweight"],
                       block.linear_bwd(c["x"], c["w"], c["d_y"])["dweight"])


@TYPES
@pytest.mark.parametrize("D", [24, 264, 333])
def test_rows_of_the_norms_far_apart(block, D, dtype, h_dtype):  # noqa: F811
    c, d = norm_case(1, 3, D, dtype, h_dtype)
    far = {k: apart(c[k], (1 << 30) + D % 8) if k in ("h", "branch", "gate") else v for k, v in c.items()}
    kw = dict(gate_act="silu", post_norm=True)
    for a, b in zip(block.block_norm_fwd(**far, **kw), block.block_norm_fwd(**c, **kw)):
        assert torch.equal(a, b)
    got, want = block.block_norm_bwd(**far, **d, **kw), block.block_norm_bwd(**c, **d, **kw)
    assert all(torch.equal(got[k], want[k]) for k in want)


@DT
def test_calls_of_two_threads(block, dtype):  # noqa: F811
    """Each on a stream of its own, both at once."""
    c, (n, d) = linear_case(5, 300, 136, 264, dtype), norm_case(6, 300, 1000, dtype, dtype)
    kw = dict(gate_act="silu", post_norm=True)

    def run():
        y, s = block.linear_fwd(c["x"], c["w"], c["bias"], act="silu", want_slope=True)
        return [y, *block.linear_bwd(c["x"], c["w"], c["d_y"], slope=s).values(),
                *block.block_norm_fwd(**n, **kw), *block.block_norm_bwd(**n, **d, **kw).values()]
    want = run()
    torch.cuda.synchronize()
    got, failed = [], []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                mine = [run() for _ in range(30)]
                torch.cuda.current_stream().synchronize()
            got.extend(mine)
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(got) == 60
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
