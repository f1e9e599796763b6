"""GPU parity of what stands around a mixer with the fp64 oracle.

Bounds, element by element, follow from the number formats.  u is half a step of the type
(bf16 2^-8, fp32 2^-24): a result is rounded once.  A sum of n terms in fp32 is off by at most
(2 n + 16) 2^-24 of the sum of their absolute values (an addition that cuts instead of
rounding loses up to 2^-23), the few operations around it included.  In bf16 the slope is held
in fp16 (2^-11, steps of 2^-24 at the bottom) and d = d_y * slope is rounded to bf16 before
its products.  A norm's sums have at most 8 + 5 + 32 additions in a row: with the reciprocal
root and the products around them below 64 steps of 2^-24, taken twice, R = 2^-17.
"""

import numpy as np
import pytest
import torch

from oracle import block as O

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
R = 2.0 ** -17
DT = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


@pytest.fixture(scope="module")
def block():
    from recurrent_associative_memory_gb300 import block
    return block


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()


def within(x, ref, err, dtype, what):
    """One rounding of the result besides ``err``."""
    x = np64(x)
    assert x.shape == ref.shape, what
    bound = U[dtype] * (np.abs(ref) + err) + err + 1e-30
    bad = ~(np.abs(x - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.abs(x - ref)[bad].max(), bound[bad].min(),
                           (np.abs(x - ref) / bound).max())


# ------------------------------------------------------------------ matrix product

def sum_error(n):
    return (2 * n + 16) * 2.0 ** -24


def linear_case(seed, M, K, N, dtype, bias=True, residual=True, transposed=False):
    g = torch.Generator().manual_seed(seed)
    return dict(x=randn(g, M, K, dtype=dtype),
                w=(randn(g, N, K, dtype=dtype, scale=K ** -0.5).t() if transposed
                   else randn(g, K, N, dtype=dtype, scale=K ** -0.5)),
                bias=randn(g, N, dtype=dtype) if bias else None,
                residual=randn(g, M, N, dtype=dtype) if residual else None,
                d_y=randn(g, M, N, dtype=dtype))


def check_linear(block, c, act="none", bwd=True):
    x, w, bias, residual, d_y = c["x"], c["w"], c["bias"], c["residual"], c["d_y"]
    dtype, K, N = x.dtype, w.shape[0], w.shape[1]
    M = x.numel() // K
    flat = lambda t: None if t is None else np64(t).reshape(M, -1)  # noqa: E731
    X, W, dY = flat(x), np64(w), flat(d_y)
    ref, g = O.linear(X, W, None if bias is None else np64(bias), flat(residual), act, dY)
    # what the sum is off by, and what comes of it: no activation's slope passes 1.13, no
    # slope's slope 1.2
    e_pre = sum_error(K + 2) * (np.abs(X) @ np.abs(W) + (0 if bias is None else np.abs(np64(bias))))
    e_y = 1.2 * e_pre + sum_error(0) * (np.abs(ref) + (0 if residual is None else np.abs(flat(residual))))
    y, slope = block.linear_fwd(x, w, bias, act=act, residual=residual, want_slope=bwd)
    assert y.shape == (*x.shape[:-1], N) and y.is_contiguous()
    within(y.reshape(M, N), ref, e_y, dtype, "y")
    if not bwd:
        return y
    assert (slope is None) == (act == "none")
    e_s = np.zeros_like(g["slope"])
    if slope is not None:
        e_s = 1.2 * e_pre + 16 * 2.0 ** -24
        if act == "relu":
            pre = X @ W + (0 if bias is None else np64(bias))
            e_s = (np.abs(pre) <= e_pre).astype(float)
        if dtype is torch.bfloat16:
            e_s = e_s + 2.0 ** -11 * np.abs(g["slope"]) + 2.0 ** -25
        assert (np.abs(np64(slope).reshape(M, N) - g["slope"]) <= e_s + 2.0 ** -24).all()
    got = block.linear_bwd(x, w, d_y, slope=slope)
    assert got["dweight"].shape == w.shape and got["dweight"].stride() == tuple(
        (1, K) if w.stride(0) == 1 and w.stride(1) != 1 else (N, 1))
    e_sum_d = np.abs(dY) * e_s
    e_d = e_sum_d + (U[dtype] * (np.abs(g["d"]) + e_sum_d) if slope is not None else 0)
    D = np.abs(g["d"])
    within(got["dx"].reshape(M, K), g["dx"], e_d @ np.abs(W).T + sum_error(N) * (D @ np.abs(W).T), dtype, "dx")
    within(got["dweight"], g["dweight"], np.abs(X).T @ e_d + sum_error(M) * (np.abs(X).T @ D), dtype, "dweight")
    within(got["dbias"], g["dbias"], e_sum_d.sum(0) + sum_error(M) * D.sum(0), dtype, "dbias")
    again = block.linear_bwd(x, w, d_y, slope=slope)
    assert all(torch.equal(got[n], again[n]) for n in got)
    return y


SIZES = [(1, 1, 1), (1, 64, 64), (2, 8, 24), (3, 7, 5), (5, 129, 33), (17, 256, 130), (64, 100, 72), (65, 64, 200),
         (127, 72, 129), (128, 128, 256), (129, 200, 264), (256, 64, 512), (300, 333, 111), (520, 96, 1031)]


@DT
@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_sizes(block, M, K, N, dtype):
    check_linear(block, linear_case(M + K + N, M, K, N, dtype), "silu")


@DT
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M", [4, 70, 200])
def test_linear_activations_and_orders(block, M, transposed, act, dtype):
    check_linear(block, linear_case(M, M, 136, 168, dtype, transposed=transposed), act)


@DT
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_linear_without(block, bias, residual, dtype):
    for M in (3, 140):
        check_linear(block, linear_case(9, M, 64, 96, dtype, bias, residual), "gelu_tanh")
        check_linear(block, linear_case(9, M, 64, 96, dtype, bias, residual))


# ------------------------------------------------------------------ norms around a block

def norm_case(seed, M, D, dtype, h_dtype, gate=True, scale=True, post=True, weights=True, branch=True):
    g = torch.Generator().manual_seed(seed)
    c = dict(h=randn(g, M, D, dtype=h_dtype, scale=2.0), branch=randn(g, M, D, dtype=dtype) if branch else None,
             gate=randn(g, M, D, dtype=dtype, scale=2.0) if gate and branch else None,
             scale=randn(g, D) if scale and branch else None,
             post_weight=randn(g, D) if post and weights and branch else None,
             pre_weight=randn(g, D) if weights else None)
    return c, dict(d_h=randn(g, M, D, dtype=h_dtype), d_y=randn(g, M, D, dtype=dtype))


def check_norm(block, c, d, gate_act="silu", post=True, eps=1e-6):
    h, branch = c["h"], c["branch"]
    h_dtype, D = h.dtype, h.shape[-1]
    dtype = h_dtype if branch is None else branch.dtype
    M = h.numel() // D
    kw = dict(gate_act=gate_act, post_norm=post and branch is not None, eps=eps)
    flat = lambda t: None if t is None else np64(t).reshape(-1, D) if t.dim() > 1 else np64(t)  # noqa: E731
    n = {k: flat(v) for k, v in c.items()}
    ref_y, ref_h, g = O.block_norm(**n, **kw, **{k: flat(v) for k, v in d.items()})
    one = np.ones(D)
    w, pw, s = (one if n[k] is None else n[k] for k in ("pre_weight", "post_weight", "scale"))
    f, fs = (np.ones((M, D)), np.zeros((M, D))) if n["gate"] is None else O.act(gate_act, n["gate"])
    rb = O.rstd(n["branch"], eps) if kw["post_norm"] else 1.0
    v = np.zeros((M, D)) if branch is None else n["branch"] * rb
    u = v * pw
    rms = lambda e: np.sqrt((e * e).mean(-1, keepdims=True))  # noqa: E731
    mean = lambda e: e.mean(-1, keepdims=True)  # noqa: E731
    r = O.rstd(ref_h, eps)
    nn = ref_h * r
    e_h = R * (np.abs(n["h"]) + np.abs(s * f * u)) if branch is not None else 0 * ref_h
    e_r = r * rms(e_h) + R                  # of rstd, relative
    e_n = r * e_h + np.abs(nn) * e_r
    y, h_new = block.block_norm_fwd(**c, **kw)
    if branch is not None:
        within(h_new.reshape(M, D), ref_h, e_h, h_dtype, "h'")
    else:
        assert h_new is h
    within(y.reshape(M, D), ref_y, np.abs(w) * e_n, dtype, "y")
    got = block.block_norm_bwd(c["h"], branch, **{k: c[k] for k in c if k not in ("h", "branch")}, **kw, **d)
    again = block.block_norm_bwd(c["h"], branch, **{k: c[k] for k in c if k not in ("h", "branch")}, **kw, **d)
    assert all(torch.equal(got[k], again[k]) for k in got)
    dy = flat(d["d_y"]) if d.get("d_y") is not None else np.zeros((M, D))
    dh0 = flat(d["d_h"]) if d.get("d_h") is not None else np.zeros((M, D))
    t = np.abs(dy * w)
    tn = mean(t * np.abs(nn))
    size = r * (t + np.abs(nn) * tn)
    e_dh = R * (np.abs(dh0) + size) + size * e_r + r * (e_n * tn + np.abs(nn) * mean(t * e_n))
    within(got["dh"].reshape(M, D), g["dh"], e_dh, h_dtype, "dh")
    e_rows = sum_error(M)
    if d.get("d_y") is not None and c["pre_weight"] is not None:
        within(got["dpre_weight"], g["dpre_weight"], (np.abs(dy) * (e_n + e_rows * np.abs(nn))).sum(0), torch.float32,
               "dpre_weight")
    if branch is None:
        assert set(got) <= {"dh", "dpre_weight"}
        return
    a_dh, e_f = np.abs(g["dh"]), R * (np.abs(f) + 0.01)
    if c["scale"] is not None:
        err = e_dh * np.abs(f * u) + a_dh * np.abs(u) * (e_f + (R + e_rows) * np.abs(f))
        within(got["dscale"], g["dscale"], err.sum(0), torch.float32, "dscale")
    if c["gate"] is not None:
        err = np.abs(s * u) * (e_dh * np.abs(fs) + a_dh * R * (np.abs(fs) + 0.1))
        within(got["dgate"].reshape(M, D), g["dgate"], err, dtype, "dgate")
    du = g["dh"] * s * f
    e_du = np.abs(s) * (e_dh * np.abs(f) + a_dh * e_f) + R * np.abs(du)
    if c["post_weight"] is not None:
        within(got["dpost_weight"], g["dpost_weight"], (np.abs(v) * (e_du + (R + e_rows) * np.abs(du))).sum(0),
               torch.float32, "dpost_weight")
    q, e_q = np.abs(du * pw), np.abs(pw) * e_du
    if kw["post_norm"]:
        av, qv = np.abs(v), mean(q * np.abs(v))
        e_b = rb * (e_q + av * mean(e_q * av) + 3 * R * (q + av * qv))
    else:
        e_b = e_q
    within(got["dbranch"].reshape(M, D), g["dbranch"], e_b, dtype, "dbranch")


TYPES = pytest.mark.parametrize("dtype,h_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                                  (torch.float32, torch.float32)], ids=["bf16", "mixed", "fp32"])
ROWS = [(1, 1), (1, 8), (3, 7), (2, 64), (5, 100), (9, 256), (4, 257), (7, 264), (3, 1000), (1, 2048), (2, 4096),
        (3, 4097), (2, 8185), (2, 8192), (333, 24), (700, 72), (400, 520)]


@TYPES
@pytest.mark.parametrize("M,D", ROWS)
def test_norm_sizes(block, M, D, dtype, h_dtype):
    check_norm(block, *norm_case(M + D, M, D, dtype, h_dtype))


@TYPES
@pytest.mark.parametrize("gate_act", ["none", "relu", "silu", "gelu_tanh", "sigmoid"])
def test_norm_gates(block, gate_act, dtype, h_dtype):
    for D in (40, 333, 1024):
        check_norm(block, *norm_case(D, 5, D, dtype, h_dtype), gate_act=gate_act)


@TYPES
@pytest.mark.parametrize("D", [48, 1200])
@pytest.mark.parametrize("without", [("gate",), ("scale",), ("post",), ("weights",), ("gate", "scale"),
                                     ("gate", "scale", "post", "weights"), ("branch",), ("branch", "weights")])
def test_norm_without(block, without, D, dtype, h_dtype):
    c, d = norm_case(4, 6, D, dtype, h_dtype, **{k: False for k in without})
    if c["branch"] is None:
        d["d_y"] = d["d_y"].to(h_dtype)
    check_norm(block, c, d, post="post" not in without)


@TYPES
@pytest.mark.parametrize("missing", ["d_h", "d_y"])
def test_norm_one_gradient(block, missing, dtype, h_dtype):
    for D in (72, 640):
        c, d = norm_case(8, 5, D, dtype, h_dtype)
        d[missing] = None
        check_norm(block, c, d)
