"""The entry points around a mixer as callers use them: strides and slices, buffers given, in
place, other streams, captured graphs, values that are not numbers, tiles by the dozen, very
large tensors, and a block's calls together."""

import math

import numpy as np
import pytest
import torch

from oracle import block as O
from test_gpu_block import DT, TYPES, block, check_linear, check_norm, linear_case, norm_case, np64, randn  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def status_ok():
    from recurrent_associative_memory_gb300 import dr
    dr.check(dr.dr_get_device_status(), "block")


# ------------------------------------------------------------------ matrix product

@DT
@pytest.mark.parametrize("M,K,N", [(2560, 96, 2560), (130, 2560, 2304), (2313, 72, 2571)])
def test_linear_many_tiles(block, M, K, N, dtype):  # noqa: F811
    """More tiles than pairs of SMs, in the forward product or in a gradient's."""
    check_linear(block, linear_case(M, M, K, N, dtype), "silu")
    status_ok()


@DT
@pytest.mark.parametrize("M", [1, 15, 16, 17, 31, 33, 63, 65, 96, 127, 129, 191, 257, 383, 513])
def test_linear_rows(block, M, dtype):  # noqa: F811
    check_linear(block, linear_case(M, M, 192, 520, dtype), "gelu_tanh")
    check_linear(block, linear_case(M, M, 1100, 136, dtype, transposed=True))


@DT
def test_linear_long_sums(block, dtype):  # noqa: F811
    """fp32 keeps its precision over thousands of k: the pieces and their sums."""
    for M in (5, 300):
        c = linear_case(11, M, 6000, 64, dtype, bias=False, residual=False)
        check_linear(block, c)
        y, _ = block.linear_fwd(c["x"], c["w"])
        ref = np64(c["x"]) @ np64(c["w"])
        if dtype is FP:
            assert np.linalg.norm(np64(y) - ref) < 1e-6 * np.linalg.norm(ref)


@DT
def test_linear_strides(block, dtype):  # noqa: F811
    """Slices of a projection, a slice of a weight, rows that a tensor map does not hold, expanded ones."""
    g = torch.Generator().manual_seed(5)
    wide, w, res = randn(g, 6, 20, 3, 64, dtype=dtype), randn(g, 64, 200, dtype=dtype, scale=0.1), randn(g, 6, 20, 300, dtype=dtype)
    bias = randn(g, 72, dtype=dtype)
    dy = randn(g, 6, 20, 72, dtype=dtype)
    views = {"slice of a projection": wide[:, :, 1], "every second token": randn(g, 6, 40, 64, dtype=dtype)[:, ::2],
             "rows of an odd length": randn(g, 6, 20, 67, dtype=dtype)[..., :64],
             "one row expanded": randn(g, 1, 1, 64, dtype=dtype).expand(6, 20, 64)}
    for x in views.values():
        for weight in (w[:, 16:88], w[:, :72].t().contiguous().t(), randn(g, 64, 73, dtype=dtype)[:, :72],
                       randn(g, 72, 65, dtype=dtype)[:, :64].t()):
            c = dict(x=x, w=weight, bias=bias, residual=res[..., 16:88], d_y=dy)
            check_linear_values(block, c)


def check_linear_values(block, c):  # noqa: F811
    """The same values in plain tensors give the same bits."""
    plain = dict(c, x=c["x"].contiguous(), residual=c["residual"].contiguous(),
                 w=c["w"].t().contiguous().t() if c["w"].stride(0) == 1 else c["w"].contiguous())
    check_linear(block, plain, "silu")
    y, s = block.linear_fwd(c["x"], c["w"], c["bias"], act="silu", residual=c["residual"], want_slope=True)
    y2, s2 = block.linear_fwd(plain["x"], plain["w"], c["bias"], act="silu", residual=plain["residual"], want_slope=True)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    g, g2 = (block.linear_bwd(t["x"], t["w"], c["d_y"], slope=s) for t in (c, plain))
    assert all(torch.equal(g[k], g2[k]) for k in g)


@DT
def test_linear_buffers(block, dtype):  # noqa: F811
    """Buffers given, y over the residual, gradients one by one, a workspace to reuse."""
    from recurrent_associative_memory_gb300 import dr
    for M in (9, 600):
        c = linear_case(M, M, 88, 72, dtype)
        args = (c["x"], c["w"], c["bias"])
        y, s = block.linear_fwd(*args, act="silu", residual=c["residual"], want_slope=True)
        assert block.linear_fwd(*args, act="silu")[1] is None and block.linear_fwd(*args, want_slope=True)[1] is None
        over, slope = c["residual"].clone(), torch.empty_like(s)
        got, kept = block.linear_fwd(*args, act="silu", residual=over, y=over, slope=slope)
        assert got is over and kept is slope and torch.equal(over, y) and torch.equal(slope, s)
        g = block.linear_bwd(c["x"], c["w"], c["d_y"], slope=s)
        for name in ("dx", "dweight", "dbias"):
            buf = torch.empty_like(g[name])
            want = {f"want_{n}": n == name for n in ("dx", "dweight", "dbias")}
            one = block.linear_bwd(c["x"], c["w"], c["d_y"], slope=s, grads={name: buf}, **want)
            assert set(one) == {name} and one[name] is buf and torch.equal(buf, g[name])
        t = block.linear_bwd(c["x"], c["w"].t().contiguous().t(), c["d_y"], slope=s)
        assert t["dweight"].stride() == (1, 88)
        np.testing.assert_allclose(np64(t["dweight"]), np64(g["dweight"]), rtol=2 ** -6, atol=1e-5 * M)
        a = dr.DrLinear(int(dtype is BF), 2, M, 88, 72, 0, 88, 72, 0)
        ws = torch.full((dr.dr_linear_bwd_workspace_bytes(a),), 255, dtype=torch.uint8, device="cuda")
        again = block.linear_bwd(c["x"], c["w"], c["d_y"], slope=s, workspace=ws)
        assert all(torch.equal(again[k], g[k]) for k in g)


@DT
@pytest.mark.parametrize("M,K,N", [(3000, 520, 264), (2600, 1032, 2056), (5000, 24, 40), (3001, 515, 1028), (2600, 136, 1112),
                                   (1, 264, 132), (7, 77, 515), (8, 520, 1028), (60, 1032, 130), (201, 333, 777)])
def test_linear_writes_no_more(block, M, K, N, dtype):  # noqa: F811
    """Rows of every remainder of 16 columns: nothing behind a result is written, and the same
    bits come each time."""
    c = linear_case(M, M, K, N, dtype)
    S = torch.float16 if dtype is BF else torch.float32

    def run():
        flat = {k: torch.full((rows * cols + 256,), 7.0, dtype=t, device="cuda")
                for k, rows, cols, t in (("y", M, N, dtype), ("slope", M, N, S), ("dx", M, K, dtype), ("dweight", K, N, dtype))}
        buf = {k: f[:-256].view(-1, K if k == "dx" else N) for k, f in flat.items()}
        block.linear_fwd(c["x"], c["w"], c["bias"], act="silu", residual=c["residual"], y=buf["y"], slope=buf["slope"])
        block.linear_bwd(c["x"], c["w"], c["d_y"], slope=buf["slope"], grads={k: buf[k] for k in ("dx", "dweight")})
        for k, f in flat.items():
            assert bool((f[-256:] == 7).all()), k
        return flat

    first, again = run(), run()
    assert all(torch.equal(first[k], again[k]) for k in first)
    check_linear(block, c, "silu")


@DT
@pytest.mark.parametrize("M,K,N", [(3000, 520, 264), (700, 2000, 1100), (300, 4000, 24), (90, 64, 2000)])
def test_linear_gradients_read_at_once(block, M, K, N, dtype):  # noqa: F811
    """What the stream does next finds every gradient done, dx (the first product) too, and the
    next call on the same workspace and buffers leaves those before as they were."""
    from recurrent_associative_memory_gb300 import dr
    a = dr.DrLinear(int(dtype is BF), 2, M, K, N, 0, K, N, 0)
    ws = torch.empty(dr.dr_linear_bwd_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    cases, want = [linear_case(M + i, M, K, N, dtype) for i in range(3)], []
    for c in cases:
        c["slope"] = block.linear_fwd(c["x"], c["w"], c["bias"], act="silu", want_slope=True)[1]
        torch.cuda.synchronize()
        g = block.linear_bwd(c["x"], c["w"], c["d_y"], slope=c["slope"])
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in g.items()})
    buffers = {k: torch.empty_like(v) for k, v in want[0].items()}
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        c = cases[i % 3]
        for b in buffers.values():
            b.fill_(float("nan"))
        block.linear_bwd(c["x"], c["w"], c["d_y"], slope=c["slope"], grads=buffers, workspace=ws)
        got.append({k: buffers[k].clone() for k in ("dx", "dbias", "dweight")})
    for i, g in enumerate(got):
        assert all(torch.equal(g[k], want[i % 3][k]) for k in g), i


@DT
def test_linear_refuses(block, dtype):  # noqa: F811
    c = linear_case(3, 10, 32, 24, dtype)
    x, w, b = c["x"], c["w"], c["bias"]
    other = FP if dtype is BF else BF
    wrong = [(ValueError, lambda: block.linear_fwd(x, w[:16])), (TypeError, lambda: block.linear_fwd(x, w.to(other))),
             (TypeError, lambda: block.linear_fwd(x, w.cpu())), (ValueError, lambda: block.linear_fwd(x, w, act="tanh")),
             (ValueError, lambda: block.linear_fwd(x, w[:, ::2])), (ValueError, lambda: block.linear_fwd(x[:, ::2], w[:16])),
             (ValueError, lambda: block.linear_fwd(x, w, b[:5])), (TypeError, lambda: block.linear_fwd(x, w, b.to(other))),
             (ValueError, lambda: block.linear_fwd(x, w, residual=c["residual"][:5])),
             (ValueError, lambda: block.linear_fwd(x, w, y=torch.empty(24, 10, dtype=dtype, device="cuda").t())),
             (TypeError, lambda: block.linear_fwd(x, w, act="silu", slope=torch.empty(10, 24, dtype=BF, device="cuda"))),
             (ValueError, lambda: block.linear_fwd(x.view(2, 5, 32).transpose(0, 1), w)),
             (ValueError, lambda: block.linear_bwd(x, w, c["d_y"][:, :8])),
             (ValueError, lambda: block.linear_bwd(x, w.t().contiguous().t(), c["d_y"], grads={"dweight": torch.empty_like(w)})),
             (ValueError, lambda: block.linear_fwd(x, w, workspace="none"))]
    for kind, call in wrong:
        with pytest.raises(kind):
            call()
    from recurrent_associative_memory_gb300 import dr
    with pytest.raises(dr.DrError):
        block.linear_fwd(x[:0], w)
    if dtype is FP:
        block.linear_fwd(x[:8], w, workspace=None)   # so few rows take none
        with pytest.raises(dr.DrError):
            block.linear_fwd(linear_case(3, 20, 32, 24, dtype)["x"], w, workspace=None)
    with pytest.raises(dr.DrError):
        block.linear_fwd(torch.zeros(4 * 32 + 1, dtype=dtype, device="cuda")[1:].view(4, 32), w)
    torch.cuda.synchronize()


def test_linear_rows_keep_to_themselves(block):  # noqa: F811
    """NaN and infinities in one row of x or of the residual reach that row only; the other rows
    keep their bits."""
    for dtype in (BF, FP):
        for M in (6, 700):
            c = linear_case(M, M, 200, 264, dtype)
            y, _ = block.linear_fwd(c["x"], c["w"], c["bias"], act="silu", residual=c["residual"])
            x, r = c["x"].clone(), c["residual"].clone()
            x[2, 7], x[3, 0], r[4, 5] = math.nan, math.inf, -math.inf
            z, _ = block.linear_fwd(x, c["w"], c["bias"], act="silu", residual=r)
            keep = [i for i in range(M) if i not in (2, 3, 4)]
            assert torch.equal(z[keep], y[keep]) and z[2].isnan().all() and not z[3].isfinite().any()
            assert z[4, 5] == -math.inf and torch.equal(z[4, :5], y[4, :5]) and torch.equal(z[4, 6:], y[4, 6:])


def test_linear_large_values(block):  # noqa: F811
    """Far ends of the activations and their slopes; sums that cancel."""
    x = torch.tensor([[1.0], [-1.0], [0.0], [-0.0]], device="cuda")
    w = torch.tensor([[1e-30, 1.0, 30.0, 100.0, 1e10, 1e30, 3e38, 0.0]], device="cuda")
    for dtype in (BF, FP):
        for act in ("none", "relu", "silu", "gelu_tanh", "sigmoid"):
            y, s = block.linear_fwd(x.to(dtype), w.to(dtype), act=act, want_slope=True)
            ref, slope = O.act(act, np64(x.to(dtype)) @ np64(w.to(dtype))) if act != "gelu_tanh" else O.act(
                act, np.clip(np64(x.to(dtype)) @ np64(w.to(dtype)), -1e10, 1e30))
            assert y.isfinite().all()
            fine = np.isfinite(ref) & ((np.abs(ref) < 1e29) | (act != "gelu_tanh"))
            np.testing.assert_allclose(np64(y)[fine], ref[fine], rtol=2 ** -7, atol=1e-30 if act == "none" else 1e-6)
            if s is not None:
                assert s.isfinite().all() and float(s.float().abs().max()) <= 1.13
                if act != "gelu_tanh":
                    np.testing.assert_allclose(np64(s), slope, atol=2e-3 if dtype is BF else 1e-5)


@DT
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "sigmoid"])
def test_linear_nan_reaches_its_slopes(block, act, dtype):  # noqa: F811
    for M in (5, 300):
        c = linear_case(M, M, 64, 136, dtype)
        c["x"][2, 3] = math.nan
        y, s = block.linear_fwd(c["x"], c["w"], c["bias"], act=act, want_slope=True)
        rest = [i for i in range(M) if i != 2]
        assert y[2].isnan().all() and s[2].isnan().all() and y[rest].isfinite().all() and s[rest].isfinite().all()
        g = block.linear_bwd(c["x"], c["w"], c["d_y"], slope=s)
        assert g["dx"][2].isnan().all() and g["dx"][rest].isfinite().all() and g["dweight"].isnan().all()


# ------------------------------------------------------------------ norms around a block

@TYPES
@pytest.mark.parametrize("M,D", [(700, 256), (700, 264), (1300, 511), (640, 2040), (640, 2042), (310, 2048), (320, 2049),
                                 (330, 4090), (400, 4096), (310, 4104), (190, 6000), (200, 8184), (170, 8191), (160, 8192)])
def test_norm_many_rows(block, M, D, dtype, h_dtype):  # noqa: F811
    """Several rows to each block, at the sizes where the blocks change their shape."""
    check_norm(block, *norm_case(M + D, M, D, dtype, h_dtype))
    status_ok()


@TYPES
@pytest.mark.parametrize("D", [64, 333, 1000])
def test_norm_strides(block, D, dtype, h_dtype):  # noqa: F811
    """Slices in three dimensions, odd strides and an expanded row give what plain tensors give."""
    g = torch.Generator().manual_seed(D)
    B, T = 3, 70
    c, d = norm_case(D, B * T, D, dtype, h_dtype)
    shape = (B, T, D)
    plain = {k: v.view(shape) if v is not None and v.dim() == 2 else v for k, v in c.items()}
    d = {k: v.view(shape) for k, v in d.items()}
    kw = dict(gate_act="silu", post_norm=True)

    def inside(t, before, after):
        wide = torch.full((B, T, D + before + after), math.nan, dtype=t.dtype, device="cuda")
        wide[..., before:before + D] = t
        return wide[..., before:before + D]

    for before, after in ((0, 8), (8, 0), (16, 40), (0, 1), (3, 2), (1, 7)):
        view = {k: inside(v, before, after) if v is not None and v.dim() == 3 else v for k, v in plain.items()}
        y, h = block.block_norm_fwd(**plain, **kw)
        y2, h2 = block.block_norm_fwd(**view, **kw)
        for a, b in ((y, y2), (h, h2)):   # other threads may take the columns: fp32 sums in another order
            np.testing.assert_allclose(np64(a), np64(b), rtol=2.0 ** -7 if a.dtype is BF else 1e-5, atol=1e-5)
        f = block.block_norm_bwd(**plain, **d, **kw)
        f2 = block.block_norm_bwd(**view, **d, **kw)
        for k in f:
            scale = float(f[k].float().abs().max())
            np.testing.assert_allclose(np64(f[k]), np64(f2[k]), rtol=2.0 ** -7 if f[k].dtype is BF else 1e-4, atol=1e-4 * scale)
    one = randn(g, 1, 1, D, dtype=dtype)
    y, _ = block.block_norm_fwd(plain["h"], one.expand(shape))
    y2, _ = block.block_norm_fwd(plain["h"], one.expand(shape).contiguous())
    np.testing.assert_allclose(np64(y), np64(y2), rtol=2.0 ** -7 if dtype is BF else 1e-5, atol=1e-5)


@TYPES
@pytest.mark.parametrize("M,D", [(1, 7), (5, 264), (3, 1111), (40, 333), (2, 4097), (333, 24), (700, 8192), (401, 2047)])
def test_norm_writes_no_more(block, M, D, dtype, h_dtype):  # noqa: F811
    """Neither before nor behind a result, on 16 bytes (264 values) or not."""
    c, d = norm_case(M, M, D, dtype, h_dtype)
    n = M * D
    types = dict(h_out=h_dtype, y=dtype, dh=h_dtype, dbranch=dtype, dgate=dtype)
    for pad in (264, 259):
        flat = {k: torch.full((n + 2 * pad,), 7.0, dtype=t, device="cuda") for k, t in types.items()}
        flat |= {k: torch.full((D + 2 * pad,), 7.0, device="cuda") for k in ("dscale", "dpost_weight", "dpre_weight")}
        buf = {k: f[pad:-pad].view((M, D) if k in types else (D,)) for k, f in flat.items()}
        kw = dict(gate_act="silu", post_norm=True)
        block.block_norm_fwd(**c, **kw, h_out=buf["h_out"], y=buf["y"])
        block.block_norm_bwd(**c, **d, **kw, grads={k: b for k, b in buf.items() if k[0] == "d"})
        for k, f in flat.items():
            assert bool((f[:pad] == 7).all()) and bool((f[-pad:] == 7).all()), k
            assert bool((buf[k] != 7).any()), k


@TYPES
def test_norm_buffers(block, dtype, h_dtype):  # noqa: F811
    """The stream taken on in place, buffers given, h returned as it is without a branch."""
    for D in (40, 333, 1024, 4096):
        c, d = norm_case(D, 400, D, dtype, h_dtype)
        kw = dict(gate_act="silu", post_norm=True)
        y, h = block.block_norm_fwd(**c, **kw)
        stream, out = c["h"].clone(), torch.empty_like(y)
        got, there = block.block_norm_fwd(**{**c, "h": stream}, **kw, h_out=stream, y=out)
        assert got is out and there is stream and torch.equal(out, y) and torch.equal(stream, h)
        none, h3 = block.block_norm_fwd(**{**c, "pre_weight": None}, **kw, want_y=False)
        assert none is None and torch.equal(h3, h)
        g = block.block_norm_bwd(**c, **d, **kw)
        bufs = {k: torch.empty_like(v) for k, v in g.items()}
        got = block.block_norm_bwd(**c, **d, **kw, grads=bufs)
        assert all(got[k] is bufs[k] and torch.equal(got[k], g[k]) for k in g)
        alone, same = block.block_norm_fwd(c["h"], pre_weight=c["pre_weight"], dtype=dtype)
        assert same is c["h"] and alone.dtype is dtype


def test_norm_refuses(block):  # noqa: F811
    from recurrent_associative_memory_gb300 import dr
    c, d = norm_case(1, 6, 64, BF, BF)
    h, b = c["h"], c["branch"]
    wrong = [(ValueError, lambda: block.block_norm_fwd(h, b[:3])), (TypeError, lambda: block.block_norm_fwd(h, b, gate=c["gate"].float())),
             (ValueError, lambda: block.block_norm_fwd(h, b, gate_act="tanh")), (ValueError, lambda: block.block_norm_fwd(h, h_out=h)),
             (TypeError, lambda: block.block_norm_fwd(h, b, scale=c["scale"].bfloat16())), (TypeError, lambda: block.block_norm_fwd(h, b, dtype=FP)),
             (ValueError, lambda: block.block_norm_fwd(h, b, pre_weight=c["pre_weight"][:8])), (TypeError, lambda: block.block_norm_fwd(h, dtype=torch.float16)),
             (ValueError, lambda: block.block_norm_fwd(h.cpu(), b)), (ValueError, lambda: block.block_norm_fwd(h, b.cpu())),
             (ValueError, lambda: block.block_norm_bwd(h, b, d_y=d["d_y"][:, :8])),
             (ValueError, lambda: block.block_norm_fwd(h.view(2, 3, 64).transpose(0, 1)))]
    for kind, call in wrong:
        with pytest.raises(kind):
            call()
    for call in (lambda: block.block_norm_fwd(h, dtype=FP), lambda: block.block_norm_bwd(h, b), lambda: block.block_norm_fwd(h, b, y=b, h_out=b),
                 lambda: block.block_norm_fwd(h, gate=c["gate"]), lambda: block.block_norm_fwd(h, b, post_weight=c["post_weight"]),
                 lambda: block.block_norm_fwd(h, b, eps=-1.0), lambda: block.block_norm_fwd(torch.zeros(2, 8200, dtype=BF, device="cuda")),
                 lambda: block.block_norm_bwd(**c, **d, post_norm=True, workspace=None)):
        with pytest.raises(dr.DrError):
            call()
    torch.cuda.synchronize()


@TYPES
def test_norm_special_values(block, dtype, h_dtype):  # noqa: F811
    """Rows of zeros, tiny and large ones, NaN and infinities: each stays in its row."""
    for D in (48, 333, 2000):
        c, d = norm_case(D, 50, D, dtype, h_dtype)
        kw = dict(gate_act="sigmoid", post_norm=True)
        y, h = block.block_norm_fwd(**c, **kw)
        x = {k: v.clone() for k, v in c.items()}
        x["h"][1], x["branch"][1] = 0, 0
        x["branch"][2] = 0
        x["h"][3, 5], x["branch"][4, 0], x["gate"][5, D - 1] = math.nan, math.inf, math.nan
        x["h"][6] *= 1e15
        x["gate"][7], x["gate"][8] = -1e30, 1e30
        y2, h2 = block.block_norm_fwd(**x, **kw)
        keep = [0, *range(9, 50)]
        assert torch.equal(y[keep], y2[keep]) and torch.equal(h[keep], h2[keep])
        assert (y2[1] == 0).all() and (h2[1] == 0).all() and torch.equal(h2[2], c["h"][2]) and torch.equal(h2[7], c["h"][7])
        assert y2[3].isnan().all() and y2[4].isnan().all() and y2[5].isnan().all() and y2[[6, 7, 8]].isfinite().all()
        g = block.block_norm_bwd(**x, **d, **kw)
        f = block.block_norm_bwd(**c, **d, **kw)
        for k in ("dh", "dbranch", "dgate"):
            assert torch.equal(g[k][keep], f[k][keep]), k
        assert g["dh"][1].isfinite().all() and (g["dgate"][7:9] == 0).all() and g["dbranch"][8].isfinite().all()


# ------------------------------------------------------------------ streams and graphs

def calls(block, dtype, M=200):  # noqa: F811
    """Every entry point over its own inputs: a list of functions of a stream that give tensors."""
    c = linear_case(1, M, 136, 264, dtype)
    odd = linear_case(2, M, 77, 51, dtype)
    n, d = norm_case(3, M, 1000, dtype, dtype)
    w, e = norm_case(4, M, 77, dtype, FP)
    kw = dict(gate_act="silu", post_norm=True)

    def product(c):
        def run(stream=None):
            y, s = block.linear_fwd(c["x"], c["w"], c["bias"], act="silu", residual=c["residual"], want_slope=True, stream=stream)
            return [y, s, *block.linear_bwd(c["x"], c["w"], c["d_y"], slope=s, stream=stream).values()]
        return run

    def norms(n, d):
        def run(stream=None):
            return [*block.block_norm_fwd(**n, **kw, stream=stream), *block.block_norm_bwd(**n, **d, **kw, stream=stream).values()]
        return run
    return [product(c), product(odd), norms(n, d), norms(w, e)]


@DT
def test_another_stream(block, dtype):  # noqa: F811
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    for run in calls(block, dtype):
        want = run()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                busy = busy @ busy * 1e-4
        got = [run(side), run(side.cuda_stream)]
        taken = [torch.full_like(t, 1) for t in want]      # what the current stream may be given meanwhile
        torch.cuda.synchronize()
        assert taken and all(torch.equal(a, b) for r in got for a, b in zip(r, want))


@DT
def test_captured_graph(block, dtype):  # noqa: F811
    """Captured once and replayed over new inputs; two graphs do not share what they write."""
    M = 200
    c, (n, d) = linear_case(1, M, 136, 264, dtype), norm_case(3, M, 1000, dtype, dtype)
    kw = dict(gate_act="silu", post_norm=True)

    def run(c, n, d):
        y, s = block.linear_fwd(c["x"], c["w"], c["bias"], act="silu", residual=c["residual"], want_slope=True)
        return [y, s, *block.linear_bwd(c["x"], c["w"], c["d_y"], slope=s).values(),
                *block.block_norm_fwd(**n, **kw), *block.block_norm_bwd(**n, **d, **kw).values()]
    run(c, n, d)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(c, n, d)
        graphs.append((g, out))
    for seed in (7, 8):
        c2, (n2, d2) = linear_case(seed, M, 136, 264, dtype), norm_case(seed, M, 1000, dtype, dtype)
        want = run(c2, n2, d2)
        for old, new in ((c, c2), (n, n2), (d, d2)):
            for k in old:
                if old[k] is not None:
                    old[k].copy_(new[k])
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    status_ok()


def test_two_streams_at_once(block):  # noqa: F811
    """Kernels of several streams share SMs and tensor memory."""
    streams = [torch.cuda.Stream() for _ in range(4)]
    for dtype in (BF, FP):
        runs = calls(block, dtype, M=900)
        want = [r() for r in runs]
        torch.cuda.synchronize()
        got = []
        for _ in range(5):
            for s, r in zip(streams, runs):
                with torch.cuda.stream(s):
                    got.append(r())
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(g, want[i % 4]))
    status_ok()


# ------------------------------------------------------------------ large tensors

def test_linear_beyond_31_bits(block):  # noqa: F811
    """x and y of more than 2^31 values: rows at both ends."""
    M, K, N = 70000, 64, 32768
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=BF)
    w = torch.randn(K, N, generator=g, device="cuda", dtype=BF) * K ** -0.5
    y, _ = block.linear_fwd(x, w)
    at = torch.tensor([0, 1, 255, 256, 65535, 65536, M - 1], device="cuda")
    ref = x[at].double() @ w.double()
    assert bool(((y[at].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4).all())
    back = block.linear_bwd(x, w, y, want_dweight=False, want_dbias=False)["dx"]
    ref = y[at].double() @ w.double().t()
    assert float((back[at].double() - ref).norm() / ref.norm()) < 2.0 ** -8


def test_norm_beyond_31_bits(block):  # noqa: F811
    M, D = 270000, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(M, D, generator=g, device="cuda", dtype=BF)
    y, h2 = block.block_norm_fwd(h, h, post_norm=True)
    at = torch.tensor([0, 1, 65536, 262144, M - 1], device="cuda")
    x = h[at].double()
    x = x + x * (x * x).mean(-1, keepdim=True).rsqrt()
    ref = x * (x * x).mean(-1, keepdim=True).rsqrt()
    assert bool(((y[at].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4).all())
    assert bool(((h2[at].double() - x).abs() <= 2.0 ** -8 * x.abs() + 1e-4).all())


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,bound", [(FP, 2e-5), (BF, 12 * 2.0 ** -8)], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,dim", [(3, 64), (150, 200), (700, 264)])
def test_a_block_forward_and_backward(block, M, dim, dtype, bound):  # noqa: F811
    """norm -> wide layer with bias and activation -> layer back -> norm, gate, scale, residual
    and the next norm, and back again, against the formulas composed in 64 bits.  Twelve
    roundings follow one another at most (bf16: half a step, 2^-8, each); fp32 sums keep
    within 2e-5."""
    g = torch.Generator().manual_seed(M)
    h = randn(g, M, dim, dtype=dtype)
    up, down = randn(g, dim, 3 * dim, dtype=dtype, scale=dim ** -0.5), randn(g, 3 * dim, dim, dtype=dtype, scale=(3 * dim) ** -0.5)
    gates = randn(g, dim, dim, dtype=dtype, scale=dim ** -0.5)
    bias = randn(g, 3 * dim, dtype=dtype, scale=0.3)
    w0, w1, pw, sc = (randn(g, dim, scale=0.1) + 1 for _ in range(4))
    dy, dh = randn(g, M, dim, dtype=dtype), randn(g, M, dim, dtype=dtype)
    end = dict(gate_act="sigmoid", scale=sc, post_norm=True, post_weight=pw, pre_weight=w1)
    x, _ = block.block_norm_fwd(h, pre_weight=w0)
    a, slope = block.linear_fwd(x, up, bias, act="silu", want_slope=True)
    o, _ = block.linear_fwd(a, down)
    z, _ = block.linear_fwd(x, gates)
    y, h2 = block.block_norm_fwd(h, o, gate=z, **end)
    ge = block.block_norm_bwd(h, o, gate=z, d_h=dh, d_y=dy, **end)
    gz = block.linear_bwd(x, gates, ge["dgate"], want_dbias=False)
    gd = block.linear_bwd(a, down, ge["dbranch"], want_dbias=False)
    gu = block.linear_bwd(x, up, gd["dx"], slope=slope)
    dx, _ = block.linear_fwd(ge["dgate"], gates.t(), residual=gu["dx"])   # both ways into x at once
    g0 = block.block_norm_bwd(h, d_h=ge["dh"], d_y=dx, pre_weight=w0)
    got = dict(y=y, h=h2, dh=g0["dh"], dw0=g0["dpre_weight"], dup=gu["dweight"], dbias=gu["dbias"], ddown=gd["dweight"],
               dgates=gz["dweight"], dscale=ge["dscale"], dpost=ge["dpost_weight"], dw1=ge["dpre_weight"])

    leaf = [t.double().requires_grad_() for t in (h, w0, up, bias, down, gates, sc, pw, w1)]
    H, W0, UP, B, DN, GT, SC, PW, W1 = leaf
    n = lambda t: t * ((t * t).mean(-1, keepdim=True) + 1e-6) ** -0.5  # noqa: E731
    X = n(H) * W0
    H2 = H + SC * torch.sigmoid(X @ GT) * n(torch.nn.functional.silu(X @ UP + B) @ DN) * PW
    Y = n(H2) * W1
    grads = torch.autograd.grad((Y, H2), leaf, (dy.double(), dh.double()))
    want = dict(zip(("dh", "dw0", "dup", "dbias", "ddown", "dgates", "dscale", "dpost", "dw1"), grads), y=Y, h=H2)
    for k, v in got.items():
        err = float((v.double() - want[k].detach()).norm() / want[k].detach().norm())
        assert err < bound, (k, err)
    status_ok()
