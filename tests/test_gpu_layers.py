"""GPU parity of the layers next to the recurrence with the fp64 oracle.

Bounds, element by element, are derived from the number formats: with u the unit of
the tensors' type (bf16 2^-8, one unit for the result and one for what the kernel rounds
on the way -- probabilities, their gradients, the saved output; fp32 2^-16, i.e. 2^-24 per
operation times 2^8 for the longest chain of operations in an exponent or a sum),
    |x - ref| <= u (|ref| + sum of the absolute values that are summed).
Recurrences in fp32 keep |x - ref| <= 2^-16 max|ref| per output besides that.
"""

import math

import numpy as np
import pytest
import torch

from oracle import layers as L

pytestmark = pytest.mark.gpu
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -16}


@pytest.fixture(scope="module")
def mods():
    from recurrent_associative_memory_gb300 import attention, ssm
    return attention, ssm


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def within(x, ref, size, dtype, what=""):
    x = np64(x)
    assert x.shape == ref.shape, what
    bound = UNIT[dtype] * (np.abs(ref) + size) + 1e-30
    bad = ~(np.abs(x - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.abs(x - ref)[bad].max(), bound[bad].min())


def close(x, ref, dtype, what=""):
    """One rounding of the result on top of an fp32 recurrence."""
    within(x, ref, np.full(ref.shape, 2.0 ** -16 / UNIT[dtype] * np.abs(ref).max(initial=0.0)), dtype, what)


def randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


# ------------------------------------------------------------------ window attention

def qkv(seed, B, T, S, H, Hk, d, dtype):
    """Slices of one projection, so every stride is larger than the slice."""
    g = torch.Generator().manual_seed(seed)
    q = randn(g, B, T, H + 1, d, dtype=dtype)[:, :, :H]
    kv = randn(g, B, S, 2 * Hk, d, dtype=dtype)
    return q, kv[:, :, :Hk], kv[:, :, Hk:], randn(g, B, T, H, d, dtype=dtype)


def check_attention(attention, T, S, window, n_sink, q_start=0, lens=None, H=2, Hk=1, d=64,
                    dtype=torch.bfloat16, B=2, scale=None, bwd=True):
    q, k, v, do = qkv(T + 7 * window + n_sink, B, T, S, H, Hk, d, dtype)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if lens is not None:             # what stands behind a sequence's end is never looked at
        for b, n in enumerate(lens):
            k[b, max(0, min(n, S)):], v[b, max(0, min(n, S)):] = math.nan, math.nan
    clamped = None if lens is None else [max(0, min(n, S)) for n in lens]
    args = (np64(q), np.nan_to_num(np64(k)), np.nan_to_num(np64(v)), window, n_sink, q_start, clamped, scale)
    ref, lse_ref, size, grads, sizes = L.window_attention(*args, d_out=np64(do))
    kw = dict(q_start=q_start, lens=lt, scale=scale)
    out, lse = attention.window_attn_fwd(q, k, v, window, n_sink, want_lse=True, **kw)
    within(out, ref, size, dtype, "out")
    got = np64(lse)
    none = np.isneginf(lse_ref)
    assert (np.isneginf(got) == none).all()
    # scores are sums of d fp32 products of at most 2^3 in size
    np.testing.assert_allclose(got[~none], lse_ref[~none], atol=2e-5 * max(1.0, (scale or 0) * d), rtol=1e-5)
    alone, no_lse = attention.window_attn_fwd(q, k, v, window, n_sink, **kw)
    assert no_lse is None and torch.equal(alone, out)
    if not bwd:
        return
    g = attention.window_attn_bwd(q, k, v, out, lse, do, window, n_sink, **kw)
    for name in ("dq", "dk", "dv"):
        within(g[name], grads[name], sizes[name], dtype, name)
    again = attention.window_attn_bwd(q, k, v, out, lse, do, window, n_sink, **kw)
    assert all(torch.equal(g[n], again[n]) for n in g)


DT = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


@DT
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,window,n_sink", [(1, 1, 0), (2, 1, 1), (63, 5, 0), (64, 64, 4), (65, 200, 1),
                                             (129, 7, 70), (300, 100, 4), (300, 1, 0), (513, 128, 128),
                                             (700, 33, 3), (1100, 257, 1)])
def test_attention_lengths_and_windows(mods, T, window, n_sink, d, dtype):
    check_attention(mods[0], T, T, window, n_sink, d=d, dtype=dtype)


@DT
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 2), (8, 1), (5, 1)])
def test_attention_head_groups(mods, H, Hk, dtype):
    check_attention(mods[0], 200, 200, 90, 2, H=H, Hk=Hk, dtype=dtype, d=128)


@DT
@pytest.mark.parametrize("T,S,q_start", [(1, 400, 399), (77, 300, 223), (130, 257, 127), (300, 100, 0),
                                         (64, 128, 500), (40, 640, 0)])
def test_attention_pieces_of_a_prompt(mods, T, S, q_start, dtype):
    """Queries behind keys that are already there, and keys that end before or after them."""
    check_attention(mods[0], T, S, 150, 3, q_start, dtype=dtype, d=128)


@DT
@pytest.mark.parametrize("lens", [[0, 300], [1, 299], [-5, 10**6], [128, 129], [260, 64]])
def test_attention_ragged_batches_and_empty_rows(mods, lens, dtype):
    for n_sink in (0, 4):
        check_attention(mods[0], 300, 300, 60, n_sink, lens=lens, dtype=dtype, d=128)


@DT
@pytest.mark.parametrize("scale", [0.001, 1.0, 3.0])
def test_attention_scales(mods, scale, dtype):
    """Scores of up to about 100: the softmax is one key's, or nearly flat.  (The gradients'
    bound does not hold where exponents carry fp32 errors of that size.)"""
    check_attention(mods[0], 150, 150, 64, 4, scale=scale, dtype=dtype, bwd=scale < 2)


@DT
def test_attention_gradient_against_differences(mods, dtype):
    """The loss' change along a direction of q, k and v: the sum of the gradients' products."""
    attention, _ = mods
    q, k, v, do = qkv(5, 1, 150, 150, 2, 1, 64, dtype)
    out, lse = attention.window_attn_fwd(q, k, v, 40, 3, want_lse=True)
    g = attention.window_attn_bwd(q, k, v, out, lse, do, 40, 3)
    r = np.random.default_rng(3)
    x = [np64(t) for t in (q, k, v)]
    way = [r.normal(size=t.shape) for t in x]
    f = lambda e: (L.window_attention(*[t + e * w for t, w in zip(x, way)], 40, 3)[0] * np64(do)).sum()  # noqa: E731
    slope = (f(1e-5) - f(-1e-5)) / 2e-5
    got = sum((np64(g[n]) * w).sum() for n, w in zip(("dq", "dk", "dv"), way))
    noise = UNIT[dtype] * math.sqrt(sum((np64(g[n]) ** 2).sum() for n in g))   # n independent errors
    assert abs(got - slope) <= 8 * noise + 1e-6 * abs(slope)


def test_attention_on_another_stream_and_in_a_graph(mods):
    attention, _ = mods
    q, k, v, do = qkv(9, 2, 300, 300, 4, 2, 128, torch.bfloat16)
    want, lse = attention.window_attn_fwd(q, k, v, 77, 4, want_lse=True)
    gw = attention.window_attn_bwd(q, k, v, want, lse, do, 77, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = attention.window_attn_fwd(q, k, v, 77, 4, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, l2 = torch.empty_like(want), torch.empty_like(lse)
    grads = {n: torch.empty_like(t) for n, t in gw.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attention.window_attn_fwd(q, k, v, 77, 4, out=out, lse=l2)
        attention.window_attn_bwd(q, k, v, out, l2, do, 77, 4, grads=grads)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(grads[n], gw[n]) for n in gw)


@DT
@pytest.mark.parametrize("window,n_sink,H,Hk,d", [(1, 0, 1, 1, 64), (5, 2, 2, 1, 128), (40, 4, 6, 2, 64),
                                                  (130, 0, 8, 1, 128), (64, 16, 5, 1, 128), (33, 3, 20, 1, 64)])
def test_attention_steps_follow_the_prompt(mods, window, n_sink, H, Hk, d, dtype):
    """A prompt, the ring's fill, then token by token over the ring's end: each step equals
    the row of one long forward."""
    attention, _ = mods
    S, lens = 150, [37, 150, 1]
    B, more = len(lens), 12
    q, k, v, _ = qkv(window, B, S + more, S + more, H, Hk, d, dtype)
    ref, _, size = L.window_attention(np64(q), np64(k), np64(v), window, n_sink)
    kc, vc = (t.fill_(math.nan) for t in attention.window_cache(B, Hk, d, window, n_sink, dtype))
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    attention.window_cache_fill(k, v, kc, vc, window, n_sink, lens=lt)
    for i in range(more):
        row = lambda t: torch.stack([t[b, n + i] for b, n in enumerate(lens)])  # noqa: E731
        out = attention.window_attn_step(row(q), row(k), row(v), kc, vc, lt + i, window, n_sink)
        for b, n in enumerate(lens):
            within(out[b], ref[b, n + i], size[b, n + i], dtype, (i, b))


@DT
@pytest.mark.parametrize("window,G", [(700, 1), (3000, 4), (9000, 3), (2048, 16)])
def test_attention_step_cut_along_the_slots(mods, window, G, dtype):
    """One sequence, a long cache: with and without the workspace; a free place of the batch."""
    attention, _ = mods
    gen = torch.Generator().manual_seed(window)
    B, Hk, d, n_sink = 2, 1, 128, 4
    q, k, v = (randn(gen, B, h, d, dtype=dtype) for h in (G * Hk, Hk, Hk))
    kc, vc = (randn(gen, B, Hk, window + n_sink, d, dtype=dtype) for _ in range(2))
    pos = torch.tensor([3 * window + 11, -1], dtype=torch.int32, device="cuda")
    before = kc.clone(), vc.clone()
    slot = n_sink + (3 * window + 11 - n_sink) % window
    a, b = (t[0, 0].clone() for t in (kc, vc))
    a[slot], b[slot] = k[0, 0], v[0, 0]
    s = np64(q)[0] @ np64(a).T / math.sqrt(d)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    for ws in ("auto", None):
        out = attention.window_attn_step(q, k, v, kc, vc, pos, window, n_sink, workspace=ws)
        within(out[0], p @ np64(b), p @ np.abs(np64(b)), dtype)
        assert (out[1] == 0).all()
    assert torch.equal(kc[1], before[0][1]) and torch.equal(vc[1], before[1][1])
    assert torch.equal(kc[0, 0], a) and torch.equal(vc[0, 0], b)


def test_attention_refuses_what_the_pointers_do_not_say(mods):
    attention, _ = mods
    q, k, v, _ = qkv(1, 2, 16, 16, 4, 2, 64, torch.bfloat16)
    with pytest.raises(TypeError):
        attention.window_attn_fwd(q, k.float(), v, 4)
    with pytest.raises(ValueError):
        attention.window_attn_fwd(q, k, v[:, :8], 4)
    with pytest.raises(ValueError):
        attention.window_attn_fwd(q.transpose(2, 3), k, v, 4)
    with pytest.raises(ValueError):
        attention.window_attn_fwd(q.cpu(), k, v, 4)
    with pytest.raises(TypeError):
        attention.window_attn_fwd(q, k, v, 4, lens=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(RuntimeError):
        attention.window_attn_fwd(q, k, v, 0)


# ------------------------------------------------------------------ short convolution

@DT
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T,D,lens,init,silu", [(1, 8, None, True, True), (2, 7, [2, 0], True, True),
                                                (33, 264, None, False, True), (300, 72, [300, 131], True, False),
                                                (257, 13, [1, 256], True, True), (64, 2056, None, True, True)])
def test_conv(mods, T, D, lens, init, silu, K, dtype):
    _, ssm = mods
    g = torch.Generator().manual_seed(T + K)
    wide = randn(g, 2, T, D + 8, dtype=dtype)
    x = wide[:, :, 8:] if D % 8 == 0 else wide[:, :, 3:3 + D]
    w, bias = randn(g, D, K) / K, randn(g, D)
    s0 = randn(g, 2, K - 1, D, dtype=dtype) if init else None
    dy, de = randn(g, 2, T, D, dtype=dtype), randn(g, 2, K - 1, D, dtype=dtype)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref, end = L.short_conv(np64(x), np64(w), np64(bias), silu, np64(s0), lens)
    y, state = ssm.short_conv_fwd(x, w, bias, silu=silu, init_state=s0, lens=lt)
    close(y, ref, dtype, "y")
    assert np.array_equal(np64(state), end)
    r = L.short_conv_bwd(np64(x), np64(w), np64(bias), np64(dy), silu, np64(s0), np64(de), lens)
    got = ssm.short_conv_bwd(x, w, bias, dy, silu=silu, init_state=s0, d_final_state=de, lens=lt)
    close(got["dx"], r["dx"], dtype, "dx")
    # sums of up to B T fp32 products
    for n in ("dweight", "dbias"):
        np.testing.assert_allclose(np64(got[n]), r[n], atol=2.0 ** -16 * math.sqrt(2 * T) * 4, rtol=2.0 ** -16)
    if init:
        close(got["dinit_state"], r["dinit_state"], dtype, "dinit_state")
    again = ssm.short_conv_bwd(x, w, bias, dy, silu=silu, init_state=s0, d_final_state=de, lens=lt)
    assert all(torch.equal(got[n], again[n]) for n in got)


@DT
@pytest.mark.parametrize("D", [16, 13, 4096])
def test_conv_steps_follow_the_prompt(mods, D, dtype):
    _, ssm = mods
    g = torch.Generator().manual_seed(D)
    x, w, bias = randn(g, 3, 20, D, dtype=dtype), randn(g, D, 4), randn(g, D)
    want, end = ssm.short_conv_fwd(x, w, bias)
    y, state = ssm.short_conv_fwd(x[:, :9], w, bias)
    rows = [y]
    for t in range(9, 20):
        other = torch.empty_like(state)
        o, _ = ssm.short_conv_step(x[:, t], w, bias, state, state_out=other)
        o2, same = ssm.short_conv_step(x[:, t], w, bias, state)
        assert same is state and torch.equal(state, other) and torch.equal(o, o2)
        rows.append(o[:, None])
    assert torch.equal(torch.cat(rows, 1), want) and torch.equal(state, end)
    y, _ = ssm.short_conv_step(x[:, 0], w, None, torch.zeros_like(state), silu=False)
    close(y, np64(x[:, 0]) * np64(w)[:, 3], dtype)


# ------------------------------------------------------------------ selective scan

def scan_inputs(seed, Bn, T, D, N, G, dtype, gated=True, wide=8):
    g = torch.Generator().manual_seed(seed)
    cut = lambda t: t[..., wide:]  # noqa: E731
    x = cut(randn(g, Bn, T, D + wide, dtype=dtype))
    dt = cut(randn(g, Bn, T, D + wide, dtype=dtype))
    z = cut(randn(g, Bn, T, D + wide, dtype=dtype)) if gated else None
    bc = randn(g, Bn, T, 2, G, N, dtype=dtype)
    A = -torch.exp(randn(g, D, N)) * torch.arange(1, N + 1, device="cuda") * 0.3
    return dict(x=x, dt=dt, A=A, B=bc[:, :, 0], C=bc[:, :, 1], D=randn(g, D), z=z, dt_bias=randn(g, D) - 2)


def check_scan(ssm, Bn, T, D, N, G, dtype, gated=True, lens=None, init=True, softplus=True, wide=8, bwd=True):
    s = scan_inputs(T + D + N, Bn, T, D, N, G, dtype, gated, wide)
    if not softplus:
        s["dt"], s["dt_bias"] = s["dt"].abs() * 0.1, None
    g = torch.Generator().manual_seed(1)
    h0 = randn(g, Bn, D, N) if init else None
    dy, de = randn(g, Bn, T, D, dtype=dtype), randn(g, Bn, D, N)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = {n: np64(t) for n, t in s.items()}
    ref, end = L.selective_scan(**o, softplus=softplus, h0=np64(h0), lens=lens)
    for ws in ("auto", None):
        y, state = ssm.selective_scan_fwd(**s, softplus=softplus, init_state=h0, lens=lt, workspace=ws)
        close(y, ref, dtype, "y")
        close(state, end, torch.float32, "state")
    if not bwd:
        return
    r = L.selective_scan_bwd(**o, d_y=np64(dy), softplus=softplus, h0=np64(h0), d_end=np64(de), lens=lens)
    kw = dict(softplus=softplus, init_state=h0, d_final_state=de, lens=lt)
    got = ssm.selective_scan_bwd(**s, d_y=dy, **kw)
    for n in ("dx", "ddt", "dB", "dC") + (("dz",) if gated else ()):
        close(got[n], r[n], dtype, n)
    for n in ("dA", "dD") + (("ddt_bias",) if s["dt_bias"] is not None else ()) + (("dinit_state",) if init else ()):
        close(got[n], r[n], torch.float32, n)
    again = ssm.selective_scan_bwd(**s, d_y=dy, **kw)
    assert all(torch.equal(got[n], again[n]) for n in got)


@DT
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("T,D,G", [(1, 8, 1), (31, 40, 1), (33, 48, 2), (65, 136, 1), (130, 13, 1), (129, 26, 2)])
def test_scan(mods, T, D, G, N, dtype):
    check_scan(mods[1], 2, T, D, N, G, dtype)


@DT
@pytest.mark.parametrize("kw", [dict(gated=False), dict(lens=[100, 0]), dict(lens=[1, 64]), dict(init=False),
                                dict(softplus=False), dict(wide=3), dict(lens=[63, 99], gated=False, wide=1)])
def test_scan_options(mods, kw, dtype):
    check_scan(mods[1], 2, 100, 72, 16, 1, dtype, **kw)


@DT
@pytest.mark.parametrize("T,N", [(1500, 16), (700, 8), (1025, 64)])
def test_scan_of_few_rows_is_cut_along_the_tokens(mods, T, N, dtype):
    from recurrent_associative_memory_gb300 import dr
    a = dr.DrScan(dtype=0, B=1, T=T, D=24, N=N, G=1, softplus=1, A=1 << 20)
    assert dr.dr_selective_scan_fwd_workspace_bytes(a) > 0
    check_scan(mods[1], 1, T, 24, N, 1, dtype, lens=[T - 40], bwd=False)


@DT
@pytest.mark.parametrize("D,N,G", [(24, 16, 2), (13, 8, 1), (40, 64, 1), (520, 32, 1)])
def test_scan_steps_follow_the_prompt(mods, D, N, G, dtype):
    _, ssm = mods
    s = scan_inputs(D, 2, 12, D, N, G, dtype)
    o = {n: np64(t) for n, t in s.items()}
    ref, end = L.selective_scan(**o)
    cut = lambda a, b: {n: (t if n in ("A", "D", "dt_bias") else t[:, a:b]) for n, t in s.items()}  # noqa: E731
    _, state = ssm.selective_scan_fwd(**cut(0, 5))
    for t in range(5, 12):
        one = {n: (v if n in ("A", "D", "dt_bias") else v[:, 0]) for n, v in cut(t, t + 1).items()}
        other = torch.empty_like(state)
        y, _ = ssm.selective_scan_step(**one, state=state, state_out=other)
        y2, same = ssm.selective_scan_step(**one, state=state)
        assert same is state and torch.equal(state, other) and torch.equal(y, y2)
        close(y, ref[:, t], dtype, t)
    close(state, end, torch.float32)


def test_scan_and_conv_refuse_what_the_pointers_do_not_say(mods):
    _, ssm = mods
    s = scan_inputs(0, 2, 8, 16, 16, 1, torch.bfloat16)
    with pytest.raises(TypeError):
        ssm.selective_scan_fwd(**{**s, "A": s["A"].bfloat16()})
    with pytest.raises(ValueError):
        ssm.selective_scan_fwd(**{**s, "B": s["B"][:, :4]})
    with pytest.raises(ValueError):
        ssm.selective_scan_fwd(**{**s, "z": s["z"].cpu()})
    with pytest.raises(TypeError):
        ssm.selective_scan_fwd(**s, lens=torch.tensor([8, 8], device="cuda"))
    with pytest.raises(RuntimeError):
        ssm.selective_scan_fwd(**{**s, "A": s["A"][:, :12].contiguous(), "B": s["B"][..., :12], "C": s["C"][..., :12]})
    with pytest.raises(ValueError):
        ssm.short_conv_fwd(s["x"], torch.zeros(8, 4, device="cuda"))
    with pytest.raises(RuntimeError):
        ssm.short_conv_fwd(s["x"], torch.zeros(16, 5, device="cuda"))
