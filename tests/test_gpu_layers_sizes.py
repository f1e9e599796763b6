"""GPU parity of the layers next to the recurrence where a size changes how a kernel works:
several pieces per warp, whole row blocks, what stands behind a sequence's end, and how far
the gradients' norms are off.  Bounds as in test_gpu_layers."""

import math

import numpy as np
import pytest
import torch

from oracle import layers as L
from test_gpu_layers import DT, check_attention, check_scan, mods, np64, qkv, randn, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@DT
@pytest.mark.parametrize("D,G", [(512, 64), (64, 64)])   # 16-byte rows, single values
def test_scan_backward_of_many_pieces(mods, D, G, dtype):  # noqa: F811
    """64 channel tiles x 41 pieces: more than eight CTAs on each of up to 152 SMs, twice over."""
    check_scan(mods[1], 1, 1300, D, 8, G, dtype, lens=[1290])


@DT
@pytest.mark.parametrize("d", [64, 128])
def test_attention_of_many_row_blocks(mods, d, dtype):  # noqa: F811
    """4 x 8 heads x 6 blocks of 64 rows: no SM without one."""
    check_attention(mods[0], 333, 333, 100, 4, lens=[333, 200, 1, 0], H=8, Hk=2, d=d, dtype=dtype, B=4)


@DT
@pytest.mark.parametrize("wide", [8, 3])
def test_scan_never_looks_behind_the_end(mods, wide, dtype):  # noqa: F811
    ssm = mods[1]
    lens = torch.tensor([40, 0, 97], dtype=torch.int32, device="cuda")
    s = scan_inputs(5, 3, 97, 72, 16, 1, dtype, wide=wide)
    dy = randn(torch.Generator().manual_seed(6), 3, 97, 72, dtype=dtype)
    past = torch.arange(97, device="cuda")[None] >= lens[:, None]
    results = []
    for fill in (0.0, math.nan, math.inf):
        for n in ("x", "dt", "z", "B", "C"):
            s[n][past] = fill
        dy[past] = fill
        y, end = ssm.selective_scan_fwd(**s, lens=lens)
        g = ssm.selective_scan_bwd(**s, d_y=dy, lens=lens)
        results.append([y, end, *(g[n] for n in sorted(g) if g[n] is not None)])
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for r in results[1:] for a, b in zip(results[0], r))


@DT
@pytest.mark.parametrize("D", [64, 33])
def test_conv_never_looks_behind_the_end(mods, D, dtype):  # noqa: F811
    ssm = mods[1]
    lens = torch.tensor([70, 0, 2, 130], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(7)
    x, dy = randn(g, 4, 130, D, dtype=dtype), randn(g, 4, 130, D, dtype=dtype)
    w, bias = randn(g, D, 4), randn(g, D)
    past = torch.arange(130, device="cuda")[None] >= lens[:, None]
    results = []
    for fill in (0.0, math.nan, math.inf):
        x[past], dy[past] = fill, fill
        y, end = ssm.short_conv_fwd(x, w, bias, lens=lens)
        grads = ssm.short_conv_bwd(x, w, bias, d_y=dy, lens=lens)
        results.append([y, end, *(grads[n] for n in sorted(grads) if grads[n] is not None)])
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for r in results[1:] for a, b in zip(results[0], r))


@pytest.mark.parametrize("T,window,n_sink,d", [(400, 64, 4, 128), (150, 16, 0, 64), (64, 8, 1, 128)])
def test_attention_gradients_are_little_further_off_than_their_rounding(mods, T, window, n_sink, d):  # noqa: F811
    """A bf16 result is off by 2^-9 of itself at most.  delta, taken from an O of that precision,
    adds less than half of that by norm, dS in two bf16 2^-17: dQ and dK keep 1.25 x 2^-9.
    dV takes a P of one bf16 besides its own rounding: sqrt(2) x 2^-9."""
    q, k, v, do = qkv(T, 2, T, T, 4, 2, d, torch.bfloat16)
    _, _, _, grads, _ = L.window_attention(np64(q), np64(k), np64(v), window, n_sink, 0, None, None, d_out=np64(do))
    out, lse = mods[0].window_attn_fwd(q, k, v, window, n_sink, want_lse=True)
    g = mods[0].window_attn_bwd(q, k, v, out, lse, do, window, n_sink)
    for name, most in (("dq", 1.25), ("dk", 1.25), ("dv", 2 ** 0.5)):
        off = np.linalg.norm(np64(g[name]) - grads[name]) / np.linalg.norm(grads[name])
        assert off < most * 2.0 ** -9, (name, off)


def test_scratch_of_a_call_on_another_stream_is_left_alone(mods):  # noqa: F811
    """While a call waits on a busy stream, the current stream allocates and overwrites blocks
    of every size that the call took: its results are those of a quiet call."""
    attention, ssm = mods
    q, k, v, do = qkv(3, 2, 300, 300, 4, 2, 128, torch.bfloat16)
    s = scan_inputs(4, 1, 1500, 24, 16, 1, torch.bfloat16)
    dy = randn(torch.Generator().manual_seed(5), 1, 1500, 24, dtype=torch.bfloat16)
    out, lse = attention.window_attn_fwd(q, k, v, 40, 4, want_lse=True)

    def work(stream):
        g = attention.window_attn_bwd(q, k, v, out, lse, do, 40, 4, stream=stream)
        y, end = ssm.selective_scan_fwd(**s, stream=stream)
        r = ssm.selective_scan_bwd(**s, d_y=dy, stream=stream)
        return [*(g[n] for n in sorted(g)), y, end, *(r[n] for n in sorted(r) if r[n] is not None)]

    want = [t.clone() for t in work(None)]
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for side in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        stream = side if isinstance(side, torch.cuda.Stream) else torch.cuda.ExternalStream(side)
        with torch.cuda.stream(stream):
            for _ in range(60):
                busy = busy @ busy * 1e-4
        got = work(side)
        taken = [torch.full((n,), math.nan, device="cuda") for n in [2 ** i for i in range(7, 20)] * 4]
        torch.cuda.synchronize()
        assert taken and all(torch.equal(a, b) for a, b in zip(got, want))
