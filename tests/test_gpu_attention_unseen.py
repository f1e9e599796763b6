"""Window attention over buffers of keys and values that reach beyond the last query, as a cache
that a prompt fills piece by piece does: what lies there is never looked at."""

import math

import pytest
import torch

from oracle import layers as L
from test_gpu_layers import DT, mods, np64, qkv, within  # noqa: F401

pytestmark = pytest.mark.gpu


@DT
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,S,q_start,lens", [(64, 300, 100, None), (1, 200, 0, None), (130, 640, 77, None),
                                              (200, 512, 250, [512, 300]), (300, 301, 0, [301, 299])])
def test_keys_behind_the_last_query_are_never_looked_at(mods, T, S, q_start, lens, d, dtype):  # noqa: F811
    attention, window, n_sink = mods[0], 60, 4
    q, k, v, do = qkv(T + S, 2, T, S, 4, 2, d, dtype)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(q_start=q_start, lens=lt)
    ref, _, size, grads, sizes = L.window_attention(np64(q), np64(k), np64(v), window, n_sink, q_start, lens,
                                                    d_out=np64(do))
    results = []
    for fill in (0.0, math.nan, math.inf):
        k[:, q_start + T:], v[:, q_start + T:] = fill, fill
        out, lse = attention.window_attn_fwd(q, k, v, window, n_sink, want_lse=True, **kw)
        g = attention.window_attn_bwd(q, k, v, out, lse, do, window, n_sink, **kw)
        results.append([out, lse, g["dq"], g["dk"], g["dv"]])
    within(results[0][0], ref, size, dtype, "out")
    for name, got in zip(("dq", "dk", "dv"), results[0][2:]):
        within(got, grads[name], sizes[name], dtype, name)
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(results[0], r))
    assert not results[0][3][:, q_start + T:].any() and not results[0][4][:, q_start + T:].any()
