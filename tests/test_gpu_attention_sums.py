"""Window attention in fp32: what long sums leave of the type's precision.  With u = 2^-24, n
terms of either sign added one after the other leave an error of about sqrt(n / 6) u by norm; in
tiles of 64, sqrt(64 / 6) u and sqrt(n / 64 / 6) u of the tiles' sums: 3.9 u at n = 1640, 4.6 u
at n = 4085 (keys that every row sees).  With about 3 u of the probabilities and the result:
less than 8 u."""

import numpy as np
import pytest
import torch

from oracle import layers as L
from test_gpu_layers import mods, np64, qkv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,window,n_sink,H,Hk", [(817, 328, 4, 5, 1), (356, 266, 16, 16, 2), (817, 20, 100, 5, 1)])
def test_gradients_of_keys_that_many_rows_see(mods, T, window, n_sink, H, Hk, d):  # noqa: F811
    q, k, v, do = qkv(T + d, 1, T, T, H, Hk, d, torch.float32)
    grads = L.window_attention(np64(q), np64(k), np64(v), window, n_sink, d_out=np64(do))[3]
    out, lse = mods[0].window_attn_fwd(q, k, v, window, n_sink, want_lse=True)
    g = mods[0].window_attn_bwd(q, k, v, out, lse, do, window, n_sink)
    for name in ("dk", "dv"):
        off = np.linalg.norm(np64(g[name]) - grads[name]) / np.linalg.norm(grads[name])
        assert off < 8 * 2.0 ** -24, (name, off)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,S,H", [(16, 4016, 4), (200, 3000, 16)])
def test_rows_that_see_many_keys(mods, T, S, H, d):  # noqa: F811
    """4.6 u of the sums at 4016 keys; one after the other 26."""
    q, k, v, _ = qkv(T + d, 1, T, S, H, 1, d, torch.float32)
    want = L.window_attention(np64(q), np64(k), np64(v), S, 0, S - T)[0]
    out, _ = mods[0].window_attn_fwd(q, k, v, S, 0, q_start=S - T)
    off = np.linalg.norm(np64(out) - want) / np.linalg.norm(want)
    assert off < 8 * 2.0 ** -24, off


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_of_rows_that_see_many_keys(mods, d):  # noqa: F811
    """Up to 2000 keys: 4.0 u of the sums, one after the other 18."""
    q, k, v, do = qkv(d, 1, 2000, 2000, 1, 1, d, torch.float32)
    grads = L.window_attention(np64(q), np64(k), np64(v), 2000, 0, d_out=np64(do))[3]
    out, lse = mods[0].window_attn_fwd(q, k, v, 2000, 0, want_lse=True)
    g = mods[0].window_attn_bwd(q, k, v, out, lse, do, 2000, 0)
    late = slice(1000, None)       # rows that see many
    off = np.linalg.norm(np64(g["dq"])[:, late] - grads["dq"][:, late]) / np.linalg.norm(grads["dq"][:, late])
    assert off < 8 * 2.0 ** -24, off
