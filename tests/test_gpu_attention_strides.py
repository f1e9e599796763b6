"""Window attention in bf16 over tensors whose strides no tensor map holds (expanded ones, stride
0): the CUDA-core kernels take them.  Bounds as in test_gpu_layers."""

import pytest
import torch

from oracle import layers as L
from test_gpu_layers import DT, mods, np64, qkv, within  # noqa: F401

pytestmark = pytest.mark.gpu


@DT
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["batch", "heads", "tokens", "queries"])
def test_expanded_tensors(mods, which, d, dtype):  # noqa: F811
    attention, (B, T, H, Hk), window, n_sink = mods[0], (2, 170, 4, 2), 50, 3
    q, k, v, do = qkv(d, B, T, T, H, Hk, d, dtype)
    if which == "batch":      # a prefix that every sequence shares
        k, v = (t[:1].expand(B, T, Hk, d) for t in (k, v))
    elif which == "heads":
        k, v = (t[:, :, :1].expand(B, T, Hk, d) for t in (k, v))
    elif which == "tokens":
        v = v[:, :1].expand(B, T, Hk, d)
    else:
        q = q[:, :, :1].expand(B, T, H, d)
    lens = torch.tensor([T, 90], dtype=torch.int32, device="cuda")
    ref, _, size, grads, sizes = L.window_attention(np64(q), np64(k), np64(v), window, n_sink, 0, [T, 90],
                                                    d_out=np64(do))
    out, lse = attention.window_attn_fwd(q, k, v, window, n_sink, lens=lens, want_lse=True)
    within(out, ref, size, dtype, "out")
    g = attention.window_attn_bwd(q, k, v, out, lse, do, window, n_sink, lens=lens)
    for name in ("dq", "dk", "dv"):
        within(g[name], grads[name], sizes[name], dtype, name)


def test_expanded_keys_in_the_ring_fill(mods):  # noqa: F811
    attention = mods[0]
    _, k, v, _ = qkv(3, 2, 100, 100, 2, 2, 64, torch.bfloat16)
    a, b = attention.window_cache(2, 2, 64, 40, 4), attention.window_cache(2, 2, 64, 40, 4)
    attention.window_cache_fill(k[:1].expand_as(k), v[:, :, :1].expand_as(v), *a, 40, 4)
    attention.window_cache_fill(k[:1].repeat(2, 1, 1, 1), v[:, :, :1].repeat(1, 1, 2, 1), *b, 40, 4)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
