"""Window attention, backward in bf16: scores of many steps pass through the same columns of
tensor memory.  Every tile of queries and of keys has a size of its own, so that scores which
replaced those of an earlier step, or were replaced by a later one's, show.  Bounds as in
test_gpu_layers."""

import pytest
import torch

from oracle import layers as L
from test_gpu_layers import mods, np64, qkv, within  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,window,n_sink,H,Hk", [(900, 900, 0, 4, 1), (640, 200, 100, 2, 2)])
def test_scores_of_many_steps_keep_apart(mods, T, window, n_sink, H, Hk, d):  # noqa: F811
    q, k, v, do = qkv(T + d, 2, T, T, H, Hk, d, BF)
    step = torch.arange(T, device="cuda") // 64
    q, k, v, do = (t * (1.0 + n * (step % m)).to(BF)[None, :, None, None]
                   for t, m, n in ((q, 3, 0.25), (k, 5, 0.125), (v, 4, 0.5), (do, 7, 0.25)))
    ref, _, size, grads, sizes = L.window_attention(np64(q), np64(k), np64(v), window, n_sink, d_out=np64(do))
    out, lse = mods[0].window_attn_fwd(q, k, v, window, n_sink, want_lse=True)
    within(out, ref, size, BF, "out")
    first = mods[0].window_attn_bwd(q, k, v, out, lse, do, window, n_sink)
    for name in ("dq", "dk", "dv"):
        within(first[name], grads[name], sizes[name], BF, name)
    for _ in range(20):
        again = mods[0].window_attn_bwd(q, k, v, out, lse, do, window, n_sink)
        assert all(torch.equal(first[n], again[n]) for n in first)
