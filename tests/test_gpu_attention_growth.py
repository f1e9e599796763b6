"""Window attention, forward, where the scores grow from key tile to key tile: the reference of
a row's exponentials is raised, and what was summed before is rescaled.  Bounds as in
test_gpu_layers."""

import math

import numpy as np
import pytest
import torch

from oracle import layers as L
from test_gpu_layers import mods, np64, within  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rising(T, d, bits, scale, seed):
    """q [1,T,2,d], k, v [1,T,1,d].  Query row i lies along direction i % len(bits[0]); the keys
    of tile n (128 each) raise the scores of the rows along direction r by bits[n][r], in base 2.
    Everything else is noise of about one bit."""
    g = torch.Generator().manual_seed(seed)
    ways = len(bits[0])
    size = math.sqrt(math.log(2) / scale)
    q, k = (torch.randn(1, T, h, d, generator=g) * size / d ** 0.25 for h in (2, 1))
    v = torch.randn(1, T, 1, d, generator=g)
    q[..., :ways], k[..., :ways] = 0.0, 0.0
    for i in range(T):
        q[:, i, :, i % ways] = 4 * size
        for r in range(ways):
            k[:, i, :, r] = bits[min(i // 128, len(bits) - 1)][r] / 4 * size
    return [t.to(BF).cuda() for t in (q, k, v)]


def check(attention, q, k, v, window, n_sink, scale):
    want, lse_ref, size = L.window_attention(np64(q), np64(k), np64(v), window, n_sink, scale=scale)
    out, lse = attention.window_attn_fwd(q, k, v, window, n_sink, scale=scale, want_lse=True)
    within(out, want, size, BF, "out")
    # scores are sums of d fp32 products that add up to at most 2^8
    np.testing.assert_allclose(np64(lse), lse_ref, atol=2.0 ** 8 * 2.0 ** -16, rtol=1e-5)
    again, _ = attention.window_attn_fwd(q, k, v, window, n_sink, scale=scale)
    assert torch.equal(again, out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,n_sink", [(640, 0), (512, 4)])
@pytest.mark.parametrize("bits", [
    [(0, 0), (20, 0), (20, 100)],                   # odd rows jump where even ones have just grown
    [(0, 0), (20, 0), (20, 100), (50, 100), (50, 200)],
    [(0, 0, 0), (12, 0, 9), (24, 80, 18), (36, 80, 100)]], ids=["twice", "again", "three"])
def test_rows_of_a_warp_that_grow_and_jump(mods, bits, window, n_sink, d):  # noqa: F811
    """Some rows' maxima grow by 2^9 to 2^30 in one key tile, others' of the same warp by more
    than 2^64 in the next: both rescale the sums, one after the other."""
    q, k, v = rising(700, d, bits, 3.0, seed=len(bits) + d)
    check(mods[0], q, k, v, window, n_sink, 3.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [[(0, 0), (40, 60)], [(0, 0), (7, 3), (14, 11), (50, 19), (56, 80)]])
def test_large_values_behind_a_jump_of_the_scores_stay_finite(mods, bits, d):  # noqa: F811
    """Values of about 2^112: what is summed stays below 2^128 as long as no probability passes
    1 by much, whatever the scores do."""
    q, k, v = rising(600, d, bits, 3.0, seed=d)
    check(mods[0], q, k, v * 2.0 ** 112, 600, 0, 3.0)
