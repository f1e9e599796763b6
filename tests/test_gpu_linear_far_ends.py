"""fp32 to its own precision far from zero, whichever kernel the sizes choose: SiLU's tails and their
slopes, large and tiny values."""

import numpy as np
import pytest
import torch

from oracle import block as O
from test_gpu_block import block, np64  # noqa: F401

pytestmark = pytest.mark.gpu
SIZES = pytest.mark.parametrize("M,N", [(4, 64), (300, 64), (300, 67), (20000, 2048), (20000, 2051)])


def far_ends(N):
    v = torch.tensor([-1e30, -200.0, -104.0, -89.0, -88.0, -87.0, -86.0, -80.0, -60.0, -45.0, -31.0, -30.0, -29.0, -17.0, -8.0,
                      -4.5, -1.0, -1e-20, 0.0, 1e-30, 0.5, 3.0, 20.0, 29.0, 31.0, 87.0, 89.0, 1e10, 3e38])
    return v.repeat(N // len(v) + 1)[:N][None].cuda()


@SIZES
def test_silu_far_ends_in_fp32(block, M, N):  # noqa: F811
    """One product is the sum, off by 2^-23 at most, and so is the exponent of the sigmoid: 2^-22
    |x| of the result, and 2^-21 for the operations around it, taken twice.  From -4 on the terms
    of the slope cancel: 2^-20.  A sigmoid below fp32's normal values (from -87.3 on) is 0."""
    w = far_ends(N)
    x = torch.ones(M, 1, device="cuda")
    y, s = block.linear_fwd(x, w, act="silu", want_slope=True)
    pre = np64(w)
    ref, slope = O.act("silu", pre)
    rel = np.where(np.abs(pre) < 100, (np.abs(pre) + 2) * 2.0 ** -21, 2.0 ** -21)
    for got, want, near in ((y, ref, 0.0), (s, slope, 2.0 ** -20 * (pre > -4))):
        bad = ~(np.abs(np64(got) - want) <= rel * np.abs(want) + near + 2e-36)
        assert not bad.any(), (np.broadcast_to(pre, bad.shape)[bad][:8], np64(got)[bad][:8], np.broadcast_to(want, bad.shape)[bad][:8])


@SIZES
def test_large_and_tiny_values_in_fp32(block, M, N):  # noqa: F811
    """Three pieces and six products of them keep fp32's precision from 2^-100 to bf16's largest."""
    w = torch.cat((far_ends(N - 7), torch.tensor([[2.0 ** -100, -1e-29, 3e-25, -7.7e-15, 1.1e20, -2.9e37, 3.3e38]]).cuda()), 1)
    x = torch.tensor([1.0, -0.7, 0.33333334, -1.0]).cuda().repeat(M // 4)[:, None].contiguous()
    y, _ = block.linear_fwd(x, w)
    ref = np64(x) @ np64(w)
    bad = ~(np.abs(np64(y) - ref) <= (2 * 3 + 16) * 2.0 ** -24 * np.abs(ref))
    assert not bad.any(), (ref[bad][:8], np64(y)[bad][:8])
