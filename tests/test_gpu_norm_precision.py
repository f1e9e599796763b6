"""The norms around a block in fp32, to a few steps of 2^-24.

In units of 2^-24: a sum of squares has a rounding for each square and at most 24 additions in a
row (8 within a thread, or 12 with 16 columns, 5 in a warp, 7 over 16 warps), all of one sign; its
mean and eps two more.  A root halves that, and the reciprocal root is off by 4 (2 steps): 18 for
rstd.  The branch's norm takes it and three more roundings on its way into h', which is rounded
once: 21 (|h| + |scale u|) = 21 A.  y = h' (rstd w) has that, the same again through the mean of
squares, rstd's 18 and two roundings."""

import numpy as np
import pytest
import torch

from oracle import block as O
from test_gpu_block import ROWS, block, norm_case, np64  # noqa: F401

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


@pytest.mark.parametrize("M,D", ROWS)
def test_norms_in_fp32(block, M, D):  # noqa: F811
    c, _ = norm_case(M + D, M, D, torch.float32, torch.float32, gate=False)
    y, h = block.block_norm_fwd(**c, post_norm=True)
    n = {k: np64(v) for k, v in c.items()}
    want_y, want_h = O.block_norm(**n, post_norm=True, eps=1e-6)
    A = np.abs(n["h"]) + np.abs(want_h - n["h"])
    assert (np.abs(np64(h) - want_h) <= 21 * STEP * A).all()
    r = O.rstd(want_h, 1e-6)
    rms = np.sqrt((A * A).mean(-1, keepdims=True))
    bound = STEP * np.abs(n["pre_weight"]) * r * (21 * A + np.abs(want_h) * (21 * r * rms + 20))
    assert (np.abs(np64(y) - want_y) <= bound + 1e-30).all()
