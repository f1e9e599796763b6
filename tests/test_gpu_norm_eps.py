"""The norms around a block with an eps of 0: rows that hold something have finite norms, and the
places of a block behind the last row add nothing to the sums over the rows."""

import pytest

from test_gpu_block import TYPES, block, check_norm, norm_case  # noqa: F401

pytestmark = pytest.mark.gpu


@TYPES
@pytest.mark.parametrize("M,D", [(1, 24), (5, 8), (3, 72), (333, 24), (7, 200), (2, 255), (9, 256), (3, 333), (5, 1000)])
def test_norm_without_eps(block, M, D, dtype, h_dtype):  # noqa: F811
    """Short rows share a block, whose last one may not be full."""
    check_norm(block, *norm_case(M + D, M, D, dtype, h_dtype), eps=0.0)
    check_norm(block, *norm_case(M, M, D, dtype, h_dtype, gate=False, post=False), post=False, eps=0.0)
