"""The matrix product where one pair of CTAs walks several tiles and the last tiles of rows are
ragged, so that lanes without a row are through with a tile before the others."""

import pytest

from test_gpu_block import DT, block, check_linear, linear_case  # noqa: F401

pytestmark = pytest.mark.gpu


@DT
@pytest.mark.parametrize("M,N", [(5129, 4112), (5343, 4096), (5129, 4099)])
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
def test_a_bias_of_its_own_for_every_tile(block, M, N, act, dtype):  # noqa: F811
    c = linear_case(M + N, M, 40, N, dtype)
    c["bias"] *= 100   # another tile's would be far off
    check_linear(block, c, act, bwd=False)
