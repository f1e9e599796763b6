"""The most rows of a matrix product: tiles behind the last row still count in 32 bits."""

import pytest

from test_block_abi_cpu import BIG, FAR, linear
from test_layers_abi_cpu import dr  # noqa: F401

MOST = (1 << 31) - 512


@pytest.mark.parametrize("dtype", ["DR_BF16", "DR_FP32"])
def test_more_rows_are_refused(dr, dtype):  # noqa: F811
    for M in (MOST + 1, MOST + 256, (1 << 31) - 1):
        a = linear(dr, dtype=getattr(dr, dtype), M=M, K=8, N=8)
        assert dr.dr_linear_fwd(a, *FAR[:6], FAR[7], BIG, stream=0) == dr.DR_ERR_SHAPE
        assert dr.dr_linear_bwd(a, *FAR[:7], FAR[8], BIG, stream=0) == dr.DR_ERR_SHAPE
        assert dr.dr_linear_fwd_workspace_bytes(a) == 0 and dr.dr_linear_bwd_workspace_bytes(a) == 0
    a = linear(dr, dtype=getattr(dr, dtype), M=MOST, K=8, N=8, act=2)
    assert dr.dr_linear_bwd_workspace_bytes(a) >= 2 * MOST * 8
