"""The slopes of the matrix product's activations: 1 without one, whichever kernel the sizes choose."""

import pytest
import torch

from test_gpu_block import block, linear_case  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,M,K,N", [(FP, 3, 64, 96), (FP, 100, 64, 96), (FP, 9, 60, 77), (FP, 20000, 32, 2048),
                                         (FP, 20000, 32, 2051), (BF, 3, 64, 96), (BF, 100, 64, 99), (BF, 20000, 32, 2048),
                                         (BF, 20000, 32, 2051)])
def test_slope_without_an_activation_is_one(block, dtype, M, K, N):  # noqa: F811
    """Through the C entry point: for few rows, small products and pairs of CTAs, rows on 32 bytes or not."""
    from recurrent_associative_memory_gb300 import dr
    c = linear_case(M, M, K, N, dtype)
    a = dr.DrLinear(int(dtype is BF), 0, M, K, N, 0, K, N, N)
    n = dr.dr_linear_fwd_workspace_bytes(a)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    y, plain = torch.empty_like(c["residual"]), torch.empty_like(c["residual"])
    slope = torch.full((M, N), 7, dtype=torch.float16 if dtype is BF else FP, device="cuda")
    for out, s in ((plain, None), (y, slope)):
        dr.check(dr.dr_linear_fwd(a, c["x"], c["w"], c["bias"], c["residual"], out, s, ws, n), "dr_linear_fwd")
    assert bool((slope == 1).all()) and torch.equal(y, plain)
