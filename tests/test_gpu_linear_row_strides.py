"""The matrix product where a row stride decides how its operands are read: fp32 weights of a few
rows' product on 16 bytes or not, and rows that overlap."""

import pytest
import torch

from test_gpu_block import DT, block, check_linear, linear_case, randn  # noqa: F401

pytestmark = pytest.mark.gpu
FP = torch.float32


@pytest.mark.parametrize("M", [1, 3, 8])
@pytest.mark.parametrize("K,N", [(64, 96), (520, 133)])
def test_few_rows_of_any_weight(block, M, K, N):  # noqa: F811
    """CUDA cores take weights whose rows stand on 16 bytes, tensor cores the others: both within
    the bounds."""
    c = linear_case(M + N, M, K, N, FP)
    for extra in (1, 2, 3, 4):
        wide = torch.full((K, N + extra), float("nan"), device="cuda")
        wide[:, :N] = c["w"]
        check_linear(block, dict(c, w=wide[:, :N]), "silu")
        tall = torch.full((N, K + extra), float("nan"), device="cuda")
        tall[:, :K] = c["w"].t()
        check_linear(block, dict(c, w=tall[:, :K].t()), "silu")


@DT
@pytest.mark.parametrize("M,step", [(5, 8), (5, 3), (130, 8), (130, 1), (2600, 24), (2600, 7)])
def test_overlapping_rows(block, M, step, dtype):  # noqa: F811
    """Windows over one signal: each row begins ``step`` values behind the one before."""
    K, N = 64, 72
    c = linear_case(M, M, K, N, dtype)
    signal = randn(torch.Generator().manual_seed(step), (M - 1) * step + K, dtype=dtype)
    x = signal.as_strided((M, K), (step, 1))
    check_linear(block, dict(c, x=x), "silu")
