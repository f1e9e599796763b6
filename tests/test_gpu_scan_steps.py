"""The scan's time step by itself: with one token, x = B = 1 and no state before it, the state
is dt = softplus(raw).  fp32: the exponential and the logarithm of the type, two units of 2^-23
each at most.  bf16, whose raw values are good to 2^-9: 2^-18 from the approximate logarithm
(absolute 2^-22 against log(17/16) > 2^-4.1), within 2^-17 with the exponential's part."""

import numpy as np
import pytest
import torch

from test_gpu_layers import DT, mods, np64  # noqa: F401

pytestmark = pytest.mark.gpu
BOUND = {torch.float32: 2.0 ** -21, torch.bfloat16: 2.0 ** -17}


def raws(dtype):
    """Around e^-|v| = 1/16, where the forms meet, and over the rest of the range."""
    near = torch.linspace(2.7, 2.85, 1024)
    wide = torch.linspace(0.0, 12.0, 1024)
    return torch.cat([near, -near, wide, -wide]).to(dtype).cuda()


def check(dt, raw, dtype):
    want = np.logaddexp(0.0, np64(raw))
    off = np.abs(np64(dt) - want) / want
    assert off.max() <= BOUND[dtype], (off.max(), np64(raw)[off.argmax()])


@DT
@pytest.mark.parametrize("N", [8, 16])
def test_time_steps(mods, N, dtype):  # noqa: F811
    _, ssm = mods
    raw = raws(dtype)
    D = raw.numel()
    A, one = -torch.ones(D, N, device="cuda"), torch.ones(1, 1, 1, N, dtype=dtype, device="cuda")
    x = torch.ones(1, 1, D, dtype=dtype, device="cuda")
    _, state = ssm.selective_scan_fwd(x, raw[None, None], A, one, one)
    check(state[0, :, N - 1], raw, dtype)
    _, state = ssm.selective_scan_step(x[0], raw[None], A, one[0], one[0], torch.zeros_like(state))
    check(state[0, :, 0], raw, dtype)


@pytest.mark.parametrize("N", [8, 16])
def test_time_steps_of_the_backward(mods, N):  # noqa: F811
    """One channel, a sequence per value: dB = dy C dt x = dt."""
    _, ssm = mods
    raw = raws(torch.float32)
    n = raw.numel()
    one = torch.ones(n, 1, 1, N, device="cuda")
    x = torch.ones(n, 1, 1, device="cuda")
    g = ssm.selective_scan_bwd(x, raw[:, None, None], -torch.ones(1, N, device="cuda"), one, one, torch.ones_like(x))
    # g B dt, summed over the one channel and its neighbours' zeros
    check(g["dB"][:, 0, 0, N - 1], raw, torch.float32)
