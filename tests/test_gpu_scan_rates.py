"""The scan's time step in the bf16 type where its fp32 part, the bias, decides: with raw values of
0 and a bias per channel, dt is softplus(bias).  For |bias| <= 4: the exponent is 4 log2(e) 2^-24
off, the exponential 2^-22, the logarithm's series 2^-22.  dt's error goes into the state (fp32)
and into dA (fp32) in full: within 2^-21 and, with dA's other factors, 2^-20."""

import numpy as np
import pytest
import torch

from oracle import layers as L
from test_gpu_layers import DT, mods, np64, randn, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@DT
def test_time_steps_of_a_bias(mods, dtype):  # noqa: F811
    _, ssm = mods
    bias = torch.cat([torch.linspace(-4, 4, 2048), torch.linspace(-2.85, -2.7, 2048)]).cuda()
    D, N = bias.numel(), 8
    A, one = -torch.ones(D, N, device="cuda"), torch.ones(1, 1, 1, N, dtype=dtype, device="cuda")
    x, raw = torch.ones(1, 1, D, dtype=dtype, device="cuda"), torch.zeros(1, 1, D, dtype=dtype, device="cuda")
    want = np.logaddexp(0.0, np64(bias))
    _, state = ssm.selective_scan_fwd(x, raw, A, one, one, dt_bias=bias)
    off = np.abs(np64(state)[0, :, 0] - want) / want
    assert off.max() <= 2.0 ** -21, (off.max(), np64(bias)[off.argmax()])
    _, state = ssm.selective_scan_step(x[0], raw[0], A, one[0], one[0], torch.zeros_like(state), dt_bias=bias)
    off = np.abs(np64(state)[0, :, 0] - want) / want
    assert off.max() <= 2.0 ** -21, (off.max(), np64(bias)[off.argmax()])


@DT
@pytest.mark.parametrize("T,D,bias", [(3, 20, -2.7648), (9, 17, -2.71), (33, 40, -2.5)])
def test_rates(mods, T, D, bias, dtype):  # noqa: F811
    _, ssm = mods
    s = scan_inputs(T, 1, T, D, 16, 1, dtype)
    s["dt"] = torch.zeros_like(s["x"])
    s["dt_bias"] = torch.full((D,), bias, device="cuda")
    dy = randn(torch.Generator().manual_seed(T), 1, T, D, dtype=dtype)
    want = L.selective_scan_bwd(**{n: np64(t) for n, t in s.items()}, d_y=np64(dy))["dA"]
    got = ssm.selective_scan_bwd(**s, d_y=dy)["dA"]
    off = np.linalg.norm(np64(got) - want) / np.linalg.norm(want)
    assert off < 2.0 ** -20, off
