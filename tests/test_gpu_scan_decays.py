"""The scan's decays by themselves: with x = 0 a state is the initial one times the product of
exp(dt A) over the tokens.  Over exponents of -0.4 to -0.005 in base 2 a decay may be 2^-27 off on
average, which adds up, and 2^-24 at random with its product's rounding, whose sum grows as the
root: after T tokens T 2^-27 + sqrt(T) 2^-24."""

import numpy as np
import pytest
import torch

from test_gpu_layers import DT, mods, np64  # noqa: F401

pytestmark = pytest.mark.gpu


@DT
@pytest.mark.parametrize("T,N", [(200, 16), (60, 8), (1000, 32)])
def test_products_of_decays(mods, T, N, dtype):  # noqa: F811
    _, ssm = mods
    g = torch.Generator().manual_seed(T)
    D, span = 512, 16.0 / T            # exponents of about 100 / T on average, at most
    x = torch.zeros(1, T, D, dtype=dtype, device="cuda")
    dt = (torch.rand(1, T, D, generator=g) * 0.9 + 0.1).to(dtype).cuda()
    A = -(torch.rand(D, N, generator=g) + 0.5).cuda() * min(0.26, span)
    one = torch.ones(1, T, 1, N, dtype=dtype, device="cuda")
    h0 = torch.ones(1, D, N, device="cuda")
    want = np.exp(np64(dt).sum(1)[0][:, None] * np64(A))
    bound = T * 2.0 ** -27 + T ** 0.5 * 2.0 ** -24
    _, state = ssm.selective_scan_fwd(x, dt, A, one, one, softplus=False, init_state=h0, workspace=None)
    off = np64(state)[0] / want - 1
    assert np.sqrt((off ** 2).mean()) <= bound, np.sqrt((off ** 2).mean())
    state = h0
    for t in range(T):
        _, state = ssm.selective_scan_step(x[:, t], dt[:, t], A, one[:, t], one[:, t], state, softplus=False)
    off = np64(state)[0] / want - 1
    assert np.sqrt((off ** 2).mean()) <= bound, np.sqrt((off ** 2).mean())


@DT
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_a_state_that_does_not_decay_stays_as_it_is(mods, N, dtype):  # noqa: F811
    """dt = 0, and rates of 0: bit for bit over a thousand tokens, forward and step."""
    _, ssm = mods
    g = torch.Generator().manual_seed(N)
    T, D = 1000, 40
    x = torch.zeros(2, T, D, dtype=dtype, device="cuda")
    bc = torch.ones(2, T, 1, N, dtype=dtype, device="cuda")
    h0 = torch.randn(2, D, N, generator=g).cuda()
    for dt, A in ((0.0, -1.0), (0.7, 0.0)):
        dts, rates = torch.full_like(x, dt), torch.full((D, N), A, device="cuda")
        for ws in ("auto", None):
            _, state = ssm.selective_scan_fwd(x, dts, rates, bc, bc, softplus=False, init_state=h0, workspace=ws)
            assert torch.equal(state, h0)
        state = h0.clone()
        for t in range(5):
            ssm.selective_scan_step(x[:, t], dts[:, t], rates, bc[:, t], bc[:, t], state, softplus=False)
        assert torch.equal(state, h0)
