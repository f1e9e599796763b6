"""States that are taken on in place: a prompt's final state written over its initial one."""

import pytest
import torch

from test_gpu_layers import DT, mods, np64, randn, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@DT
@pytest.mark.parametrize("K", [2, 4])
@pytest.mark.parametrize("T,lens", [(1, None), (130, None), (700, None), (200, [200, 3, 0]), (150, [1, 2, 150])])
def test_conv_takes_its_state_on_in_place(mods, T, lens, K, dtype):  # noqa: F811
    """Runs of tokens that other threads walk must not meet the new state in place of the old."""
    _, ssm = mods
    g = torch.Generator().manual_seed(T + K)
    for D in (2048, 33):
        x, w, s0 = randn(g, 3, T, D, dtype=dtype), randn(g, D, K), randn(g, 3, K - 1, D, dtype=dtype)
        lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        want, end = ssm.short_conv_fwd(x, w, init_state=s0, lens=lt)
        for _ in range(10):
            state = s0.clone()
            y, same = ssm.short_conv_fwd(x, w, init_state=state, final_state=state, lens=lt)
            assert same is state and torch.equal(y, want) and torch.equal(state, end)


@DT
@pytest.mark.parametrize("T,D,N", [(1500, 24, 16), (90, 40, 8), (65, 2048, 16)])
def test_scan_takes_its_state_on_in_place(mods, T, D, N, dtype):  # noqa: F811
    _, ssm = mods
    s = scan_inputs(T, 2, T, D, N, 1, dtype)
    h0 = randn(torch.Generator().manual_seed(2), 2, D, N)
    for ws in ("auto", None):
        want, end = ssm.selective_scan_fwd(**s, init_state=h0, workspace=ws)
        for _ in range(5):
            state = h0.clone()
            y, same = ssm.selective_scan_fwd(**s, init_state=state, final_state=state, workspace=ws)
            assert same is state and torch.equal(y, want) and torch.equal(state, end)
