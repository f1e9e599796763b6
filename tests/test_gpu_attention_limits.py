"""Window attention with numbers beyond 32 bits."""

import pytest
import torch

from test_gpu_layers import mods, qkv  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_window_beyond_32_bits_sees_everything(mods):  # noqa: F811
    q, k, v, _ = qkv(1, 1, 200, 200, 2, 1, 64, torch.bfloat16)
    want, _ = mods[0].window_attn_fwd(q, k, v, 200)
    for window in (2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1):
        assert torch.equal(mods[0].window_attn_fwd(q, k, v, window)[0], want)
    with pytest.raises(ValueError):
        mods[0].window_attn_fwd(q, k, v, 5, q_start=2 ** 32)
    with pytest.raises(ValueError):
        mods[0].window_attn_fwd(q, k, v, 5, 2 ** 32)
