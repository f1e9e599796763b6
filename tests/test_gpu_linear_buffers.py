"""Buffers that a caller gives to the gradients of the matrix product."""

import pytest
import torch

from test_gpu_block import DT, block, linear_case  # noqa: F401

pytestmark = pytest.mark.gpu


@DT
def test_linear_returns_what_is_wanted(block, dtype):  # noqa: F811
    """A buffer of a gradient that is not wanted is neither written nor handed back as one."""
    c = linear_case(1, 40, 64, 72, dtype)
    full = block.linear_bwd(c["x"], c["w"], c["d_y"])
    for name in ("dx", "dweight", "dbias"):
        buffers = {k: torch.full_like(v, 7) for k, v in full.items()}
        got = block.linear_bwd(c["x"], c["w"], c["d_y"], grads=buffers, **{f"want_{name}": False})
        assert set(got) == set(full) - {name} and bool((buffers[name] == 7).all())
        assert all(got[k] is buffers[k] and torch.equal(got[k], full[k]) for k in got)
