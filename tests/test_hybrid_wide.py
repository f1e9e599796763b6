"""The hybrid stack at widths that the norms' kernels do not take."""

import numpy as np
import pytest
import torch

from oracle import block as O

D = 8448


def test_wide_rows_between_blocks():
    """Against the formulas: h' and y are rounded once each (half a step of bf16, 2^-8), y is the
    norm of the rounded h' (2^-8 again), and fp32 sums of 8448 terms add less than 2^-10."""
    from recurrent_associative_memory_gb300 import block, hybrid
    assert D > block.MAX_CHANNELS
    g = torch.Generator().manual_seed(1)
    h, o, gate = (torch.randn(2, 3, D, generator=g).bfloat16() for _ in range(3))
    weight, scale = torch.randn(D, generator=g) * 0.1 + 1, torch.randn(D, generator=g) * 0.1 + 0.5
    np64 = lambda t: t.double().numpy()  # noqa: E731
    for kw in ({}, dict(gate=gate, gate_act="sigmoid", scale=scale, post_norm=True, post_weight=weight)):
        y, h2 = hybrid._join(h, o, **kw)
        want_y, want_h = O.block_norm(np64(h), np64(o), eps=hybrid.EPS,
                                      **{k: np64(v) if torch.is_tensor(v) else v for k, v in kw.items()})
        assert y.dtype is h2.dtype is torch.bfloat16
        assert (np.abs(np64(h2) - want_h) <= 2.0 ** -8 * np.abs(want_h) + 2.0 ** -10).all()
        assert (np.abs(np64(y) - want_y) <= 2 * 2.0 ** -8 * np.abs(want_y) + 2.0 ** -10).all()
    y, same = hybrid._join(h)
    assert same is h and torch.equal(y, torch.nn.functional.rms_norm(h.float(), (D,)).bfloat16())


@pytest.mark.gpu
def test_a_wide_stack_decodes_what_its_prompt_form_gives():
    from recurrent_associative_memory_gb300 import hybrid
    assert hybrid.main(B=2, T=40, more=3, dim=D) < 4.7e-2   # three layers and the unembedding: 3 (3 + 1) 2^-8
