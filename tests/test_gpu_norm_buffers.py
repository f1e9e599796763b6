"""The buffers of the gradients of the norms around a block: which of them may be one."""

import pytest
import torch

from test_gpu_block import TYPES, block, norm_case  # noqa: F401

pytestmark = pytest.mark.gpu
GRADS = ("dh", "dbranch", "dgate", "dscale", "dpost_weight", "dpre_weight")
INPUTS = ("h", "branch", "gate", "scale", "post_weight", "pre_weight", "d_h", "d_y")
OVER = (("dh", "h"), ("dh", "d_h"), ("dbranch", "branch"), ("dgate", "gate"))
KW = dict(gate_act="silu", post_norm=True)


def test_one_buffer_for_two_gradients(block):  # noqa: F811
    """Refused before anything is launched; every tensor holds what the largest needs."""
    from recurrent_associative_memory_gb300 import dr
    M, D = 6, 64
    buffer = {n: torch.full((M * D,), 7.0, device="cuda") for n in GRADS + INPUTS}
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def call(M=M, h_s=D, b_s=D, g_s=D, **one):
        at = {n: one.get(n, b.data_ptr()) for n, b in buffer.items()}
        a = dr.DrBlockNorm(dr.DR_FP32, dr.DR_FP32, M, D, 1, 2, 1e-6, h_s, b_s, g_s)
        g = dr.DrBlockNormGrads(*(at[n] for n in GRADS))
        return dr.dr_block_norm_bwd(a, *(at[n] for n in INPUTS), g, ws, ws.numel())

    for out in GRADS:
        for of in GRADS + INPUTS:
            if of != out and (out, of) not in OVER:
                assert call(**{out: buffer[of].data_ptr()}) == dr.DR_ERR_ARG, (out, of)
    # rows of another stride are not the gradient's
    for out, of, stride in (("dh", "h", "h_s"), ("dbranch", "branch", "b_s"), ("dgate", "gate", "g_s")):
        assert call(**{out: buffer[of].data_ptr(), stride: 8}) == dr.DR_ERR_ARG, (out, of)
    torch.cuda.synchronize()
    assert all(bool((b == 7).all()) for b in buffer.values())
    for out, of in OVER:
        assert call(**{out: buffer[of].data_ptr()}) == dr.DR_OK, (out, of)
    assert call(M=1, h_s=8, dh=buffer["h"].data_ptr()) == dr.DR_OK   # one row has no stride
    torch.cuda.synchronize()


@TYPES
@pytest.mark.parametrize("M,D", [(5, 24), (333, 77), (700, 264), (400, 333), (310, 2047), (300, 4096), (200, 4099), (170, 8185),
                                 (160, 8192)])
def test_gradients_in_place(block, M, D, dtype, h_dtype):  # noqa: F811
    """A row's gradient over what it is the gradient of: the same bits as in a buffer of its own."""
    c, d = norm_case(M + D, M, D, dtype, h_dtype)
    want = block.block_norm_bwd(**c, **d, **KW)
    for which in (("h", "branch", "gate"), ("d_h", "gate"), ("branch",)):
        copy = {k: v.clone() if k in which else v for k, v in {**c, **d}.items()}
        over = {("dh" if n == "d_h" else "d" + n): copy[n] for n in which}
        got = block.block_norm_bwd(**copy, **KW, grads=over)
        assert all(got[n] is t for n, t in over.items())
        assert all(torch.equal(got[k], want[k]) for k in want), which
