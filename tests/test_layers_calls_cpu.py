"""Host side of the layers' entry points (no kernel runs): buffers that may not be one."""

from test_layers_abi_cpu import A, conv, dr  # noqa: F401


def test_conv_backward_refuses_one_buffer_for_both_state_gradients(dr):  # noqa: F811
    a = conv(dr)
    need = dr.dr_short_conv_bwd_workspace_bytes(a)
    other = A + (1 << 18)
    assert dr.dr_short_conv_bwd(a, A, A, A, A, A, other, A, A, A, other, A, need, stream=0) == dr.DR_ERR_ARG
