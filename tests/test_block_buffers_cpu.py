"""One buffer for two in the forward calls around a mixer: outputs over the vectors that every row reads."""

from test_block_abi_cpu import FAR, linear, norm
from test_layers_abi_cpu import dr  # noqa: F401


def test_linear_outputs_over_the_bias(dr):  # noqa: F811
    names = ("x", "weight", "bias", "residual", "y", "slope")
    at = dict(zip(names, FAR))
    for out in ("y", "slope"):
        for M in (1, 5):
            p = {**at, out: at["bias"]}
            assert dr.dr_linear_fwd(linear(dr, M=M, N=64, act=2), *(p[n] for n in names), None, 0, stream=0) == dr.DR_ERR_ARG


def test_norm_outputs_over_the_weights(dr):  # noqa: F811
    names = ("h", "branch", "gate", "scale", "post_weight", "pre_weight", "h_out", "y")
    at = dict(zip(names, FAR))
    for out in ("h_out", "y"):
        for of in ("scale", "post_weight", "pre_weight"):
            p = {**at, out: at[of]}
            assert dr.dr_block_norm_fwd(norm(dr), *(p[n] for n in names), stream=0) == dr.DR_ERR_ARG, (out, of)
