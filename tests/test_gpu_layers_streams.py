"""Layers on a stream that is not the current one: inputs may be let go as soon as the call
is back."""

import math

import pytest
import torch

from test_gpu_layers import mods, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_inputs_of_a_call_on_another_stream_may_be_let_go(mods, raw):  # noqa: F811
    """While the stream is busy the inputs lose their last reference, and the current stream
    allocates and overwrites blocks of their sizes."""
    _, ssm = mods
    g = torch.Generator().manual_seed(1)
    x, w = randn(g, 2, 300, 64), randn(g, 64, 4)
    want, end = ssm.short_conv_fwd(x, w)
    dx = ssm.short_conv_bwd(x, w, None, x)["dx"]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    busy = torch.randn(4096, 4096, device="cuda")
    for call, expected in ((lambda a, b: ssm.short_conv_fwd(a, b, stream=stream), (want, end)),
                           (lambda a, b: (ssm.short_conv_bwd(a, b, None, a, stream=stream)["dx"],), (dx,))):
        mine, filt = x.clone(), w.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(60):
                busy = busy @ busy * 1e-4
        got = call(mine, filt)
        del mine, filt
        taken = [torch.full((n,), math.nan, device="cuda") for n in [x.numel(), w.numel()] * 4]
        torch.cuda.synchronize()
        assert taken and all(torch.equal(a, b) for a, b in zip(got, expected))
