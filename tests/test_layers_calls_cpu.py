"""Host side of the layers' entry points (no kernel runs): buffers that may not be one, and
calls where there is no device."""

import os
import subprocess
import sys

import pytest
import torch

from test_layers_abi_cpu import A, conv, dr  # noqa: F401


def test_conv_backward_refuses_one_buffer_for_both_state_gradients(dr):  # noqa: F811
    a = conv(dr)
    need = dr.dr_short_conv_bwd_workspace_bytes(a)
    other = A + (1 << 18)
    assert dr.dr_short_conv_bwd(a, A, A, A, A, A, other, A, A, A, other, A, need, stream=0) == dr.DR_ERR_ARG


CALLS = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
from test_layers_abi_cpu import A, attn, conv, scan
from recurrent_associative_memory_gb300 import dr
n, size = 1 << 40, dict(T=8192, D=2048)
g = dr.DrScanGrads(*[A] * 9)
for dtype in (dr.DR_BF16, dr.DR_FP32):
    a, c, s = attn(dr, dtype=dtype), conv(dr, dtype=dtype), scan(dr, dtype=dtype, **size)
    print(dr.dr_window_attn_fwd(a, A, A, A, A, A, stream=0))
    print(dr.dr_window_attn_bwd(a, *[A] * 9, A, n, stream=0))
    print(dr.dr_window_attn_step(a, *[A] * 7, A, n, stream=0))
    print(dr.dr_window_attn_step(a, *[A] * 7, stream=0))
    print(dr.dr_window_cache_fill(a, A, A, A, A, stream=0))
    print(dr.dr_short_conv_fwd(c, A, A, A, A, A, A, stream=0))
    print(dr.dr_short_conv_bwd(c, A, A, A, None, A, None, A, A, A, None, A, n, stream=0))
    print(dr.dr_short_conv_step(c, A, A, A, A, A, A, stream=0))
    print(dr.dr_selective_scan_fwd(s, A, A, A, A, A, A, A, A, A, n, stream=0))
    print(dr.dr_selective_scan_fwd(s, A, A, A, A, A, A, A, A, stream=0))
    print(dr.dr_selective_scan_bwd(s, A, A, A, A, A, A, A, A, g, A, n, stream=0))
    print(dr.dr_selective_scan_step(s, A, A, A, A, A, A, A, A, stream=0))
    for size_of, d in ((dr.dr_window_attn_step_workspace_bytes, a), (dr.dr_selective_scan_fwd_workspace_bytes, s)):
        size_of(d)
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no tensors")
def test_without_a_device_a_valid_call_returns_an_error(dr):  # noqa: F811
    """In a process of its own: nothing may end it."""
    code = CALLS.format(tests=os.path.dirname(__file__), root=os.path.dirname(os.path.dirname(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert set(r.stdout.split()) == {str(dr.DR_ERR_CUDA)} and len(r.stdout.split()) == 24
