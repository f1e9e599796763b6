"""Host-side checks of the entry points around a mixer (no GPU needed, no kernel launched):
struct layouts, refusals, workspace sizes, calls where there is no device."""

import os
import subprocess
import sys

import pytest
import torch

from test_layers_abi_cpu import A, MIS, dr, test_struct_layout_matches_c as layout  # noqa: F401

BIG = 1 << 45
OTHER = A + (1 << 16)
FAR = [A + (i << 16) for i in range(12)]   # aligned addresses of which no two are one


@pytest.mark.parametrize("c_name,py_name", [("dr_linear", "DrLinear"), ("dr_block_norm", "DrBlockNorm"),
                                            ("dr_block_norm_grads", "DrBlockNormGrads")])
def test_struct_layouts(dr, c_name, py_name):  # noqa: F811
    layout(dr, c_name, py_name)


def linear(dr, **kw):  # noqa: F811
    f = dict(dtype=dr.DR_BF16, act=0, M=5, K=64, N=48, w_transposed=0, x_s=64, w_s=48, r_s=48)
    return dr.DrLinear(*({**f, **kw}[n] for n, _ in dr.DrLinear._fields_))


BAD_LINEAR = [(dict(dtype=2), "DR_ERR_DTYPE"), (dict(dtype=-1), "DR_ERR_DTYPE"), (dict(act=-1), "DR_ERR_ARG"),
              (dict(act=5), "DR_ERR_ARG"), (dict(M=0), "DR_ERR_SHAPE"), (dict(M=-3), "DR_ERR_SHAPE"),
              (dict(K=0), "DR_ERR_SHAPE"), (dict(N=0), "DR_ERR_SHAPE"), (dict(K=(1 << 24) + 1), "DR_ERR_SHAPE"),
              (dict(N=(1 << 24) + 1), "DR_ERR_SHAPE"), (dict(M=(1 << 31) - 1, K=1024), "DR_ERR_SHAPE"),
              (dict(M=(1 << 31) - 1, N=1024), "DR_ERR_SHAPE"), (dict(K=1 << 24, N=1 << 20), "DR_ERR_SHAPE")]


@pytest.mark.parametrize("kw,want", BAD_LINEAR)
def test_linear_refuses(dr, kw, want):  # noqa: F811
    a = linear(dr, **kw)
    assert dr.dr_linear_fwd(a, A, A, None, None, A, None, A, BIG, stream=0) == getattr(dr, want)
    assert dr.dr_linear_bwd(a, A, A, A, A, A, A, A, A, BIG, stream=0) == getattr(dr, want)
    assert dr.dr_linear_fwd_workspace_bytes(a) == 0 and dr.dr_linear_bwd_workspace_bytes(a) == 0


def test_linear_pointers(dr):  # noqa: F811
    a, fp = linear(dr), linear(dr, dtype=dr.DR_FP32, M=20)
    for i in (0, 1, 4):
        p = [A, A, None, None, A, None]
        p[i] = None
        assert dr.dr_linear_fwd(a, *p, stream=0) == dr.DR_ERR_NULL
    for i in (0, 1, 3, 4, 5):
        p = [A, A, A, A, A, A]
        p[i] = MIS
        assert dr.dr_linear_fwd(a, *p, stream=0) == dr.DR_ERR_ALIGN
    need = dr.dr_linear_fwd_workspace_bytes(fp)
    assert need >= 6 * (20 * 64 + 64 * 48)
    assert dr.dr_linear_fwd(fp, A, A, None, None, OTHER, None, None, 0, stream=0) == dr.DR_ERR_WORKSPACE
    assert dr.dr_linear_fwd(fp, A, A, None, None, A, None, A, need - 1, stream=0) == dr.DR_ERR_WORKSPACE
    assert dr.dr_linear_fwd(fp, A, A, None, None, A, None, A + 16, need, stream=0) == dr.DR_ERR_ALIGN
    s = linear(dr, act=2)
    assert dr.dr_linear_bwd(a, A, A, None, None, A, A, A, A, BIG, stream=0) == dr.DR_ERR_NULL
    assert dr.dr_linear_bwd(a, A, A, A, None, None, None, None, A, BIG, stream=0) == dr.DR_ERR_NULL
    assert dr.dr_linear_bwd(a, A, None, A, None, A, A, A, A, BIG, stream=0) == dr.DR_ERR_NULL
    assert dr.dr_linear_bwd(a, None, A, A, None, A, A, A, A, BIG, stream=0) == dr.DR_ERR_NULL
    assert dr.dr_linear_bwd(s, A, A, A, None, A, A, A, A, BIG, stream=0) == dr.DR_ERR_NULL
    need = dr.dr_linear_bwd_workspace_bytes(s)
    assert dr.dr_linear_bwd(s, A, A, A, A, A, A, A, A, need - 1, stream=0) == dr.DR_ERR_WORKSPACE
    assert dr.dr_linear_bwd(s, A, A, A, A, A, A, A, None, need, stream=0) == dr.DR_ERR_WORKSPACE
    assert dr.dr_linear_bwd(s, A, A, A, A, A, A, A, MIS, need, stream=0) == dr.DR_ERR_ALIGN
    for i in (0, 1, 2, 3, 4, 5):
        p = [A] * 7
        p[i] = MIS
        assert dr.dr_linear_bwd(s, *p, A, BIG, stream=0) == dr.DR_ERR_ALIGN


def test_one_buffer_for_two(dr):  # noqa: F811
    """Outputs over inputs that other blocks still read, or over each other."""
    a = linear(dr, N=64, act=2)
    names = ("x", "weight", "bias", "residual", "y", "slope")
    at = dict(zip(names, FAR))
    fwd = lambda a, **kw: dr.dr_linear_fwd(a, *({**at, **kw}[n] for n in names), None, 0, stream=0)  # noqa: E731
    for out, of in (("y", "x"), ("y", "weight"), ("slope", "x"), ("slope", "weight"), ("slope", "residual"), ("slope", "y")):
        assert fwd(a, **{out: at[of]}) == dr.DR_ERR_ARG, (out, of)
    wide = linear(dr, N=64, r_s=72)
    assert fwd(wide, y=at["residual"]) == dr.DR_ERR_ARG
    back = ("x", "weight", "d_y", "slope", "dx", "d_weight", "d_bias")
    there = dict(zip(back, FAR))
    for out in back[4:]:
        for of in back:
            if of != out:
                p = {**there, out: there[of]}
                assert dr.dr_linear_bwd(a, *(p[n] for n in back), FAR[10], BIG, stream=0) == dr.DR_ERR_ARG, (out, of)
    n = norm(dr, h_s=72)
    parts = ("h", "branch", "gate", "scale", "post_weight", "pre_weight", "h_out", "y")
    place = dict(zip(parts, FAR))
    for out, of in (("y", "h"), ("y", "branch"), ("y", "gate"), ("y", "h_out"), ("h_out", "branch"), ("h_out", "gate"),
                    ("h_out", "h")):   # the last: rows further apart than what is written
        p = {**place, out: place[of]}
        assert dr.dr_block_norm_fwd(n, *(p[k] for k in parts), stream=0) == dr.DR_ERR_ARG, (out, of)


def test_linear_workspace(dr):  # noqa: F811
    """bf16 in place where a tensor map holds it; copies otherwise."""
    size = dr.dr_linear_fwd_workspace_bytes
    assert size(linear(dr)) == 0
    assert size(linear(dr, w_transposed=1, w_s=64)) == 0
    assert size(linear(dr, x_s=68)) >= 2 * 5 * 64 and size(linear(dr, x_s=0)) > 0
    assert size(linear(dr, M=1, x_s=3)) == 0
    assert size(linear(dr, w_s=50)) >= 2 * 64 * 48
    assert size(linear(dr, N=47, w_s=47)) >= 2 * 64 * 48
    assert size(linear(dr, dtype=dr.DR_FP32, M=9)) >= 6 * (9 * 64 + 64 * 48) and size(linear(dr, dtype=dr.DR_FP32, M=8)) == 0
    assert size(linear(dr, dtype=dr.DR_FP32, M=8, w_s=50)) > 0   # rows that no 16 bytes start
    assert size(linear(dr, dtype=dr.DR_FP32, M=40, K=63)) % 256 == 0


def norm(dr, **kw):  # noqa: F811
    f = dict(dtype=dr.DR_BF16, h_dtype=dr.DR_BF16, M=5, D=64, post_norm=1, gate_act=2, eps=1e-6, h_s=64, b_s=64, g_s=64)
    return dr.DrBlockNorm(*({**f, **kw}[n] for n, _ in dr.DrBlockNorm._fields_))


BAD_NORM = [(dict(dtype=2), "DR_ERR_DTYPE"), (dict(h_dtype=3), "DR_ERR_DTYPE"), (dict(dtype=0), "DR_ERR_DTYPE"),
            (dict(gate_act=5), "DR_ERR_ARG"), (dict(gate_act=-1), "DR_ERR_ARG"), (dict(eps=-1.0), "DR_ERR_ARG"),
            (dict(eps=float("nan")), "DR_ERR_ARG"), (dict(eps=float("inf")), "DR_ERR_ARG"), (dict(M=0), "DR_ERR_SHAPE"),
            (dict(D=0), "DR_ERR_SHAPE"), (dict(D=8193), "DR_ERR_SHAPE"), (dict(M=(1 << 31) - 1, D=1024), "DR_ERR_SHAPE")]


@pytest.mark.parametrize("kw,want", BAD_NORM)
def test_block_norm_refuses(dr, kw, want):  # noqa: F811
    a = norm(dr, **kw)
    g = dr.DrBlockNormGrads(*[A] * 6)
    assert dr.dr_block_norm_fwd(a, A, A, A, A, A, A, A, OTHER, stream=0) == getattr(dr, want)
    assert dr.dr_block_norm_bwd(a, A, A, A, A, A, A, A, A, g, A, BIG, stream=0) == getattr(dr, want)
    assert dr.dr_block_norm_bwd_workspace_bytes(a) == 0


def test_block_norm_combinations(dr):  # noqa: F811
    a, plain = norm(dr), norm(dr, post_norm=0)
    fwd = lambda a, *p: dr.dr_block_norm_fwd(a, *p, stream=0)  # noqa: E731
    assert fwd(a, None, A, A, A, A, A, A, OTHER) == dr.DR_ERR_NULL
    assert fwd(a, A, A, A, A, A, A, None, OTHER) == dr.DR_ERR_NULL       # branch without h_out
    assert fwd(plain, A, None, None, None, None, None, None, None) == dr.DR_ERR_NULL
    assert fwd(plain, A, None, A, None, None, None, None, OTHER) == dr.DR_ERR_ARG     # a gate of nothing
    assert fwd(plain, A, None, None, A, None, None, None, OTHER) == dr.DR_ERR_ARG
    assert fwd(plain, A, None, None, None, None, None, A, OTHER) == dr.DR_ERR_ARG
    assert fwd(a, A, None, None, None, None, None, None, OTHER) == dr.DR_ERR_ARG
    assert fwd(plain, A, A, None, None, A, None, A, OTHER) == dr.DR_ERR_ARG           # post_weight, no norm
    assert fwd(plain, A, A, None, None, None, A, A, None) == dr.DR_ERR_ARG            # pre_weight, no y
    assert fwd(plain, A, A, None, None, None, None, OTHER, A) == dr.DR_ERR_ARG        # y over h
    assert fwd(plain, A, A, None, None, None, None, OTHER, OTHER) == dr.DR_ERR_ARG
    bwd = lambda a, p, g, ws=A, n=BIG: dr.dr_block_norm_bwd(a, *p, dr.DrBlockNormGrads(*g), ws, n, stream=0)  # noqa: E731
    full = [A] * 8
    assert bwd(a, [None] + full[1:], [A] * 6) == dr.DR_ERR_NULL
    assert bwd(a, full[:6] + [None, None], [A] * 6) == dr.DR_ERR_NULL
    assert bwd(plain, [A, A, None, None, None, None, A, A], [A, A, A, None, None, None]) == dr.DR_ERR_ARG   # dgate
    assert bwd(plain, [A, A, None, None, None, None, A, A], [A, A, None, A, None, None]) == dr.DR_ERR_ARG   # dscale
    assert bwd(a, [A, A, None, None, None, None, A, A], [A, A, None, None, A, None]) == dr.DR_ERR_ARG
    assert bwd(a, [A, A, None, None, None, None, A, A], [A, A, None, None, None, A]) == dr.DR_ERR_ARG
    assert bwd(a, full[:7] + [None], [A] * 6) == dr.DR_ERR_ARG                        # dpre_weight without d_y
    assert bwd(plain, [A, None, None, None, None, None, A, A], [A, A, None, None, None, None]) == dr.DR_ERR_ARG


def test_alignment_of_single_values(dr):  # noqa: F811
    """What needs no 16 bytes still stands on its own type's."""
    a = linear(dr)
    assert dr.dr_linear_fwd(a, A, A, A + 1, None, A, None, stream=0) == dr.DR_ERR_ALIGN
    assert dr.dr_linear_bwd(a, A, A, A, None, A, A, A + 1, A, BIG, stream=0) == dr.DR_ERR_ALIGN
    n = norm(dr, h_dtype=dr.DR_FP32)
    for i in range(8):
        p = FAR[:8]
        p[i] += 2 if i in (0, 3, 4, 5, 6) else 1
        assert dr.dr_block_norm_fwd(n, *p, stream=0) == dr.DR_ERR_ALIGN
        for j in range(6):
            g = [A] * 6
            g[j] += 1
            q = [A] * 8
            assert dr.dr_block_norm_bwd(n, *q, dr.DrBlockNormGrads(*g), A, BIG, stream=0) == dr.DR_ERR_ALIGN
        q = [A] * 8
        q[i] += 2 if i in (0, 3, 4, 5, 6) else 1
        assert dr.dr_block_norm_bwd(n, *q, dr.DrBlockNormGrads(*[A] * 6), A, BIG, stream=0) == dr.DR_ERR_ALIGN


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no tensors")
def test_block_norm_workspace_where_there_is_no_device(dr):  # noqa: F811
    """Sums over the rows need one; its size is the device's, so without a device it is 0."""
    assert dr.dr_block_norm_bwd_workspace_bytes(norm(dr)) == 0


CALLS = """
import sys
sys.path[:0] = [{tests!r}, {root!r}]
from test_block_abi_cpu import A, BIG, FAR, linear, norm
from recurrent_associative_memory_gb300 import dr
for dtype in (dr.DR_BF16, dr.DR_FP32):
    a, s = linear(dr, dtype=dtype), linear(dr, dtype=dtype, act=3)
    print(dr.dr_linear_fwd(a, *FAR[:6], A, BIG, stream=0))
    print(dr.dr_linear_bwd(s, *FAR[:7], FAR[8], BIG, stream=0))
    n, g = norm(dr, dtype=dtype, h_dtype=dr.DR_FP32), dr.DrBlockNormGrads(*[A] * 6)
    print(dr.dr_block_norm_fwd(n, *FAR[:8], stream=0))
    print(dr.dr_block_norm_bwd(n, A, A, A, A, A, A, A, A, g, A, BIG, stream=0))
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no tensors")
def test_without_a_device_a_valid_call_returns_an_error(dr):  # noqa: F811
    """In a process of its own: nothing may end it."""
    code = CALLS.format(tests=os.path.dirname(__file__), root=os.path.dirname(os.path.dirname(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert r.stdout.split() == [str(dr.DR_ERR_CUDA)] * 8


# ------------------------------------------------------------------ Python's checks

def test_python_refuses_what_is_no_cuda_tensor(dr):  # noqa: F811
    from recurrent_associative_memory_gb300 import block
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.bfloat16)
    for call in (lambda: block.linear_fwd(x, w), lambda: block.linear_bwd(x, w, x), lambda: block.block_norm_fwd(x),
                 lambda: block.block_norm_bwd(x, d_y=x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: block.linear_fwd(3, w), lambda: block.block_norm_fwd([1.0]),
                 lambda: block.linear_fwd(x.long(), w), lambda: block.block_norm_fwd(x.double())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: block.linear_fwd(x[0], w), lambda: block.block_norm_fwd(x[None, None])):
        with pytest.raises(ValueError):
            call()
