"""Host-side checks of the layers' entry points (no GPU needed, no kernel launched):
struct layouts, refusals, workspace sizes.  Every call here is refused before any
pointer is used."""

import ctypes
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "recurrent_associative_memory_gb300", "libdr.so")
A = 1 << 20          # an aligned address that is never dereferenced
MIS = A + 4


@pytest.fixture(scope="module")
def dr():
    if not os.path.exists(LIB):
        from recurrent_associative_memory_gb300 import build
        build.build()
    from recurrent_associative_memory_gb300 import dr as mod
    return mod


@pytest.mark.parametrize("c_name,py_name", [("dr_attn", "DrAttn"), ("dr_conv", "DrConv"),
                                            ("dr_scan", "DrScan"), ("dr_scan_grads", "DrScanGrads")])
def test_struct_layout_matches_c(dr, c_name, py_name):
    cls = getattr(dr, py_name)
    names = [f[0] for f in cls._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"dr.h\"\nint main(void){\n"
    src += f'printf("%zu\\n", sizeof({c_name}));\n'
    src += "".join(f'printf("%zu\\n", offsetof({c_name}, {n}));\n' for n in names) + "return 0;}\n"
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "l.c"), os.path.join(td, "l")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe],
                       check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True,
                                              check=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, n).offset for n in names]


def attn(dr, **kw):
    a = dr.dr_attn_init()
    f = dict(dtype=dr.DR_BF16, B=2, T=65, S=65, H=4, Hkv=2, d=64, window=16, n_sink=4)
    for t in "qkv":
        f.update({f"{t}_sb": 65 * 256, f"{t}_st": 256, f"{t}_sh": 64})
    for k, v in {**f, **kw}.items():
        setattr(a, k, v)
    return a


BAD_HEADS = [(dict(dtype=7), "DR_ERR_DTYPE"), (dict(B=0), "DR_ERR_SHAPE"), (dict(H=5), "DR_ERR_SHAPE"),
             (dict(Hkv=0), "DR_ERR_SHAPE"), (dict(d=96), "DR_ERR_SHAPE"), (dict(window=0), "DR_ERR_ARG"),
             (dict(n_sink=-1), "DR_ERR_ARG"), (dict(n_sink=129), "DR_ERR_ARG"),
             (dict(scale=-1.0), "DR_ERR_ARG"), (dict(scale=float("nan")), "DR_ERR_ARG"),
             (dict(scale=float("inf")), "DR_ERR_ARG")]
BAD_ROWS = [(dict(T=0), "DR_ERR_SHAPE"), (dict(S=0), "DR_ERR_SHAPE"), (dict(q_start=-1), "DR_ERR_ARG"),
            (dict(q_start=2**31 - 10), "DR_ERR_ARG"),
            (dict(B=2**20, T=2**20), "DR_ERR_SHAPE"), (dict(q_st=260), "DR_ERR_ALIGN"),
            (dict(k_sh=4), "DR_ERR_ALIGN"), (dict(v_sb=3), "DR_ERR_ALIGN")]


@pytest.mark.parametrize("kw,want", BAD_HEADS + BAD_ROWS)
def test_attention_refuses(dr, kw, want):
    a = attn(dr, **kw)
    assert dr.dr_window_attn_fwd(a, A, A, A, A, None, stream=0) == getattr(dr, want)
    assert dr.dr_window_attn_bwd(a, A, A, A, A, A, A, A, A, A, A, 1 << 40, stream=0) == getattr(dr, want)


@pytest.mark.parametrize("kw,want", BAD_HEADS)
def test_attention_step_refuses(dr, kw, want):
    a = attn(dr, **kw)
    assert dr.dr_window_attn_step(a, A, A, A, A, A, A, A, stream=0) == getattr(dr, want)
    assert dr.dr_window_cache_fill(a, A, A, A, A, stream=0) == getattr(dr, want)


def test_attention_pointers(dr):
    a = attn(dr)
    for i in range(4):
        p = [A] * 4
        p[i] = None
        assert dr.dr_window_attn_fwd(a, *p, None, stream=0) == dr.DR_ERR_NULL
        p[i] = MIS
        assert dr.dr_window_attn_fwd(a, *p, None, stream=0) == dr.DR_ERR_ALIGN
    for i in range(9):
        p = [A] * 9
        p[i] = None
        assert dr.dr_window_attn_bwd(a, *p, A, 1 << 30, stream=0) == dr.DR_ERR_NULL
    need = dr.dr_window_attn_bwd_workspace_bytes(a)
    assert need >= 4 * 2 * 4 * 65 and need % 256 == 0
    assert dr.dr_window_attn_bwd(a, *[A] * 9, None, need, stream=0) == dr.DR_ERR_WORKSPACE
    assert dr.dr_window_attn_bwd(a, *[A] * 9, A, need - 1, stream=0) == dr.DR_ERR_WORKSPACE
    assert dr.dr_window_attn_bwd(a, *[A] * 9, A + 16, need, stream=0) == dr.DR_ERR_ALIGN
    for i in range(7):
        p = [A] * 7
        p[i] = None
        assert dr.dr_window_attn_step(a, *p, stream=0) == dr.DR_ERR_NULL
    for i in range(4):
        p = [A] * 4
        p[i] = None
        assert dr.dr_window_cache_fill(a, *p, stream=0) == dr.DR_ERR_NULL
        p[i] = MIS
        assert dr.dr_window_cache_fill(a, *p, stream=0) == dr.DR_ERR_ALIGN
    assert dr.dr_window_cache_fill(attn(dr, S=0), A, A, A, A, stream=0) == dr.DR_ERR_SHAPE
    assert dr.dr_window_attn_bwd_workspace_bytes(attn(dr, d=96)) == 0


def conv(dr, **kw):
    return dr.DrConv(**{**dict(dtype=dr.DR_BF16, B=2, T=33, D=40, K=4, silu=1, x_sb=33 * 40, x_st=40), **kw})


@pytest.mark.parametrize("kw,want", [(dict(dtype=-1), "DR_ERR_DTYPE"), (dict(B=0), "DR_ERR_SHAPE"),
                                     (dict(D=0), "DR_ERR_SHAPE"), (dict(K=1), "DR_ERR_SHAPE"),
                                     (dict(K=5), "DR_ERR_SHAPE")])
def test_conv_refuses(dr, kw, want):
    a = conv(dr, **kw)
    assert dr.dr_short_conv_fwd(a, A, A, A, None, A, None, stream=0) == getattr(dr, want)
    assert dr.dr_short_conv_bwd(a, A, A, A, None, A, None, A, A, A, None, A, 1 << 40,
                                stream=0) == getattr(dr, want)
    assert dr.dr_short_conv_step(a, A, A, A, A, A, A, stream=0) == getattr(dr, want)


def test_conv_pointers(dr):
    a = conv(dr)
    assert dr.dr_short_conv_fwd(conv(dr, T=0), A, A, A, None, A, None, stream=0) == dr.DR_ERR_SHAPE
    assert dr.dr_short_conv_fwd(a, None, A, A, None, A, None, stream=0) == dr.DR_ERR_NULL
    assert dr.dr_short_conv_fwd(a, A, None, A, None, A, None, stream=0) == dr.DR_ERR_NULL
    assert dr.dr_short_conv_fwd(a, A, A, A, None, None, None, stream=0) == dr.DR_ERR_NULL
    need = dr.dr_short_conv_bwd_workspace_bytes(a)
    assert need >= 4 * 5 * 40
    assert dr.dr_short_conv_bwd(a, A, A, A, None, A, None, A, A, A, None, A, need - 4,
                                stream=0) == dr.DR_ERR_WORKSPACE
    assert dr.dr_short_conv_bwd(a, A, A, A, None, A, None, A, A, A, None, A + 4, need,
                                stream=0) == dr.DR_ERR_ALIGN
    assert dr.dr_short_conv_bwd(a, A, A, A, None, A, None, A, None, A, None, A, need,
                                stream=0) == dr.DR_ERR_NULL
    assert dr.dr_short_conv_step(a, A, A, A, A, None, A, stream=0) == dr.DR_ERR_NULL


def scan(dr, **kw):
    return dr.DrScan(**{**dict(dtype=dr.DR_BF16, B=2, T=33, D=40, N=16, G=2, softplus=1, A=A), **kw})


@pytest.mark.parametrize("kw,want", [(dict(dtype=3), "DR_ERR_DTYPE"), (dict(B=0), "DR_ERR_SHAPE"),
                                     (dict(G=3), "DR_ERR_SHAPE"), (dict(G=0), "DR_ERR_SHAPE"),
                                     (dict(N=12), "DR_ERR_SHAPE"), (dict(A=None), "DR_ERR_NULL"),
                                     (dict(A=MIS), "DR_ERR_ALIGN")])
def test_scan_refuses(dr, kw, want):
    a = scan(dr, **kw)
    g = dr.DrScanGrads(*[A] * 9)
    assert dr.dr_selective_scan_fwd(a, A, A, A, A, None, None, A, None, stream=0) == getattr(dr, want)
    assert dr.dr_selective_scan_bwd(a, A, A, A, A, None, None, A, None, g, A, 1 << 40,
                                    stream=0) == getattr(dr, want)
    assert dr.dr_selective_scan_step(a, A, A, A, A, None, A, A, A, stream=0) == getattr(dr, want)


def test_scan_pointers(dr):
    a = scan(dr)
    g = dr.DrScanGrads(*[A] * 9)
    assert dr.dr_selective_scan_fwd(scan(dr, T=0), A, A, A, A, None, None, A, None, stream=0) == dr.DR_ERR_SHAPE
    for i in range(4):
        p = [A] * 4
        p[i] = None
        assert dr.dr_selective_scan_fwd(a, *p, None, None, A, None, stream=0) == dr.DR_ERR_NULL
        assert dr.dr_selective_scan_step(a, *p, None, A, A, A, stream=0) == dr.DR_ERR_NULL
    assert dr.dr_selective_scan_fwd(a, A, A, A, A, None, MIS, A, None, stream=0) == dr.DR_ERR_ALIGN
    assert dr.dr_selective_scan_step(a, A, A, A, A, None, A, MIS, A, stream=0) == dr.DR_ERR_ALIGN
    need = dr.dr_selective_scan_bwd_workspace_bytes(a)
    assert need > 0 and need % 256 == 0
    assert dr.dr_selective_scan_bwd(a, A, A, A, A, None, None, A, None, g, A, need - 1,
                                    stream=0) == dr.DR_ERR_WORKSPACE
    no_dz = dr.DrScanGrads(A, A, None, *[A] * 6)
    assert dr.dr_selective_scan_bwd(a, A, A, A, A, A, None, A, None, no_dz, A, need,
                                    stream=0) == dr.DR_ERR_NULL
