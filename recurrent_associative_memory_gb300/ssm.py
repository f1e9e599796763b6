"""The short causal convolution and the selective state space scan.

Short convolution, one filter of K = 2 .. 4 taps per channel:
``u_t = bias + sum_j weight[:, j] x_{t-K+1+j}``, ``y = silu(u)``.

Selective scan, N = 8, 16, 32 or 64 states per channel:
``dt = softplus(dt + dt_bias)``, ``h_t = exp(dt A) h_{t-1} + dt B_t x_t``,
``y_t = (C_t . h_t + D x_t) silu(z_t)``.

Each has a prompt form that returns the state after the last token, a backward pass,
and a form for single tokens that takes the state one token further.  ``lens`` int32
[B] (on the device) gives the sequences' real lengths: rows from there on give y = 0
and leave the state alone.

The functions allocate outputs and call ``dr``; they compute nothing themselves.
Work runs on ``stream`` (default: the current one) of x's device.
"""

from __future__ import annotations

import torch

from . import dr
from .tensors import activations, check, launch, like_x, scratch, size_of

__all__ = ["short_conv_fwd", "short_conv_bwd", "short_conv_step", "selective_scan_fwd",
           "selective_scan_bwd", "selective_scan_step"]


def _new(t, shape, dtype, x):
    return torch.empty(shape, dtype=dtype, device=x.device) if t is None else t


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ short convolution

def _conv(x, weight, bias, silu, lens, dims):
    a = dr.DrConv()
    a.dtype = activations(x, "x", dims)
    D = x.shape[-1]
    if not torch.is_tensor(weight) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [D, K]")
    check(weight, "weight", (D, weight.shape[1]), torch.float32, x)
    check(bias, "bias", (D,), torch.float32, x)
    check(lens, "lens", (x.shape[0],), torch.int32, x)
    a.B, a.T, a.D, a.K, a.silu = x.shape[0], x.shape[1] if dims == 3 else 1, D, weight.shape[1], int(silu)
    a.lens = _ptr(lens)
    a.x_sb, a.x_st = x.stride(0), x.stride(1) if dims == 3 else 0
    return a


def short_conv_fwd(x, weight, bias=None, *, silu=True, init_state=None, lens=None, want_final=True,
                   y=None, final_state=None, stream=None):
    """x [B,T,D] (any batch and token strides), weight fp32 [D,K], bias fp32 [D], init_state
    [B,K-1,D] in x's type (the inputs before the first token, oldest first; None: zeros).
    Returns (y [B,T,D], final_state [B,K-1,D] or None)."""
    a = _conv(x, weight, bias, silu, lens, 3)
    state = (a.B, a.K - 1, a.D)
    check(init_state, "init_state", state, x.dtype, x)
    y = _new(y, x.shape, x.dtype, x)
    check(y, "y", x.shape, x.dtype, x)
    if want_final or final_state is not None:
        final_state = _new(final_state, state, x.dtype, x)
        check(final_state, "final_state", state, x.dtype, x)
    with launch(x, stream) as s:
        dr.check(dr.dr_short_conv_fwd(a, x, weight, bias, init_state, y, final_state, s),
                 "dr_short_conv_fwd")
    return y, final_state


def short_conv_bwd(x, weight, bias, d_y, *, silu=True, init_state=None, d_final_state=None,
                   lens=None, workspace="auto", grads=None, stream=None):
    """Returns dict(dx [B,T,D] in x's type, dweight fp32 [D,K], dbias fp32 [D]) and with
    init_state dinit_state [B,K-1,D].  ``grads`` may hold output tensors under these names."""
    a = _conv(x, weight, bias, silu, lens, 3)
    state = (a.B, a.K - 1, a.D)
    check(init_state, "init_state", state, x.dtype, x)
    check(d_y, "d_y", x.shape, x.dtype, x)
    check(d_final_state, "d_final_state", state, x.dtype, x)
    g = dict(grads or {})
    shapes = {"dx": (x.shape, x.dtype), "dweight": (weight.shape, torch.float32),
              "dbias": ((a.D,), torch.float32)}
    if init_state is not None:
        shapes["dinit_state"] = (state, x.dtype)
    for name, (shape, dtype) in shapes.items():
        g[name] = _new(g.get(name), shape, dtype, x)
        check(g[name], name, shape, dtype, x)
    with launch(x, stream) as s:
        ws = scratch(dr.dr_short_conv_bwd_workspace_bytes(a), x, workspace)
        dr.check(dr.dr_short_conv_bwd(a, x, weight, bias, init_state, d_y, d_final_state, g["dx"],
                                      g["dweight"], g["dbias"], g.get("dinit_state"), ws,
                                      size_of(ws), s), "dr_short_conv_bwd")
    return g


def short_conv_step(x, weight, bias, state, *, silu=True, state_out=None, y=None, stream=None):
    """One token: x [B,D], state [B,K-1,D].  The new state goes to ``state_out`` (default: in
    place).  Returns (y [B,D], the new state)."""
    a = _conv(x, weight, bias, silu, None, 2)
    shape = (a.B, a.K - 1, a.D)
    check(state, "state", shape, x.dtype, x)
    state_out = state if state_out is None else state_out
    check(state_out, "state_out", shape, x.dtype, x)
    y = _new(y, x.shape, x.dtype, x)
    check(y, "y", x.shape, x.dtype, x)
    with launch(x, stream) as s:
        dr.check(dr.dr_short_conv_step(a, x, weight, bias, state, state_out, y, s),
                 "dr_short_conv_step")
    return y, state_out


# ------------------------------------------------------------------ selective scan

def _scan(x, dt, A, B, C, D, z, dt_bias, softplus, lens, dims):
    a = dr.DrScan()
    a.dtype = activations(x, "x", dims)
    Dm = x.shape[-1]
    like_x(dt, "dt", x.shape, x)
    like_x(z, "z", x.shape, x)
    if not torch.is_tensor(A) or A.dim() != 2:
        raise ValueError("A must be a tensor [D, N]")
    N = A.shape[1]
    check(A, "A", (Dm, N), torch.float32, x)
    check(D, "D", (Dm,), torch.float32, x)
    check(dt_bias, "dt_bias", (Dm,), torch.float32, x)
    check(lens, "lens", (x.shape[0],), torch.int32, x)
    activations(B, "B", dims + 1)
    G = B.shape[-2]
    for t, name in ((B, "B"), (C, "C")):
        like_x(t, name, (*x.shape[:-1], G, N), x)
        if G > 1 and t.stride(-2) != N:
            raise ValueError(f"{name} must have contiguous groups (stride N)")
    a.B, a.T, a.D, a.N, a.G = x.shape[0], x.shape[1] if dims == 3 else 1, Dm, N, G
    a.softplus = int(softplus)
    a.lens, a.A, a.Dskip, a.dt_bias = _ptr(lens), _ptr(A), _ptr(D), _ptr(dt_bias)
    for name, t in (("x", x), ("dt", dt), ("z", z), ("B", B), ("C", C)):
        if t is not None:
            setattr(a, name + "_sb", t.stride(0))
            setattr(a, name + "_st", t.stride(1) if dims == 3 else 0)
    return a


def selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, softplus=True,
                       init_state=None, lens=None, want_final=True, y=None, final_state=None,
                       workspace="auto", stream=None):
    """x, dt, z [B,T,D] and B, C [B,T,G,N] in one type with any batch and token strides; A fp32
    [D,N]; D, dt_bias fp32 [D]; init_state fp32 [B,D,N] (None: zeros).  Returns (y [B,T,D],
    final_state fp32 [B,D,N] or None).  ``workspace``: "auto" lets few rows with many tokens
    be cut along the tokens, None runs without one, or a uint8 tensor to reuse."""
    a = _scan(x, dt, A, B, C, D, z, dt_bias, softplus, lens, 3)
    state = (a.B, a.D, a.N)
    check(init_state, "init_state", state, torch.float32, x)
    y = _new(y, x.shape, x.dtype, x)
    check(y, "y", x.shape, x.dtype, x)
    if want_final or final_state is not None:
        final_state = _new(final_state, state, torch.float32, x)
        check(final_state, "final_state", state, torch.float32, x)
    with launch(x, stream) as s:
        ws = scratch(dr.dr_selective_scan_fwd_workspace_bytes(a), x, workspace)
        dr.check(dr.dr_selective_scan_fwd(a, x, dt, B, C, z, init_state, y, final_state, ws,
                                          size_of(ws), s), "dr_selective_scan_fwd")
    return y, final_state


def selective_scan_bwd(x, dt, A, B, C, d_y, D=None, z=None, dt_bias=None, *, softplus=True,
                       init_state=None, d_final_state=None, lens=None, workspace="auto",
                       grads=None, stream=None):
    """Returns a dict of dx, ddt (of dt as given), dB, dC, with z dz, in x's type; dA, with D dD,
    with dt_bias ddt_bias, and with init_state dinit_state, in fp32.  ``grads`` may hold output
    tensors under these names."""
    a = _scan(x, dt, A, B, C, D, z, dt_bias, softplus, lens, 3)
    state = (a.B, a.D, a.N)
    check(init_state, "init_state", state, torch.float32, x)
    check(d_y, "d_y", x.shape, x.dtype, x)
    check(d_final_state, "d_final_state", state, torch.float32, x)
    f32 = torch.float32
    shapes = {"dx": (x.shape, x.dtype), "ddt": (x.shape, x.dtype), "dB": (B.shape, x.dtype),
              "dC": (C.shape, x.dtype), "dA": (A.shape, f32)}
    for name, given, shape in (("dz", z, x.shape), ("dD", D, (a.D,)), ("ddt_bias", dt_bias, (a.D,)),
                               ("dinit_state", init_state, state)):
        if given is not None:
            shapes[name] = (shape, x.dtype if name == "dz" else f32)
    g = dict(grads or {})
    for name, (shape, dtype) in shapes.items():
        g[name] = _new(g.get(name), shape, dtype, x)
        check(g[name], name, shape, dtype, x)
    gs = dr.DrScanGrads(*(_ptr(g.get(n)) for n in ("dx", "ddt", "dz", "dB", "dC", "dA", "dD",
                                                   "ddt_bias", "dinit_state")))
    with launch(x, stream) as s:
        ws = scratch(dr.dr_selective_scan_bwd_workspace_bytes(a), x, workspace)
        dr.check(dr.dr_selective_scan_bwd(a, x, dt, B, C, z, init_state, d_y, d_final_state, gs, ws,
                                          size_of(ws), s), "dr_selective_scan_bwd")
    return g


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, *, softplus=True,
                        state_out=None, y=None, stream=None):
    """One token: x, dt, z [B,D], B, C [B,G,N], state fp32 [B,D,N].  The new state goes to
    ``state_out`` (default: in place).  Returns (y [B,D], the new state)."""
    a = _scan(x, dt, A, B, C, D, z, dt_bias, softplus, None, 2)
    shape = (a.B, a.D, a.N)
    check(state, "state", shape, torch.float32, x)
    state_out = state if state_out is None else state_out
    check(state_out, "state_out", shape, torch.float32, x)
    y = _new(y, x.shape, x.dtype, x)
    check(y, "y", x.shape, x.dtype, x)
    with launch(x, stream) as s:
        dr.check(dr.dr_selective_scan_step(a, x, dt, B, C, z, state, state_out, y, s),
                 "dr_selective_scan_step")
    return y, state_out
