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
Work runs on ``stream``, a stream of x's device (a torch stream or a raw handle; default:
the current one), and the tensors passed in may be let go as soon as the call is back.
"""

from __future__ import annotations

import torch

from . import dr
from .tensors import activations, call, check, check_rows, on_stream, ptr, scratch

__all__ = ["short_conv_fwd", "short_conv_bwd", "short_conv_step", "selective_scan_fwd",
           "selective_scan_bwd", "selective_scan_step"]


def _given_or_new(t, name, shape, dtype, x, dev):
    if t is None:
        return x.new_empty(shape, dtype=dtype)
    check(t, name, shape, dtype, dev)
    return t


def _gradients(grads, shapes, x, dev):
    g = dict(grads or {})
    for name, (shape, dtype) in shapes.items():
        g[name] = _given_or_new(g.get(name), name, shape, dtype, x, dev)
    return g


# ------------------------------------------------------------------ short convolution

def _conv(x, weight, bias, silu, lens, dims):
    """The call's dr_conv and its device, its tensors checked."""
    code, dev = activations(x, "x", dims)
    D = x.shape[-1]
    if not torch.is_tensor(weight) or weight.dim() != 2:
        raise ValueError("weight must be a tensor [D, K]")
    K = weight.shape[1]
    check(weight, "weight", (D, K), torch.float32, dev)
    if bias is not None:
        check(bias, "bias", (D,), torch.float32, dev)
    if dims == 2:
        return dr.DrConv(code, x.shape[0], 1, D, K, silu, None, x.stride(0), 0), dev
    if lens is not None:
        check(lens, "lens", (x.shape[0],), torch.int32, dev)
    sb, st, _ = x.stride()
    return dr.DrConv(code, x.shape[0], x.shape[1], D, K, silu, ptr(lens), sb, st), dev


@on_stream
def short_conv_fwd(x, weight, bias=None, *, silu=True, init_state=None, lens=None, want_final=True,
                   y=None, final_state=None, stream=None):
    """x [B,T,D] (any batch and token strides), weight fp32 [D,K], bias fp32 [D], init_state
    [B,K-1,D] in x's type (the inputs before the first token, oldest first; None: zeros).
    ``final_state`` may be ``init_state``.  Returns (y [B,T,D], final_state [B,K-1,D] or None)."""
    a, dev = _conv(x, weight, bias, silu, lens, 3)
    state = (a.B, a.K - 1, a.D)
    if init_state is not None:
        check(init_state, "init_state", state, x.dtype, dev)
    y = _given_or_new(y, "y", x.shape, x.dtype, x, dev)
    if want_final or final_state is not None:
        final_state = _given_or_new(final_state, "final_state", state, x.dtype, x, dev)
    call("dr_short_conv_fwd", dev, dr.dr_short_conv_fwd, a, x, weight, bias, init_state, y,
         final_state)
    return y, final_state


@on_stream
def short_conv_bwd(x, weight, bias, d_y, *, silu=True, init_state=None, d_final_state=None,
                   lens=None, workspace="auto", grads=None, stream=None):
    """Returns dict(dx [B,T,D] in x's type, dweight fp32 [D,K], dbias fp32 [D]) and with
    init_state dinit_state [B,K-1,D].  ``grads`` may hold output tensors under these names."""
    a, dev = _conv(x, weight, bias, silu, lens, 3)
    state = (a.B, a.K - 1, a.D)
    check(d_y, "d_y", x.shape, x.dtype, dev)
    if d_final_state is not None:
        check(d_final_state, "d_final_state", state, x.dtype, dev)
    shapes = {"dx": (x.shape, x.dtype), "dweight": (weight.shape, torch.float32),
              "dbias": ((a.D,), torch.float32)}
    if init_state is not None:
        check(init_state, "init_state", state, x.dtype, dev)
        shapes["dinit_state"] = (state, x.dtype)
    g = _gradients(grads, shapes, x, dev)
    ws, n = scratch(dr.dr_short_conv_bwd_workspace_bytes, a, x, dev, workspace)
    call("dr_short_conv_bwd", dev, dr.dr_short_conv_bwd, a, x, weight, bias, init_state, d_y,
         d_final_state, g["dx"], g["dweight"], g["dbias"], g.get("dinit_state"), ws, n)
    return g


@on_stream
def short_conv_step(x, weight, bias, state, *, silu=True, state_out=None, y=None, stream=None):
    """One token: x [B,D], state [B,K-1,D].  The new state goes to ``state_out`` (default: in
    place).  Returns (y [B,D], the new state)."""
    a, dev = _conv(x, weight, bias, silu, None, 2)
    shape = (a.B, a.K - 1, a.D)
    check(state, "state", shape, x.dtype, dev)
    if state_out is None:
        state_out = state
    else:
        check(state_out, "state_out", shape, x.dtype, dev)
    y = _given_or_new(y, "y", x.shape, x.dtype, x, dev)
    call("dr_short_conv_step", dev, dr.dr_short_conv_step, a, x, weight, bias, state,
         state_out, y)
    return y, state_out


# ------------------------------------------------------------------ selective scan

def _scan(x, dt, A, B, C, D, z, dt_bias, softplus, lens, dims):
    """The call's dr_scan and its device, its tensors checked."""
    code, dev = activations(x, "x", dims)
    shape = x.shape
    Dm = shape[-1]
    f32 = torch.float32
    check_rows(dt, "dt", shape, x.dtype, dev)
    if z is not None:
        check_rows(z, "z", shape, x.dtype, dev)
    if not torch.is_tensor(A) or A.dim() != 2:
        raise ValueError("A must be a tensor [D, N]")
    N = A.shape[1]
    check(A, "A", (Dm, N), f32, dev)
    if D is not None:
        check(D, "D", (Dm,), f32, dev)
    if dt_bias is not None:
        check(dt_bias, "dt_bias", (Dm,), f32, dev)
    activations(B, "B", dims + 1)
    G = B.shape[-2]
    groups = (*shape[:-1], G, N)
    check_rows(B, "B", groups, x.dtype, dev)
    check_rows(C, "C", groups, x.dtype, dev)
    if G > 1 and (B.stride(-2) != N or C.stride(-2) != N):
        raise ValueError("B and C must have contiguous groups (stride N)")
    if lens is not None:
        check(lens, "lens", (shape[0],), torch.int32, dev)
    if dims == 3:
        strides = (*x.stride()[:2], *dt.stride()[:2], *(z.stride()[:2] if z is not None else (0, 0)),
                   *B.stride()[:2], *C.stride()[:2])
    else:
        strides = (x.stride(0), 0, dt.stride(0), 0, z.stride(0) if z is not None else 0, 0,
                   B.stride(0), 0, C.stride(0), 0)
    return dr.DrScan(code, shape[0], shape[1] if dims == 3 else 1, Dm, N, G, softplus, ptr(lens),
                     A.data_ptr(), ptr(D), ptr(dt_bias), *strides), dev


@on_stream
def selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, softplus=True,
                       init_state=None, lens=None, want_final=True, y=None, final_state=None,
                       workspace="auto", stream=None):
    """x, dt, z [B,T,D] and B, C [B,T,G,N] in one type with any batch and token strides; A fp32
    [D,N]; D, dt_bias fp32 [D]; init_state fp32 [B,D,N] (None: zeros).  Returns (y [B,T,D],
    final_state fp32 [B,D,N] or None).  ``workspace``: "auto" lets few rows with many tokens
    be cut along the tokens, None runs without one, or a uint8 tensor to reuse."""
    a, dev = _scan(x, dt, A, B, C, D, z, dt_bias, softplus, lens, 3)
    state = (a.B, a.D, a.N)
    if init_state is not None:
        check(init_state, "init_state", state, torch.float32, dev)
    y = _given_or_new(y, "y", x.shape, x.dtype, x, dev)
    if want_final or final_state is not None:
        final_state = _given_or_new(final_state, "final_state", state, torch.float32, x, dev)
    ws, n = scratch(dr.dr_selective_scan_fwd_workspace_bytes, a, x, dev, workspace)
    call("dr_selective_scan_fwd", dev, dr.dr_selective_scan_fwd, a, x, dt, B, C, z,
         init_state, y, final_state, ws, n)
    return y, final_state


@on_stream
def selective_scan_bwd(x, dt, A, B, C, d_y, D=None, z=None, dt_bias=None, *, softplus=True,
                       init_state=None, d_final_state=None, lens=None, workspace="auto",
                       grads=None, stream=None):
    """Returns a dict of dx, ddt (of dt as given), dB, dC, with z dz, in x's type; dA, with D dD,
    with dt_bias ddt_bias, and with init_state dinit_state, in fp32.  ``grads`` may hold output
    tensors under these names."""
    a, dev = _scan(x, dt, A, B, C, D, z, dt_bias, softplus, lens, 3)
    state = (a.B, a.D, a.N)
    f32 = torch.float32
    check(d_y, "d_y", x.shape, x.dtype, dev)
    if d_final_state is not None:
        check(d_final_state, "d_final_state", state, f32, dev)
    shapes = {"dx": (x.shape, x.dtype), "ddt": (x.shape, x.dtype), "dB": (B.shape, x.dtype),
              "dC": (C.shape, x.dtype), "dA": (A.shape, f32)}
    if z is not None:
        shapes["dz"] = (x.shape, x.dtype)
    if D is not None:
        shapes["dD"] = ((a.D,), f32)
    if dt_bias is not None:
        shapes["ddt_bias"] = ((a.D,), f32)
    if init_state is not None:
        check(init_state, "init_state", state, f32, dev)
        shapes["dinit_state"] = (state, f32)
    g = _gradients(grads, shapes, x, dev)
    gs = dr.DrScanGrads(*(ptr(g.get(n)) for n in ("dx", "ddt", "dz", "dB", "dC", "dA", "dD",
                                                  "ddt_bias", "dinit_state")))
    ws, n = scratch(dr.dr_selective_scan_bwd_workspace_bytes, a, x, dev, workspace)
    call("dr_selective_scan_bwd", dev, dr.dr_selective_scan_bwd, a, x, dt, B, C, z,
         init_state, d_y, d_final_state, gs, ws, n)
    return g


@on_stream
def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, *, softplus=True,
                        state_out=None, y=None, stream=None):
    """One token: x, dt, z [B,D], B, C [B,G,N], state fp32 [B,D,N].  The new state goes to
    ``state_out`` (default: in place).  Returns (y [B,D], the new state)."""
    a, dev = _scan(x, dt, A, B, C, D, z, dt_bias, softplus, None, 2)
    shape = (a.B, a.D, a.N)
    check(state, "state", shape, torch.float32, dev)
    if state_out is None:
        state_out = state
    else:
        check(state_out, "state_out", shape, torch.float32, dev)
    y = _given_or_new(y, "y", x.shape, x.dtype, x, dev)
    call("dr_selective_scan_step", dev, dr.dr_selective_scan_step, a, x, dt, B, C, z, state,
         state_out, y)
    return y, state_out
