"""What stands around a mixer in a block: projections with their epilogue, and the norms
before and after the mixer with its gate and residual scale.

``linear_fwd`` / ``linear_bwd``: ``y = act(x W + bias) + residual`` and its gradients, for
prompts, training and single tokens alike (few rows take kernels of their own).

``block_norm_fwd`` / ``block_norm_bwd``, over a residual stream ``h`` and what a mixer gave::

    h' = h + scale * f(gate) * n(branch; post_weight)
    y  = n(h'; pre_weight)              n(x; w) = w * x / sqrt(mean(x^2) + eps)

so one call ends a block (its norm, gate, scale and residual) and begins the next one (its
norm).  The norm takes h' as it was summed, before it is rounded to the stream's type.

Activations and gates are "none" (x itself), "relu", "silu", "gelu_tanh" or "sigmoid".
Rows may be given as [M,D] or [B,T,D].  Tensors that are read may have any row stride;
outputs are contiguous.

The functions allocate outputs and call ``dr``; they compute nothing themselves.  Work runs on
``stream``, a stream of the first tensor's device (a torch stream or a raw handle; default: the
current one), and the tensors passed in may be let go as soon as the call is back.
"""

from __future__ import annotations

import torch

from . import dr
from .tensors import DTYPES, activations, call, check, check_rows, on_stream, ptr, scratch

__all__ = ["linear_fwd", "linear_bwd", "block_norm_fwd", "block_norm_bwd", "MAX_CHANNELS"]

MAX_CHANNELS = 8192   # of a norm's row

_SLOPES = {torch.bfloat16: torch.float16, torch.float32: torch.float32}
_FP32 = torch.float32
_empty, _empty_like = torch.empty, torch.empty_like


# A call is a few microseconds of GPU work: what follows spends its time on the usual case.

def _given_or_new(t, name, shape, dtype, like, dev):
    """A contiguous tensor; ``like`` is on device dev."""
    if t is None:
        if like.shape == shape and like.dtype is dtype and like.is_contiguous():
            return _empty_like(like)
        return _empty(shape, dtype=dtype, device=like.device)
    check(t, name, shape, dtype, dev)
    return t


def _rows(t, name):
    """(rows, row stride) of a tensor of 2 or 3 dimensions as one list of rows."""
    shape = t.shape
    if len(shape) == 2:
        return shape[0], t.stride(0)
    B, T = shape[0], shape[1]
    sb, st, _ = t.stride()
    if B == 1 or sb == T * st:
        return B * T, st
    if T == 1:
        return B, sb
    raise ValueError(f"{name} must step evenly over its rows: batch stride {sb} is not "
                     f"{T} tokens of {st}")


def _row_stride(t, name, shape, dtype, dev):
    """As ``check_rows``, and the row stride."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return shape[-1]
    except AttributeError:
        pass
    check_rows(t, name, shape, dtype, dev)
    return _rows(t, name)[1]


def _act(name, what):
    code = dr.ACT_IDS.get(name)
    if code is None:
        raise ValueError(f"{what} must be one of {', '.join(dr.ACT_IDS)}, got {name!r}")
    return code


def _first(t, name):
    """(dr_dtype, device, rows, row stride) of a call's first tensor."""
    try:
        code, dev, shape = DTYPES[t.dtype], t.get_device(), t.shape
        if dev >= 0 and t.is_contiguous() and 2 <= len(shape) <= 3:
            D = shape[-1]
            return code, dev, shape[0] if len(shape) == 2 else shape[0] * shape[1], D
    except (AttributeError, KeyError):
        pass
    d = t.dim() if torch.is_tensor(t) else 2
    code, dev = activations(t, name, d if d == 3 else 2)
    return code, dev, *_rows(t, name)


# ------------------------------------------------------------------ matrix product

def _linear(x, weight, act):
    """The call's dr_linear and its device, its tensors checked; a weight [K,N] may be the
    transpose of a matrix [N,K] (``w.t()``)."""
    code, dev, M, xs = _first(x, "x")
    if not torch.is_tensor(weight) or weight.dim() != 2 or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"weight must be a tensor [{x.shape[-1]}, N]")
    K, N = weight.shape
    s0, s1 = weight.stride()
    if weight.dtype is not x.dtype or weight.get_device() != dev:
        raise TypeError(f"weight must be {x.dtype} on {x.device}, got {weight.dtype} on {weight.device}")
    if s1 == 1 or N == 1 and s0 != 1:
        t, ws = 0, s0
    elif s0 == 1 or K == 1:
        t, ws = 1, s1
    else:
        raise ValueError("weight must have contiguous rows or contiguous columns")
    return dr.DrLinear(code, _act(act, "act"), M, K, N, t, xs, ws, 0), dev


@on_stream
def linear_fwd(x, weight, bias=None, *, act="none", residual=None, want_slope=False, y=None,
               slope=None, workspace="auto", stream=None):
    """x [M,K] or [B,T,K], weight [K,N] in x's type (rows or columns contiguous, so also
    ``w.t()`` of a matrix [N,K]), bias [N], residual [..,N] in x's type; y may be residual.
    Returns (y [..,N], slope).  With ``want_slope`` slope [..,N] is act'(x W + bias), which
    ``linear_bwd`` takes: fp16 for bf16, fp32 for fp32; None otherwise, or where act is
    "none"."""
    a, dev = _linear(x, weight, act)
    shape = (*x.shape[:-1], a.N)
    if bias is not None:
        check(bias, "bias", (a.N,), x.dtype, dev)
    if residual is not None:
        a.r_s = _row_stride(residual, "residual", shape, x.dtype, dev)
    y = _given_or_new(y, "y", shape, x.dtype, x if residual is None else residual, dev)
    if (want_slope or slope is not None) and a.act:
        slope = _given_or_new(slope, "slope", shape, _SLOPES[x.dtype], x, dev)
    else:
        slope = None
    ws, n = scratch(dr.dr_linear_fwd_workspace_bytes, a, x, dev, workspace)
    call("dr_linear_fwd", dev, dr.dr_linear_fwd, a, x, weight, bias, residual, y, slope, ws, n)
    return y, slope


@on_stream
def linear_bwd(x, weight, d_y, *, slope=None, want_dx=True, want_dweight=True, want_dbias=True,
               workspace="auto", grads=None, stream=None):
    """d_y [..,N]; ``slope`` from the forward (None: act "none").  Returns dict(dx [..,K],
    dweight [K,N] (columns contiguous where weight's are), dbias [N]), all in x's type, without
    the ones that are not wanted.  The residual's gradient is d_y.  ``grads`` may hold output
    tensors under these names; dweight has weight's contiguous direction."""
    a, dev = _linear(x, weight, "none" if slope is None else "sigmoid")
    shape = (*x.shape[:-1], a.N)
    check(d_y, "d_y", shape, x.dtype, dev)
    if slope is not None:
        check(slope, "slope", shape, _SLOPES[x.dtype], dev)
    given, g = grads or {}, {}
    if want_dx:
        g["dx"] = _given_or_new(given.get("dx"), "dx", x.shape, x.dtype, x, dev)
    if want_dweight:
        dw = given.get("dweight")
        if a.w_transposed:
            if dw is not None:
                check(dw.t(), "dweight.t()", (a.N, a.K), x.dtype, dev)
            g["dweight"] = x.new_empty((a.N, a.K)).t() if dw is None else dw
        else:
            g["dweight"] = _given_or_new(dw, "dweight", (a.K, a.N), x.dtype, x, dev)
    if want_dbias:
        g["dbias"] = _given_or_new(given.get("dbias"), "dbias", (a.N,), x.dtype, x, dev)
    ws, n = scratch(dr.dr_linear_bwd_workspace_bytes, a, x, dev, workspace)
    call("dr_linear_bwd", dev, dr.dr_linear_bwd, a, x, weight, d_y, slope,
         g["dx"] if want_dx else None, g["dweight"] if want_dweight else None,
         g["dbias"] if want_dbias else None, ws, n)
    return g


# ------------------------------------------------------------------ norms around a block

def _block_norm(h, branch, gate, gate_act, scale, post_norm, post_weight, pre_weight, eps, dtype):
    """The call's dr_block_norm, its device and the activations' type, its tensors checked."""
    h_code, dev, M, hs = _first(h, "h")
    shape, bs, gs = h.shape, 0, 0
    D = shape[-1]
    if branch is not None:
        kind = getattr(branch, "dtype", None)
        if dtype is not None and kind is not None and dtype is not kind:
            raise TypeError(f"dtype {dtype} is not the branch's, {kind}")
        code = DTYPES.get(kind)
        if code is None:
            activations(branch, "branch", len(shape))
        bs = _row_stride(branch, "branch", shape, kind, dev)
        dtype = kind
    else:
        dtype = h.dtype if dtype is None else dtype
        code = DTYPES.get(dtype)
        if code is None:
            raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    if gate is not None:
        gs = _row_stride(gate, "gate", shape, dtype, dev)
    a = dr.DrBlockNorm(code, h_code, M, D, 1 if post_norm else 0, _act(gate_act, "gate_act"), eps, hs, bs, gs)
    for t, name in ((scale, "scale"), (post_weight, "post_weight"), (pre_weight, "pre_weight")):
        if t is not None:
            check(t, name, (D,), _FP32, dev)
    return a, dev, dtype


@on_stream
def block_norm_fwd(h, branch=None, *, gate=None, gate_act="none", scale=None, post_norm=False,
                   post_weight=None, pre_weight=None, eps=1e-6, want_y=True, dtype=None, y=None,
                   h_out=None, stream=None):
    """h, branch, gate [M,D] or [B,T,D], D up to ``MAX_CHANNELS``; scale, post_weight, pre_weight
    fp32 [D].  branch and gate share a type, h has the same or fp32.  ``post_norm``: the branch's
    norm is taken.
    Without a branch y is the norm of h, in ``dtype`` (default: h's).  ``h_out`` may be h.
    Returns (y or None without ``want_y``, h'); h' is h itself without a branch."""
    a, dev, dtype = _block_norm(h, branch, gate, gate_act, scale, post_norm, post_weight,
                                pre_weight, eps, dtype)
    if want_y or y is not None:
        y = _given_or_new(y, "y", h.shape, dtype, h if branch is None else branch, dev)
    if branch is not None:
        h_out = _given_or_new(h_out, "h_out", h.shape, h.dtype, h, dev)
    elif h_out is not None:
        raise ValueError("h_out needs a branch")
    call("dr_block_norm_fwd", dev, dr.dr_block_norm_fwd, a, h, branch, gate, scale, post_weight,
         pre_weight, h_out, y)
    return y, h if branch is None else h_out


_GRADS = ("dh", "dbranch", "dgate", "dscale", "dpost_weight", "dpre_weight")


@on_stream
def block_norm_bwd(h, branch=None, *, d_h=None, d_y=None, gate=None, gate_act="none", scale=None,
                   post_norm=False, post_weight=None, pre_weight=None, eps=1e-6, dtype=None,
                   workspace="auto", grads=None, stream=None):
    """The forward's inputs (h as it was before the call) and the gradients of its outputs: d_h
    [..,D] in h's type, d_y in the branch's; one of them may be None (0).  Returns dict(dh, and
    where the input is given dbranch, dgate, dscale, dpost_weight and, with d_y, dpre_weight);
    the last three fp32 [D].  ``grads`` may hold output tensors under these names; dh may be d_h or
    h, dbranch branch and dgate gate, no other two may be one."""
    a, dev, dtype = _block_norm(h, branch, gate, gate_act, scale, post_norm, post_weight,
                                pre_weight, eps, dtype)
    if d_h is not None:
        check(d_h, "d_h", h.shape, h.dtype, dev)
    if d_y is not None:
        check(d_y, "d_y", h.shape, dtype, dev)
    given = grads or {}
    g = {"dh": _given_or_new(given.get("dh"), "dh", h.shape, h.dtype, h, dev)}
    if branch is not None:
        g["dbranch"] = _given_or_new(given.get("dbranch"), "dbranch", h.shape, dtype, branch, dev)
    if gate is not None:
        g["dgate"] = _given_or_new(given.get("dgate"), "dgate", h.shape, dtype, gate, dev)
    ws, n, vec = None, 0, (a.D,)
    for name, t in (("dscale", scale), ("dpost_weight", post_weight),
                    ("dpre_weight", None if d_y is None else pre_weight)):
        if t is not None:
            g[name] = _given_or_new(given.get(name), name, vec, _FP32, t, dev)
            n = 1
    if n:
        ws, n = scratch(dr.dr_block_norm_bwd_workspace_bytes, a, h, dev, workspace)
    out = dr.DrBlockNormGrads(*(ptr(g.get(k)) for k in _GRADS))
    call("dr_block_norm_bwd", dev, dr.dr_block_norm_bwd, a, h, branch, gate, scale, post_weight,
         pre_weight, d_h, d_y, out, ws, n)
    return g
