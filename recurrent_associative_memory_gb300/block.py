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

__all__ = ["linear_fwd", "linear_bwd", "block_norm_fwd", "block_norm_bwd"]

_SLOPES = {torch.bfloat16: torch.float16, torch.float32: torch.float32}
_FP32 = torch.float32


def _given_or_new(t, name, shape, dtype, like, dev):
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    check(t, name, shape, dtype, dev)
    return t


def _rows(t, name):
    """(rows, row stride) of a tensor of 2 or 3 dimensions as one list of rows."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        return shape[0], stride[0]
    B, T = shape[0], shape[1]
    if B == 1 or stride[0] == T * stride[1]:
        return B * T, stride[1]
    if T == 1:
        return B, stride[0]
    raise ValueError(f"{name} must step evenly over its rows: batch stride {stride[0]} is not "
                     f"{T} tokens of {stride[1]}")


def _act(name, what):
    code = dr.ACT_IDS.get(name)
    if code is None:
        raise ValueError(f"{what} must be one of {', '.join(dr.ACT_IDS)}, got {name!r}")
    return code


def _dims(t):
    d = t.dim() if torch.is_tensor(t) else 2
    return d if d == 3 else 2


# ------------------------------------------------------------------ matrix product

def _linear(x, weight, act):
    """The call's dr_linear and its device, its tensors checked; a weight [K,N] may be the
    transpose of a matrix [N,K] (``w.t()``)."""
    code, dev = activations(x, "x", _dims(x))
    if not torch.is_tensor(weight) or weight.dim() != 2 or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"weight must be a tensor [{x.shape[-1]}, N]")
    K, N = weight.shape
    s0, s1 = weight.stride()
    if weight.dtype is not x.dtype or weight.device != x.device:
        raise TypeError(f"weight must be {x.dtype} on {x.device}, got {weight.dtype} on {weight.device}")
    if s1 == 1 or N == 1 and s0 != 1:
        t, ws = 0, s0
    elif s0 == 1 or K == 1:
        t, ws = 1, s1
    else:
        raise ValueError("weight must have contiguous rows or contiguous columns")
    M, xs = _rows(x, "x")
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
        check_rows(residual, "residual", shape, x.dtype, dev)
        a.r_s = _rows(residual, "residual")[1]
    y = _given_or_new(y, "y", shape, x.dtype, x, dev)
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
    g = dict(grads or {})
    if want_dx:
        g["dx"] = _given_or_new(g.get("dx"), "dx", x.shape, x.dtype, x, dev)
    if want_dweight:
        if a.w_transposed:
            given = g.get("dweight")
            if given is not None:
                check(given.t(), "dweight.t()", (a.N, a.K), x.dtype, dev)
            g["dweight"] = x.new_empty((a.N, a.K)).t() if given is None else given
        else:
            g["dweight"] = _given_or_new(g.get("dweight"), "dweight", (a.K, a.N), x.dtype, x, dev)
    if want_dbias:
        g["dbias"] = _given_or_new(g.get("dbias"), "dbias", (a.N,), x.dtype, x, dev)
    ws, n = scratch(dr.dr_linear_bwd_workspace_bytes, a, x, dev, workspace)
    call("dr_linear_bwd", dev, dr.dr_linear_bwd, a, x, weight, d_y, slope,
         g["dx"] if want_dx else None, g["dweight"] if want_dweight else None,
         g["dbias"] if want_dbias else None, ws, n)
    return g


# ------------------------------------------------------------------ norms around a block

def _block_norm(h, branch, gate, gate_act, scale, post_norm, post_weight, pre_weight, eps, dtype):
    """The call's dr_block_norm, its device and the activations' type, its tensors checked."""
    h_code, dev = activations(h, "h", _dims(h))
    if branch is not None:
        if dtype is not None and torch.is_tensor(branch) and dtype is not branch.dtype:
            raise TypeError(f"dtype {dtype} is not the branch's, {branch.dtype}")
        code, _ = activations(branch, "branch", h.dim())
        check_rows(branch, "branch", h.shape, branch.dtype, dev)
        dtype = branch.dtype
    else:
        dtype = h.dtype if dtype is None else dtype
        code = DTYPES.get(dtype)
        if code is None:
            raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    M, hs = _rows(h, "h")
    D = h.shape[-1]
    a = dr.DrBlockNorm(code, h_code, M, D, bool(post_norm), _act(gate_act, "gate_act"), eps, hs, 0, 0)
    if branch is not None:
        a.b_s = _rows(branch, "branch")[1]
    if gate is not None:
        check_rows(gate, "gate", h.shape, dtype, dev)
        a.g_s = _rows(gate, "gate")[1]
    for t, name in ((scale, "scale"), (post_weight, "post_weight"), (pre_weight, "pre_weight")):
        if t is not None:
            check(t, name, (D,), _FP32, dev)
    return a, dev, dtype


@on_stream
def block_norm_fwd(h, branch=None, *, gate=None, gate_act="none", scale=None, post_norm=False,
                   post_weight=None, pre_weight=None, eps=1e-6, want_y=True, dtype=None, y=None,
                   h_out=None, stream=None):
    """h, branch, gate [M,D] or [B,T,D]; scale, post_weight, pre_weight fp32 [D].  branch and
    gate share a type, h has the same or fp32.  ``post_norm``: the branch's norm is taken.
    Without a branch y is the norm of h, in ``dtype`` (default: h's).  ``h_out`` may be h.
    Returns (y or None without ``want_y``, h'); h' is h itself without a branch."""
    a, dev, dtype = _block_norm(h, branch, gate, gate_act, scale, post_norm, post_weight,
                                pre_weight, eps, dtype)
    if want_y or y is not None:
        y = _given_or_new(y, "y", h.shape, dtype, h, dev)
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
    the last three fp32 [D].  ``grads`` may hold output tensors under these names."""
    a, dev, dtype = _block_norm(h, branch, gate, gate_act, scale, post_norm, post_weight,
                                pre_weight, eps, dtype)
    if d_h is not None:
        check(d_h, "d_h", h.shape, h.dtype, dev)
    if d_y is not None:
        check(d_y, "d_y", h.shape, dtype, dev)
    vec, given = (a.D,), dict(grads or {})
    g = {}
    for name, there, shape, kind in (
            ("dh", h, h.shape, h.dtype), ("dbranch", branch, h.shape, dtype),
            ("dgate", gate, h.shape, dtype), ("dscale", scale, vec, _FP32),
            ("dpost_weight", post_weight, vec, _FP32),
            ("dpre_weight", None if d_y is None else pre_weight, vec, _FP32)):
        if there is not None:
            g[name] = _given_or_new(given.get(name), name, shape, kind, h, dev)
    ws, n = (scratch(dr.dr_block_norm_bwd_workspace_bytes, a, h, dev, workspace)
             if "dscale" in g or "dpost_weight" in g or "dpre_weight" in g else (None, 0))
    out = dr.DrBlockNormGrads(*(ptr(g.get(k)) for k in _GRADS))
    call("dr_block_norm_bwd", dev, dr.dr_block_norm_bwd, a, h, branch, gate, scale, post_weight,
         pre_weight, d_h, d_y, out, ws, n)
    return g
