"""Attention with a sliding window and sinks: prompts, training, single tokens.

A query at position p sees key j where ``j <= p``, ``j < lens[b]`` and
``p - j < window or j < n_sink``: the last ``window`` positions and the first
``n_sink``.  A row that sees nothing gives 0 (log-sum-exp -inf).  Heads have 64
or 128 channels, and H query heads share Hkv key/value heads.

``lens`` bounds the keys, not the rows: a padded row at ``p >= lens[b]`` still sees the
keys before ``lens[b]`` that its window holds.  Its output is not 0, and its ``d_out``
reaches dk and dv, so that has to be 0 there.  (The convolution and the scan in ``ssm``
give 0 behind a sequence's end and take no gradient from there.)

``window_attn_fwd`` / ``window_attn_bwd`` run a prompt, the next piece of one
(``q_start``) or a training step.  For decoding, ``window_cache`` makes a cache of
constant size, ``window_cache_fill`` lays a prompt's keys and values out in it and
``window_attn_step`` takes it one token further.

The functions allocate outputs and call ``dr``; they compute nothing themselves.
Work runs on ``stream``, a stream of q's device (a torch stream or a raw handle; default:
the current one), and the tensors passed in may be let go as soon as the call is back.
"""

from __future__ import annotations

import torch

from . import dr
from .tensors import activations, call, check, check_rows, on_stream, ptr, scratch

__all__ = ["window_attn_fwd", "window_attn_bwd", "window_attn_step", "window_cache",
           "window_cache_fill"]


_MOST = 0x7fffffff


def _limits(window, n_sink, q_start=0):
    """The three as C ints.  A window wider than every position is the widest one."""
    if window > _MOST:
        window = _MOST
    if not (-_MOST <= window and -_MOST <= n_sink <= _MOST and -_MOST <= q_start <= _MOST):
        raise ValueError(f"window {window}, n_sink {n_sink} and q_start {q_start} must fit 32 bits")
    return window, n_sink, q_start


def _describe(q, k, v, window, n_sink, q_start, lens, scale):
    """The call's dr_attn and its device, its tensors checked."""
    code, dev = activations(q, "q", 4)
    activations(k, "k", 4)
    B, T, H, d = q.shape
    S, Hkv = k.shape[1:3]
    keys = (B, S, Hkv, d)
    check_rows(k, "k", keys, q.dtype, dev)
    check_rows(v, "v", keys, q.dtype, dev)
    if lens is not None:
        check(lens, "lens", (B,), torch.int32, dev)
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    return dr.DrAttn(code, B, T, S, H, Hkv, d, *_limits(window, n_sink, q_start), _scale(scale), ptr(lens),
                     qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2]), dev


def _scale(scale):
    if scale is None:
        return 0.0   # 1 / sqrt(d)
    if not scale > 0:
        raise ValueError(f"scale must be positive, got {scale}")
    return scale


@on_stream
def window_attn_fwd(q, k, v, window, n_sink=0, *, q_start=0, lens=None, scale=None, want_lse=False,
                    out=None, lse=None, stream=None):
    """Returns (out [B,T,H,d], lse fp32 [B,H,T] or None).

    q [B,T,H,d] stands at positions q_start .. q_start+T-1; k, v [B,S,Hkv,d] at 0 .. S-1.
    They may be slices with any batch, token and head strides of whole 16 bytes; expanded
    ones (stride 0) run on the CUDA cores, in bf16 far slower than a contiguous copy.
    ``lens`` int32 [B]: the sequences' real keys.  ``scale``: default 1/sqrt(d)."""
    a, dev = _describe(q, k, v, window, n_sink, q_start, lens, scale)
    if out is None:
        out = q.new_empty(q.shape)
    else:
        check(out, "out", q.shape, q.dtype, dev)
    if lse is not None:
        check(lse, "lse", (a.B, a.H, a.T), torch.float32, dev)
    elif want_lse:
        lse = q.new_empty((a.B, a.H, a.T), dtype=torch.float32)
    call("dr_window_attn_fwd", dev, dr.dr_window_attn_fwd, a, q, k, v, out, lse)
    return out, lse


@on_stream
def window_attn_bwd(q, k, v, out, lse, d_out, window, n_sink=0, *, q_start=0, lens=None, scale=None,
                    workspace="auto", grads=None, stream=None):
    """Returns dict(dq [B,T,H,d], dk, dv [B,S,Hkv,d]) in q's type, from the forward's out
    and lse.  ``grads`` may hold output tensors under these names."""
    a, dev = _describe(q, k, v, window, n_sink, q_start, lens, scale)
    check(out, "out", q.shape, q.dtype, dev)
    check(lse, "lse", (a.B, a.H, a.T), torch.float32, dev)
    check(d_out, "d_out", q.shape, q.dtype, dev)
    g = dict(grads or {})
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        if g.get(name) is None:
            g[name] = q.new_empty(t.shape)
        else:
            check(g[name], name, t.shape, q.dtype, dev)
    ws, n = scratch(dr.dr_window_attn_bwd_workspace_bytes, a, q, dev, workspace)
    call("dr_window_attn_bwd", dev, dr.dr_window_attn_bwd, a, q, k, v, out, lse, d_out,
         g["dq"], g["dk"], g["dv"], ws, n)
    return g


def window_cache(B, Hkv, d, window, n_sink=0, dtype=torch.bfloat16, device="cuda"):
    """An empty cache: (k_cache, v_cache) [B,Hkv,n_sink+window,d].  Slots that no position
    has reached are never read, so they are not cleared."""
    return tuple(torch.empty(B, Hkv, n_sink + window, d, dtype=dtype, device=device)
                 for _ in range(2))


def _check_cache(k_cache, v_cache, B, Hkv, slots, d, dtype, dev):
    check(k_cache, "k_cache", (B, Hkv, slots, d), dtype, dev)
    check(v_cache, "v_cache", (B, Hkv, slots, d), dtype, dev)


@on_stream
def window_cache_fill(k, v, k_cache, v_cache, window, n_sink=0, *, lens=None, stream=None):
    """Lays a prompt's k, v [B,S,Hkv,d] out in the caches, for decoding to go on at position
    lens[b] (default S)."""
    a, dev = _describe(k, k, v, window, n_sink, 0, lens, None)
    _check_cache(k_cache, v_cache, a.B, a.Hkv, n_sink + window, a.d, k.dtype, dev)
    call("dr_window_cache_fill", dev, dr.dr_window_cache_fill, a, k, v, k_cache, v_cache)


@on_stream
def window_attn_step(q, k, v, k_cache, v_cache, pos, window, n_sink=0, *, scale=None, out=None,
                     workspace="auto", stream=None):
    """One token per sequence: writes k, v [B,Hkv,d] at positions pos (int32 [B], on the
    device) into the caches and returns out [B,H,d].  A sequence with pos < 0 is left alone
    and gives 0.  ``workspace``: "auto" lets few sequences with a long cache be cut along
    the slots, None runs without one, or a uint8 tensor to reuse."""
    code, dev = activations(q, "q", 3)
    activations(k, "k", 3)
    B, H, d = q.shape
    Hkv = k.shape[1]
    check(q, "q", (B, H, d), q.dtype, dev)
    check(k, "k", (B, Hkv, d), q.dtype, dev)
    check(v, "v", (B, Hkv, d), q.dtype, dev)
    check(pos, "pos", (B,), torch.int32, dev)
    _check_cache(k_cache, v_cache, B, Hkv, n_sink + window, d, q.dtype, dev)
    a = dr.DrAttn(code, B, 1, 1, H, Hkv, d, *_limits(window, n_sink), _scale(scale))
    if out is None:
        out = q.new_empty(q.shape)
    else:
        check(out, "out", q.shape, q.dtype, dev)
    ws, n = scratch(dr.dr_window_attn_step_workspace_bytes, a, q, dev, workspace)
    call("dr_window_attn_step", dev, dr.dr_window_attn_step, a, q, k, v, k_cache, v_cache,
         pos, out, ws, n)
    return out
