"""Attention with a sliding window and sinks: prompts, training, single tokens.

A query at position p sees key j where ``j <= p``, ``j < lens[b]`` and
``p - j < window or j < n_sink``: the last ``window`` positions and the first
``n_sink``.  A row that sees nothing gives 0 (log-sum-exp -inf).  Heads have 64
or 128 channels, and H query heads share Hkv key/value heads.

``window_attn_fwd`` / ``window_attn_bwd`` run a prompt, the next piece of one
(``q_start``) or a training step.  For decoding, ``window_cache`` makes a cache of
constant size, ``window_cache_fill`` lays a prompt's keys and values out in it and
``window_attn_step`` takes it one token further.

The functions allocate outputs and call ``dr``; they compute nothing themselves.
Work runs on ``stream`` (default: the current one) of q's device.
"""

from __future__ import annotations

import torch

from . import dr
from .tensors import activations, check, launch, like_x, scratch, size_of

__all__ = ["window_attn_fwd", "window_attn_bwd", "window_attn_step", "window_cache",
           "window_cache_fill"]


def _describe(q, k, v, window, n_sink, q_start, lens, scale):
    a = dr.DrAttn()
    a.dtype = activations(q, "q", 4)
    B, T, H, d = q.shape
    activations(k, "k", 4)
    S, Hkv = k.shape[1:3]
    like_x(k, "k", (B, S, Hkv, d), q)
    like_x(v, "v", (B, S, Hkv, d), q)
    check(lens, "lens", (B,), torch.int32, q)
    a.B, a.T, a.S, a.H, a.Hkv, a.d = B, T, S, H, Hkv, d
    a.window, a.n_sink, a.q_start = window, n_sink, q_start
    a.scale = 0.0 if scale is None else _positive(scale)
    a.lens = None if lens is None else lens.data_ptr()
    a.q_sb, a.q_st, a.q_sh = q.stride()[:3]
    a.k_sb, a.k_st, a.k_sh = k.stride()[:3]
    a.v_sb, a.v_st, a.v_sh = v.stride()[:3]
    return a


def _positive(scale):
    if not scale > 0:
        raise ValueError(f"scale must be positive, got {scale}")
    return float(scale)


def window_attn_fwd(q, k, v, window, n_sink=0, *, q_start=0, lens=None, scale=None, want_lse=False,
                    out=None, lse=None, stream=None):
    """Returns (out [B,T,H,d], lse fp32 [B,H,T] or None).

    q [B,T,H,d] stands at positions q_start .. q_start+T-1; k, v [B,S,Hkv,d] at 0 .. S-1.
    They may be slices with any batch, token and head strides of whole 16 bytes.
    ``lens`` int32 [B]: the sequences' real keys.  ``scale``: default 1/sqrt(d)."""
    a = _describe(q, k, v, window, n_sink, q_start, lens, scale)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(a.B, a.H, a.T, dtype=torch.float32, device=q.device)
    check(out, "out", q.shape, q.dtype, q)
    check(lse, "lse", (a.B, a.H, a.T), torch.float32, q)
    with launch(q, stream) as s:
        dr.check(dr.dr_window_attn_fwd(a, q, k, v, out, lse, s), "dr_window_attn_fwd")
    return out, lse


def window_attn_bwd(q, k, v, out, lse, d_out, window, n_sink=0, *, q_start=0, lens=None, scale=None,
                    workspace="auto", grads=None, stream=None):
    """Returns dict(dq [B,T,H,d], dk, dv [B,S,Hkv,d]) in q's type, from the forward's out
    and lse.  ``grads`` may hold output tensors under these names."""
    a = _describe(q, k, v, window, n_sink, q_start, lens, scale)
    check(out, "out", q.shape, q.dtype, q)
    check(lse, "lse", (a.B, a.H, a.T), torch.float32, q)
    check(d_out, "d_out", q.shape, q.dtype, q)
    g = dict(grads or {})
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        if g.get(name) is None:
            g[name] = torch.empty(t.shape, dtype=q.dtype, device=q.device)
        check(g[name], name, t.shape, q.dtype, q)
    with launch(q, stream) as s:
        ws = scratch(dr.dr_window_attn_bwd_workspace_bytes(a), q, workspace)
        dr.check(dr.dr_window_attn_bwd(a, q, k, v, out, lse, d_out, g["dq"], g["dk"], g["dv"], ws,
                                       size_of(ws), s), "dr_window_attn_bwd")
    return g


def window_cache(B, Hkv, d, window, n_sink=0, dtype=torch.bfloat16, device="cuda"):
    """An empty cache: (k_cache, v_cache) [B,Hkv,n_sink+window,d].  Slots that no position
    has reached are never read, so they are not cleared."""
    return tuple(torch.empty(B, Hkv, n_sink + window, d, dtype=dtype, device=device)
                 for _ in range(2))


def _cache(k_cache, v_cache, window, n_sink, B, Hkv, d, like):
    shape = (B, Hkv, n_sink + window, d)
    check(k_cache, "k_cache", shape, like.dtype, like)
    check(v_cache, "v_cache", shape, like.dtype, like)


def window_cache_fill(k, v, k_cache, v_cache, window, n_sink=0, *, lens=None, stream=None):
    """Lays a prompt's k, v [B,S,Hkv,d] out in the caches, for decoding to go on at position
    lens[b] (default S)."""
    a = _describe(k, k, v, window, n_sink, 0, lens, None)
    _cache(k_cache, v_cache, window, n_sink, a.B, a.Hkv, a.d, k)
    with launch(k, stream) as s:
        dr.check(dr.dr_window_cache_fill(a, k, v, k_cache, v_cache, s), "dr_window_cache_fill")


def window_attn_step(q, k, v, k_cache, v_cache, pos, window, n_sink=0, *, scale=None, out=None,
                     workspace="auto", stream=None):
    """One token per sequence: writes k, v [B,Hkv,d] at positions pos (int32 [B], on the
    device) into the caches and returns out [B,H,d].  A sequence with pos < 0 is left alone
    and gives 0.  ``workspace``: "auto" lets few sequences with a long cache be cut along
    the slots, None runs without one, or a uint8 tensor to reuse."""
    a = dr.DrAttn()
    a.dtype = activations(q, "q", 3)
    B, H, d = q.shape
    activations(k, "k", 3)
    Hkv = k.shape[1]
    check(q, "q", (B, H, d), q.dtype, q)
    check(k, "k", (B, Hkv, d), q.dtype, q)
    check(v, "v", (B, Hkv, d), q.dtype, q)
    check(pos, "pos", (B,), torch.int32, q)
    _cache(k_cache, v_cache, window, n_sink, B, Hkv, d, q)
    a.B, a.H, a.Hkv, a.d, a.window, a.n_sink = B, H, Hkv, d, window, n_sink
    a.scale = 0.0 if scale is None else _positive(scale)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    check(out, "out", q.shape, q.dtype, q)
    with launch(q, stream) as s:
        ws = scratch(dr.dr_window_attn_step_workspace_bytes(a), q, workspace)
        dr.check(dr.dr_window_attn_step(a, q, k, v, k_cache, v_cache, pos, out, ws, size_of(ws), s),
                 "dr_window_attn_step")
    return out
