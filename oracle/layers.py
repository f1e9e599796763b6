"""fp64 numpy forms of the layers next to the recurrence, written from their formulas:
window attention with sinks, short causal convolution, selective scan, and the gradients
of each.  ``lens`` [B] are the sequences' real lengths (None: all full)."""

from __future__ import annotations

import numpy as np


def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


# ------------------------------------------------------------------ window attention

def visible(T, S, window, n_sink, q_start=0, length=None):
    """[T, S] truth values: does the query at position q_start + i see key j?"""
    p = q_start + np.arange(T)[:, None]
    j = np.arange(S)[None]
    return (j <= p) & (j < (S if length is None else length)) & ((p - j < window) | (j < n_sink))


def window_attention(q, k, v, window, n_sink=0, q_start=0, lens=None, scale=None, d_out=None):
    """q [B,T,H,d], k, v [B,S,Hkv,d].  Returns (out, lse [B,H,T], size of out's terms); with
    d_out also a dict of dq, dk, dv and of the sizes of their terms (sums of absolute
    values, for error bounds)."""
    B, T, H, d = q.shape
    S, G = k.shape[1], H // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, size = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((B, H, T), -np.inf)
    g = {n: np.zeros_like(t) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    s_ = {n: np.zeros_like(t) for n, t in g.items()}
    for b in range(B):
        ok = visible(T, S, window, n_sink, q_start, None if lens is None else lens[b])
        some = ok.any(1)
        for h in range(H):
            kh, vh = (np.where(ok.any(0)[:, None], t[b, :, h // G], 0.0) for t in (k, v))
            x = np.where(ok, scale * q[b, :, h] @ kh.T, -np.inf)
            m = np.where(some, x.max(1, initial=-np.inf), 0.0)
            e = np.exp(x - m[:, None])
            with np.errstate(divide="ignore"):
                lse[b, h] = m + np.log(e.sum(1))
            p = e / np.where(some, e.sum(1), 1.0)[:, None]
            out[b, :, h], size[b, :, h] = p @ vh, p @ np.abs(vh)
            if d_out is None:
                continue
            do = d_out[b, :, h]
            ds = p * (do @ vh.T - (do * out[b, :, h]).sum(1, keepdims=True))
            # an error of out, relative to its size, moves a whole row of ds
            dsz = np.abs(ds) + p * (np.abs(do) * size[b, :, h]).sum(1, keepdims=True)
            for n, i, val, sz in (("dq", h, scale * ds @ kh, scale * dsz @ np.abs(kh)),
                                  ("dk", h // G, scale * ds.T @ q[b, :, h], scale * dsz.T @ np.abs(q[b, :, h])),
                                  ("dv", h // G, p.T @ do, p.T @ np.abs(do))):
                g[n][b, :, i] += val
                s_[n][b, :, i] += sz
    return (out, lse, size) if d_out is None else (out, lse, size, g, s_)


# ------------------------------------------------------------------ short convolution

def short_conv(x, w, bias=None, silu=True, s0=None, lens=None):
    """x [B,T,D], w [D,K].  Returns (y, final state [B,K-1,D])."""
    B, T, D = x.shape
    K = w.shape[1]
    ext = np.concatenate([np.zeros((B, K - 1, D)) if s0 is None else s0, x], 1)
    y, end = np.zeros_like(x), np.zeros((B, K - 1, D))
    for b in range(B):
        n = T if lens is None else lens[b]
        for t in range(n):
            u = (ext[b, t:t + K].T * w).sum(1) + (0 if bias is None else bias)
            y[b, t] = u * _sigmoid(u) if silu else u
        end[b] = ext[b, n:n + K - 1]
    return y, end


def short_conv_bwd(x, w, bias, d_y, silu=True, s0=None, d_end=None, lens=None):
    B, T, D = x.shape
    K = w.shape[1]
    ext = np.concatenate([np.zeros((B, K - 1, D)) if s0 is None else s0, x], 1)
    d_ext, dw, db = np.zeros_like(ext), np.zeros_like(w), np.zeros(D)
    for b in range(B):
        n = T if lens is None else lens[b]
        for t in range(n):
            du = d_y[b, t]
            if silu:
                u = (ext[b, t:t + K].T * w).sum(1) + (0 if bias is None else bias)
                s = _sigmoid(u)
                du = du * (s + u * s * (1 - s))
            d_ext[b, t:t + K] += (du[:, None] * w).T
            dw += du[:, None] * ext[b, t:t + K].T
            db += du
        if d_end is not None:
            d_ext[b, n:n + K - 1] += d_end[b]
    return dict(dx=d_ext[:, K - 1:], dweight=dw, dbias=db, dinit_state=d_ext[:, :K - 1])


# ------------------------------------------------------------------ selective scan

def _steps(dt, bias, softplus):
    raw = dt + (0 if bias is None else bias)
    return raw, np.logaddexp(0.0, raw) if softplus else raw


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, h0=None, lens=None):
    """x, dt, z [Bn,T,Dm], A [Dm,N], B, C [Bn,T,G,N].  Returns (y, final state [Bn,Dm,N])."""
    Bn, T, Dm = x.shape
    of = np.arange(Dm) // (Dm // B.shape[2])
    _, step = _steps(dt, dt_bias, softplus)
    y = np.zeros_like(x)
    h = np.zeros((Bn, *A.shape)) if h0 is None else h0.copy()
    for b in range(Bn):
        for t in range(T if lens is None else lens[b]):
            h[b] = np.exp(step[b, t][:, None] * A) * h[b] + (step[b, t] * x[b, t])[:, None] * B[b, t][of]
            y[b, t] = (h[b] * C[b, t][of]).sum(1) + (0 if D is None else D * x[b, t])
            if z is not None:
                y[b, t] *= z[b, t] * _sigmoid(z[b, t])
    return y, h


def selective_scan_bwd(x, dt, A, B, C, d_y, D=None, z=None, dt_bias=None, softplus=True, h0=None,
                       d_end=None, lens=None):
    Bn, T, Dm = x.shape
    G = B.shape[2]
    of = np.arange(Dm) // (Dm // G)
    raw, step = _steps(dt, dt_bias, softplus)
    r = {n: np.zeros_like(t) for n, t in (("dx", x), ("ddt", x), ("dz", x), ("dA", A), ("dB", B), ("dC", C))}
    dD, dh0 = np.zeros(Dm), np.zeros((Bn, *A.shape))

    def per_group(v):                       # [Dm, N] -> [G, N]
        return v.reshape(G, Dm // G, -1).sum(1)

    for b in range(Bn):
        n = T if lens is None else lens[b]
        hs = [np.zeros_like(A) if h0 is None else h0[b]]
        for t in range(n):
            hs.append(np.exp(step[b, t][:, None] * A) * hs[-1] + (step[b, t] * x[b, t])[:, None] * B[b, t][of])
        g = np.zeros_like(A) if d_end is None else d_end[b].copy()
        for t in reversed(range(n)):
            dy = d_y[b, t]
            if z is not None:
                s = _sigmoid(z[b, t])
                y = (hs[t + 1] * C[b, t][of]).sum(1) + (0 if D is None else D * x[b, t])
                r["dz"][b, t] = dy * y * (s + z[b, t] * s * (1 - s))
                dy = dy * z[b, t] * s
            a = np.exp(step[b, t][:, None] * A)
            r["dC"][b, t] = per_group(dy[:, None] * hs[t + 1])
            g = g + dy[:, None] * C[b, t][of]
            r["dB"][b, t] = per_group(g * (step[b, t] * x[b, t])[:, None])
            gb = (g * B[b, t][of]).sum(1)
            g = g * a
            r["dx"][b, t] = gb * step[b, t] + (0 if D is None else D * dy)
            d_step = (g * hs[t] * A).sum(1) + gb * x[b, t]
            r["ddt"][b, t] = d_step * (_sigmoid(raw[b, t]) if softplus else 1.0)
            r["dA"] += g * hs[t] * step[b, t][:, None]
            dD += dy * x[b, t]
        dh0[b] = g
    return r | dict(dD=dD, ddt_bias=r["ddt"].sum((0, 1)), dinit_state=dh0)
