"""fp64 numpy forms of what stands around a mixer, written from their formulas: the matrix
product with its epilogue, the norms before and after a block, and the gradients of each."""

from __future__ import annotations

import numpy as np


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def act(name, x):
    """(f(x), f'(x))."""
    if name == "relu":
        return np.maximum(x, 0.0), (x > 0).astype(float)
    if name == "sigmoid":
        s = _sigmoid(x)
        return s, s * _sigmoid(-x)
    if name == "silu":
        s = _sigmoid(x)
        return x * s, s + x * s * _sigmoid(-x)
    if name == "gelu_tanh":
        c = np.sqrt(2.0 / np.pi)
        t = np.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    return x, np.ones_like(x)


def linear(x, w, bias=None, residual=None, name="none", d_y=None):
    """x [M,K], w [K,N]: y, and with d_y also dict(dx, dweight, dbias, slope, d)."""
    pre = x @ w + (0.0 if bias is None else bias)
    y, slope = act(name, pre)
    y = y + (0.0 if residual is None else residual)
    if d_y is None:
        return y
    d = d_y * slope
    return y, dict(dx=d @ w.T, dweight=x.T @ d, dbias=d.sum(0), slope=slope, d=d)


def rstd(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def block_norm(h, branch=None, gate=None, gate_act="none", scale=None, post_norm=False, post_weight=None,
               pre_weight=None, eps=1e-6, d_h=None, d_y=None):
    """Rows [M,D]: (y, h'), and with d_h or d_y also the dict of gradients."""
    one = np.ones(h.shape[-1])
    w, pw, s = (one if t is None else t for t in (pre_weight, post_weight, scale))
    f, fs = (np.ones_like(h), np.zeros_like(h)) if gate is None else act(gate_act, gate)
    rb = rstd(branch, eps) if post_norm else 1.0
    v = np.zeros_like(h) if branch is None else branch * rb
    u = v * pw if post_norm else v
    hn = h + s * f * u
    r = rstd(hn, eps)
    n = hn * r
    if d_h is None and d_y is None:
        return n * w, hn
    dy = np.zeros_like(h) if d_y is None else d_y
    t = dy * w
    dh = (0.0 if d_h is None else d_h) + r * (t - n * (t * n).mean(-1, keepdims=True))
    du = dh * s * f
    q = du * pw
    g = dict(dh=dh, dpre_weight=(dy * n).sum(0), dscale=(dh * f * u).sum(0), dgate=dh * s * u * fs,
             dpost_weight=(du * v).sum(0),
             dbranch=rb * (q - v * (q * v).mean(-1, keepdims=True)) if post_norm else du)
    return n * w, hn, g
