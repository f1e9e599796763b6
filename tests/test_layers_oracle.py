"""The layers' fp64 oracles: every gradient against the central difference of the forward
oracle, and the forward against forms written another way."""

import numpy as np
import pytest

from oracle import layers as L

H = 1e-6      # central difference: error ~ H^2 f''' + 1e-16 |f| / H, about 1e-9 at these sizes
TOL = 1e-6


def difference(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + H
        hi = f()
        x[i] = old - H
        lo = f()
        x[i] = old
        g[i] = (hi - lo) / (2 * H)
    return g


def close(a, b):
    assert np.abs(a - b).max(initial=0.0) <= TOL * max(1.0, np.abs(b).max(initial=0.0))


@pytest.mark.parametrize("window,n_sink,q_start,lens", [(3, 0, 0, None), (2, 1, 0, [6, 2]), (4, 2, 3, [0, 7]),
                                                        (100, 0, 1, None)])
def test_attention_gradients(window, n_sink, q_start, lens):
    r = np.random.default_rng(window)
    B, T, Hq, Hk, d = 2, 4, 2, 1, 3
    S = T + q_start
    q, k, v = r.normal(size=(B, T, Hq, d)), r.normal(size=(B, S, Hk, d)), r.normal(size=(B, S, Hk, d))
    do = r.normal(size=q.shape)
    f = lambda: (L.window_attention(q, k, v, window, n_sink, q_start, lens)[0] * do).sum()  # noqa: E731
    g = L.window_attention(q, k, v, window, n_sink, q_start, lens, d_out=do)[3]
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        close(g[name], difference(f, t))


def test_attention_rows_that_see_nothing_and_full_causal():
    r = np.random.default_rng(0)
    q, k, v = (r.normal(size=(1, 5, 1, 4)) for _ in range(3))
    out, lse, _ = L.window_attention(q, k, v, 2, 0, 0, [1])
    assert (out[0, 2:] == 0).all() and np.isneginf(lse[0, 0, 2:]).all() and np.isfinite(lse[0, 0, :2]).all()
    out, _, _ = L.window_attention(q, k, v, 10**6)
    x = np.tril(np.exp(q[0, :, 0] @ k[0, :, 0].T / 2))
    close(out[0, :, 0], x / x.sum(1, keepdims=True) @ v[0, :, 0])
    ok = L.visible(12, 12, 3, 2)
    assert [list(np.flatnonzero(row)) for row in ok[[0, 4, 11]]] == [[0], [0, 1, 2, 3, 4], [0, 1, 9, 10, 11]]


@pytest.mark.parametrize("K,silu,lens,init", [(2, True, None, False), (4, True, [5, 2], True), (3, False, [0, 5], True)])
def test_conv_gradients(K, silu, lens, init):
    r = np.random.default_rng(K)
    x, w, bias = r.normal(size=(2, 5, 3)), r.normal(size=(3, K)), r.normal(size=3)
    s0 = r.normal(size=(2, K - 1, 3)) if init else None
    dy, de = r.normal(size=x.shape), r.normal(size=(2, K - 1, 3))

    def f():
        y, e = L.short_conv(x, w, bias, silu, s0, lens)
        return (y * dy).sum() + (e * de).sum()

    g = L.short_conv_bwd(x, w, bias, dy, silu, s0, de, lens)
    for name, t in (("dx", x), ("dweight", w), ("dbias", bias), ("dinit_state", s0)):
        if t is not None:
            close(g[name], difference(f, t))


@pytest.mark.parametrize("G,gated,softplus,lens,init", [(1, True, True, None, False), (2, False, True, [4, 1], True),
                                                        (2, True, False, [0, 4], True)])
def test_scan_gradients(G, gated, softplus, lens, init):
    r = np.random.default_rng(G + gated)
    Bn, T, Dm, N = 2, 4, 4, 2
    x, dt = r.normal(size=(Bn, T, Dm)), r.normal(size=(Bn, T, Dm))
    if not softplus:
        dt = np.abs(dt)
    A, B, C = -np.exp(r.normal(size=(Dm, N))), r.normal(size=(Bn, T, G, N)), r.normal(size=(Bn, T, G, N))
    D, bias = r.normal(size=Dm), r.normal(size=Dm) * 0.1
    z = r.normal(size=x.shape) if gated else None
    h0 = r.normal(size=(Bn, Dm, N)) if init else None
    dy, de = r.normal(size=x.shape), r.normal(size=(Bn, Dm, N))

    def f():
        y, e = L.selective_scan(x, dt, A, B, C, D, z, bias, softplus, h0, lens)
        return (y * dy).sum() + (e * de).sum()

    g = L.selective_scan_bwd(x, dt, A, B, C, dy, D, z, bias, softplus, h0, de, lens)
    for name, t in (("dx", x), ("ddt", dt), ("dz", z), ("dA", A), ("dB", B), ("dC", C), ("dD", D),
                    ("ddt_bias", bias), ("dinit_state", h0)):
        if t is not None:
            close(g[name], difference(f, t))


def test_scan_with_one_decay_is_a_weighted_sum():
    """A constant time step and rate: h_T = sum_t a^(T-t) dt B_t x_t."""
    r = np.random.default_rng(5)
    x, B, C = r.normal(size=(1, 6, 1)), r.normal(size=(1, 6, 1, 1)), np.ones((1, 6, 1, 1))
    y, h = L.selective_scan(x, np.full((1, 6, 1), 0.5), np.array([[-0.7]]), B, C, softplus=False)
    w = np.exp(-0.35) ** np.arange(5, -1, -1)
    close(h[0, 0, 0], (w * 0.5 * B[0, :, 0, 0] * x[0, :, 0]).sum())
    close(y[0, -1, 0], h[0, 0, 0])
