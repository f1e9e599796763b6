"""The forward oracles of the short convolution and the selective scan against forms written
another way: a library convolution, and loops over single values."""

import math

import numpy as np
import pytest
import torch

from oracle import layers as L

TOL = 1e-12


def close(a, b):
    assert a.shape == b.shape and np.abs(a - b).max(initial=0.0) <= TOL * max(1.0, np.abs(b).max(initial=0.0))


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("silu,bias,init,lens", [(True, True, True, None), (False, True, True, [6, 1, 0]),
                                                 (True, False, False, [2, 6, 3])])
def test_conv_is_a_depthwise_cross_correlation(K, silu, bias, init, lens):
    r = np.random.default_rng(K)
    B, T, D = 3, 6, 5
    x, w = r.normal(size=(B, T, D)), r.normal(size=(D, K))
    b = r.normal(size=D) if bias else None
    s0 = r.normal(size=(B, K - 1, D)) if init else None
    y, end = L.short_conv(x, w, b, silu, s0, lens)
    before = np.zeros((B, K - 1, D)) if s0 is None else s0
    whole = torch.from_numpy(np.concatenate([before, x], 1)).transpose(1, 2)
    u = torch.nn.functional.conv1d(whole, torch.from_numpy(w)[:, None], None if b is None else torch.from_numpy(b),
                                   groups=D)
    want = (torch.nn.functional.silu(u) if silu else u).transpose(1, 2).numpy().copy()
    for i, n in enumerate([T] * B if lens is None else lens):
        want[i, n:] = 0.0
        history = np.concatenate([before[i], x[i, :n]])
        close(end[i], history[len(history) - (K - 1):])
    close(y, want)


@pytest.mark.parametrize("G", [1, 2, 4])
@pytest.mark.parametrize("gated,skip,bias,softplus,init,lens", [(True, True, True, True, True, [5, 3]),
                                                                (False, True, False, True, False, None),
                                                                (True, False, True, False, True, [0, 5])])
def test_scan_of_single_values(G, gated, skip, bias, softplus, init, lens):
    r = np.random.default_rng(G)
    Bn, T, Dm, N = 2, 5, 8, 3
    x, dt = r.normal(size=(Bn, T, Dm)), r.normal(size=(Bn, T, Dm))
    if not softplus:
        dt = np.abs(dt) + 1.0
    A = -np.exp(r.normal(size=(Dm, N)))
    B, C = r.normal(size=(Bn, T, G, N)), r.normal(size=(Bn, T, G, N))
    D, db = (r.normal(size=Dm) if skip else None), (r.normal(size=Dm) * 0.1 if bias else None)
    z = r.normal(size=x.shape) if gated else None
    h0 = r.normal(size=(Bn, Dm, N)) if init else None
    y, end = L.selective_scan(x, dt, A, B, C, D, z, db, softplus, h0, lens)
    for b in range(Bn):
        n_real = T if lens is None else lens[b]
        for c in range(Dm):
            g = c // (Dm // G)          # neighbouring channels share a group
            h = [0.0] * N if h0 is None else [float(h0[b, c, n]) for n in range(N)]
            for t in range(T):
                out = 0.0
                if t < n_real:
                    step = dt[b, t, c] + (db[c] if bias else 0.0)
                    if softplus:
                        step = math.log1p(math.exp(step))
                    for n in range(N):
                        h[n] = math.exp(step * A[c, n]) * h[n] + step * B[b, t, g, n] * x[b, t, c]
                        out += C[b, t, g, n] * h[n]
                    if skip:
                        out += D[c] * x[b, t, c]
                    if gated:           # the gate is behind the skip
                        out *= z[b, t, c] / (1.0 + math.exp(-z[b, t, c]))
                assert abs(y[b, t, c] - out) <= TOL * max(1.0, abs(out))
            close(end[b, c], np.array(h))
