"""The fp64 forms of the matrix product with its epilogue and of the norms around a block,
against forms written another way and against differences."""

import numpy as np
import pytest

from oracle import block as O

ACTS = ["none", "relu", "silu", "gelu_tanh", "sigmoid"]


def differences(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        for s in (1, -1):
            y = x.copy()
            y[i] += s * eps
            g[i] += s * f(y) / (2 * eps)
    return g


@pytest.mark.parametrize("name", ACTS)
def test_activations(name):
    torch = pytest.importorskip("torch")
    F = torch.nn.functional
    x = np.concatenate([np.linspace(-40, 40, 801) + 0.013, [-1e30, -700.0, 700.0]])
    t = torch.from_numpy(x).requires_grad_()
    f = {"none": lambda v: v * 1, "relu": torch.relu, "silu": F.silu, "sigmoid": torch.sigmoid,
         "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name]
    got, slope = O.act(name, x[:-3] if name == "gelu_tanh" else x)
    want = f(t)
    d, = torch.autograd.grad(want.sum(), t)
    n = len(got)
    np.testing.assert_allclose(got, want.detach().numpy()[:n], rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(slope, d.numpy()[:n], rtol=1e-9, atol=1e-13)


@pytest.mark.parametrize("name", ACTS)
def test_linear_gradients_against_differences(name):
    g = np.random.default_rng(3)
    x, w, b, r, dy = (g.standard_normal(s) for s in ((3, 4), (4, 5), (5,), (3, 5), (3, 5)))
    y, grads = O.linear(x, w, b, r, name, dy)
    direct = np.array([[sum(x[i, k] * w[k, j] for k in range(4)) + b[j] for j in range(5)] for i in range(3)])
    np.testing.assert_allclose(y, O.act(name, direct)[0] + r, atol=1e-12)
    for got, f, at in (("dx", lambda v: O.linear(v, w, b, r, name), x),
                       ("dweight", lambda v: O.linear(x, v, b, r, name), w),
                       ("dbias", lambda v: O.linear(x, w, v, r, name), b)):
        np.testing.assert_allclose(grads[got], differences(lambda v: (f(v) * dy).sum(), at), atol=1e-7)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, *ACTS])
def test_block_norm_gradients_against_differences(gate, post):
    g = np.random.default_rng(5)
    M, D = 2, 6
    t = {k: g.standard_normal((M, D)) for k in ("h", "branch", "gate", "d_h", "d_y")}
    v = {k: g.standard_normal(D) for k in ("scale", "post_weight", "pre_weight")}
    kw = dict(gate_act=gate or "none", post_norm=post, eps=1e-3)
    args = dict(h=t["h"], branch=t["branch"], **v)
    if gate:
        args["gate"] = t["gate"]
    if not post:
        del args["post_weight"]
    y, hn, grads = O.block_norm(**args, **kw, d_h=t["d_h"], d_y=t["d_y"])
    for i in range(M):   # by the row
        u = t["branch"][i]
        if post:
            u = u / np.sqrt(np.sum(u ** 2) / D + 1e-3) * v["post_weight"]
        if gate:
            u = u * O.act(gate, t["gate"][i])[0]
        row = t["h"][i] + v["scale"] * u
        np.testing.assert_allclose(hn[i], row, atol=1e-12)
        np.testing.assert_allclose(y[i], row / np.sqrt(np.sum(row ** 2) / D + 1e-3) * v["pre_weight"], atol=1e-12)
    for name, at in args.items():
        def loss(x):
            y, hn = O.block_norm(**{**args, name: x}, **kw)
            return (y * t["d_y"]).sum() + (hn * t["d_h"]).sum()
        np.testing.assert_allclose(grads["d" + name], differences(loss, at), atol=2e-7, err_msg=name)
