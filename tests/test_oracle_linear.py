"""Pins of the dense product's oracle: torch's functions in fp64, its autograd, and differences."""

import numpy as np
import pytest
import torch

from oracle import linear


def torch_act(z, name):
    F = torch.nn.functional
    return {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name](z)


@pytest.mark.parametrize("name", linear.ACTS)
def test_against_torch(name):
    g = np.random.default_rng(0)
    x, w, b, r = (torch.tensor(g.standard_normal(s)) for s in ((7, 5), (4, 5), (4,), (7, 4)))
    for t in (x, w, b):
        t.requires_grad_()
    z = x @ w.t() + b
    z.retain_grad()
    out = torch_act(z, name) + r
    dout = torch.tensor(g.standard_normal((7, 4)))
    out.backward(dout)
    n = lambda t: t.detach().numpy()  # noqa: E731
    y, bound, zz, zb = linear.forward(n(x), n(w), n(b), n(r), name, False)
    assert np.allclose(y, n(out), rtol=1e-12) and np.allclose(zz, n(z), rtol=1e-12)
    assert (bound > np.abs(y) * 2.0 ** -9).all() and (bound < 0.02 + 0.02 * np.abs(y)).all() and (zb > 0).all()
    got = linear.backward(n(dout), n(z), n(x), n(w), None, name)
    for k, t in (("dx", x), ("dw", w), ("db", b)):
        assert np.allclose(got[k][0], n(t.grad), rtol=1e-10, atol=1e-12), k
    added = linear.backward(n(dout), n(z), n(x), n(w), np.ones((7, 5)), name)["dx"][0]
    assert np.allclose(added, n(x.grad) + 1)


@pytest.mark.parametrize("name", linear.ACTS)
def test_slope_against_differences(name):
    z = np.linspace(-6, 6, 97) + 0.013
    h = 1e-5
    d = (linear.act(z + h, name) - linear.act(z - h, name)) / (2 * h)
    assert np.allclose(d, linear.slope(z, name), atol=1e-8)
