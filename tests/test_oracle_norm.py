"""Pins of the norm's oracle: torch's fp64 autograd, differences, and the closed form of a constant row."""

import numpy as np
import pytest
import torch

from oracle import mxfp8 as mx
from oracle import norm


def test_against_autograd_and_differences():
    g = np.random.default_rng(0)
    r, w, dy, ds = g.standard_normal((5, 32)), g.standard_normal(32), g.standard_normal((5, 32)), g.standard_normal((5, 32))
    t = torch.tensor(r).requires_grad_()
    tw = torch.tensor(w).requires_grad_()
    y = torch.nn.functional.rms_norm(t, (32,), tw, 1e-3)
    assert np.allclose(norm.forward(r, w, 1e-3)[0], y.detach().numpy(), rtol=1e-12)
    dr, dw = torch.autograd.grad(y, (t, tw), torch.tensor(dy))
    got = norm.backward(dy, r, ds, w, 1e-3, False)
    assert np.allclose(got["dres"][0], dr.numpy() + ds, rtol=1e-11) and np.allclose(got["dw"][0], dw.numpy(), rtol=1e-11)
    assert got["dx"][0] is got["dres"][0]
    v, h = g.standard_normal((5, 32)), 1e-6
    f = lambda a: (norm.forward(a, w, 1e-3)[0] * dy).sum()  # noqa: E731
    assert abs((f(r + h * v) - f(r - h * v)) / (2 * h) - (dr.numpy() * v).sum()) < 1e-7


def test_a_constant_row():
    y, _ = norm.forward(np.full((1, 64), -3.0), np.ones(64), 0.0)
    assert np.allclose(y, -1.0, rtol=1e-15)
    assert (norm.forward(np.zeros((2, 64)), np.ones(64), 1e-6)[0] == 0).all()


@pytest.mark.parametrize("f32", [False, True])
def test_the_sum_is_rounded_once(f32):
    """In fp32 and then to bf16: 1 + 2^-8 lies half way between two bf16, and goes to the even one."""
    x, res = np.array([[1.0]]), np.array([[2.0 ** -8]])
    assert norm.stream_sum(x, res, f32)[0, 0] == (1 + 2.0 ** -8 if f32 else 1.0)
    assert norm.stream_sum(x, None, f32)[0, 0] == 1.0 and norm.stream_sum(None, res, f32)[0, 0] == 2.0 ** -8
    assert mx.bf16_to_f64(mx.f64_to_bf16(np.array([1 + 3 * 2.0 ** -8])))[0] == 1 + 2.0 ** -6
