"""Pins of the cross entropy's oracle: torch's fp64 function and its autograd, and differences."""

import numpy as np
import torch

from oracle import xent


def test_against_torch():
    g = np.random.default_rng(0)
    x, w = g.standard_normal((6, 8)), g.standard_normal((11, 8))
    t = np.array([3, 0, -100, 10, 5, 11])
    rw = g.random(6)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    z = tx @ tw.t()
    lab = torch.tensor(np.where((t >= 0) & (t < 11), t, -100))
    loss = torch.nn.functional.cross_entropy(z, lab, reduction="none", ignore_index=-100)
    (loss * torch.tensor(rw)).sum().backward()
    got = xent.run(x, w, t, rw)
    n = lambda a: a.detach().numpy()  # noqa: E731
    assert np.allclose(got["loss"][0], n(loss), rtol=1e-12) and np.allclose(got["lse"][0], n(torch.logsumexp(z, 1)), rtol=1e-12)
    assert np.allclose(got["dx"][0], n(tx.grad), rtol=1e-11) and np.allclose(got["dw"][0], n(tw.grad), rtol=1e-11)
    assert all((b > 0).all() for _, b in got.values()) and (got["dx"][1] < 0.1).all() and (got["loss"][1] < 1e-4).all()


def test_differences_and_rows_left_out():
    g = np.random.default_rng(1)
    x, w, t = g.standard_normal((4, 8)), g.standard_normal((5, 8)), np.array([1, 4, -1, 0])
    got, h = xent.run(x, w, t), 1e-6
    for name, v in (("dx", g.standard_normal((4, 8))), ("dw", g.standard_normal((5, 8)))):
        f = lambda s: xent.run(x + s * v, w, t)["loss"][0].sum() if name == "dx" else xent.run(x, w + s * v, t)["loss"][0].sum()  # noqa: E731,B023
        assert abs((f(h) - f(-h)) / (2 * h) - (got[name][0] * v).sum()) < 1e-7
    x[2] = np.nan
    with_nan = xent.run(x, w, t)
    assert with_nan["loss"][0][2] == 0 and (with_nan["dx"][0][2] == 0).all()
    assert np.array_equal(with_nan["dw"][0], got["dw"][0]) and np.isfinite(with_nan["dw"][1]).all()


def test_the_bound_of_an_improbable_word_is_its_own():
    """Not the row's largest probability's: words 20 and 40 nats below one of their row, alone in their 64 or beside it."""
    x, w = np.ones((1, 1)), np.zeros((256, 1))
    w[1:64], w[64:128], w[128:192], w[192:] = -20.0, -40.0, -12.0, -43.0
    value, bound = (a[:, 0] for a in xent.run(x, w, [0])["dw"])
    assert np.allclose(value[1:], np.exp(w[1:, 0]) / np.exp(w).sum(), rtol=1e-12)
    # a rounding of dz and one of dw to bf16, half a step of the logarithm and fp32's
    assert (bound[1:] > 2.0 ** -7 * value[1:]).all() and (bound[1:] < (2.0 ** -7 + 2.0 ** -11) * 1.02 * value[1:]).all()
