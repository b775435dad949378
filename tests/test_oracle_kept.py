"""Pins of the kept activations' oracle: the dots give the router oracle's gradient and autograd's."""

import numpy as np
import torch

from oracle import glue, kept, router
from oracle import mxfp8 as mx

import workloads


def test_dots_are_the_routers_gradient():
    """With y = W2 A and dA = w W2^T dout, sum_f dA A = w <dout, y>."""
    g = np.random.default_rng(1)
    T, k, E, F, H = 6, 3, 8, 32, 64
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    w = g.random((T, k))
    w /= w.sum(1, keepdims=True)
    a, w2, dout = g.standard_normal((T * k, F)), g.standard_normal((H, F)), g.standard_normal((T, H))
    y = a @ w2.T
    da = w.reshape(-1, 1) * (np.repeat(dout, k, 0) @ w2)
    dst = g.permutation(T * k)
    dot = np.zeros(T * k)
    dot[dst] = (da * a).sum(1)
    got, bound = kept.dlogits(dot, dst, ids, w, E)
    t = torch.tensor(g.standard_normal((T, E)))
    logits = torch.where(torch.zeros(T, E, dtype=torch.bool).scatter_(1, torch.tensor(ids), True), t, -torch.inf)
    logits.scatter_(1, torch.tensor(ids), torch.log(torch.tensor(w)))
    logits.requires_grad_()
    p = torch.softmax(logits, 1).gather(1, torch.tensor(ids))
    (p * torch.tensor((np.repeat(dout, k, 0) * y).sum(1).reshape(T, k))).sum().backward()
    assert np.allclose(got, logits.grad.numpy(), rtol=1e-10, atol=1e-10) and (bound > 0).all()
    # the router's oracle on values that bf16 holds
    db, yb = mx.f64_to_bf16(dout), mx.f64_to_bf16(y)
    rows = np.zeros((T * k, H), np.uint16)
    rows[dst] = yb
    dw, _, dl, _ = router.router_bwd(db, rows, dst, ids, w.astype(np.float32), E)
    dot[dst] = (w.astype(np.float32).astype(np.float64) * dw).ravel()
    assert np.allclose(kept.dlogits(dot, dst, ids, w.astype(np.float32), E)[0], dl, rtol=1e-10, atol=1e-12)


def test_rows_outside_and_repeated_experts():
    out, _ = kept.dlogits(np.array([2.0, 3.0]), np.array([0, 5, -1, 1]), np.array([[1, 2], [0, 0]]),
                          np.array([[0.5, 0.5], [0.25, 0.75]]), 3)
    assert np.allclose(out, [[0, 1, -1], [0, 0, 0]])


def test_dots_against_the_glue():
    g = np.random.default_rng(2)
    h, da = workloads.normal_bf16(g, (3, 64), 1.0), workloads.normal_bf16(g, (3, 32), 1.0)
    d, bound = kept.dots(h, da, 32)
    a, _ = glue.swiglu(h, 32)
    assert np.allclose(d, np.einsum("rf,rf->r", a, mx.bf16_to_f64(da)), rtol=1e-12) and (bound < 1e-4 * np.abs(a).sum(1) * 4).all()
