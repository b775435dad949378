"""Oracle: the dense product with bias, activation and residual, and its
backward, with bounds of what fp32 sums and the documented roundings may be off.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Plain NumPy in fp64.
"""

import math

import numpy as np

F32 = 2.0 ** -24
BF16 = 2.0 ** -8
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0)
    if name == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + np.exp(-z)) if name == "silu" else z


def slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def forward(x, w, bias, residual, name, f32):
    """(out, its bound, z, its bound).  An fp32 sum of K products and the bias
    is off by K + 16 roundings of its magnitude sum at most; the activations'
    slopes are at most 1.13 and their own arithmetic 32 roundings of |z|."""
    z = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, mag = z + bias, mag + np.abs(bias)
    dz = (x.shape[1] + 16) * F32 * mag
    y, dy = act(z, name), dz if name == "none" else 1.13 * dz + 32 * F32 * np.abs(z)
    if residual is not None:
        y, dy = y + residual, dy + F32 * (np.abs(y) + np.abs(residual))
    return y, (dy + np.abs(y) * (F32 if f32 else BF16)) * 1.01 + 2.0 ** -126, z, (dz + np.abs(z) * BF16) * 1.01 + 2.0 ** -126


def backward(dout, z, x, w, add, name):
    """{"dx", "dw", "db"}: (value, bound).  The slope is off by 96 fp32
    roundings (of terms of at most about 1) and dz is rounded to bf16 once for
    the products; sums as in the forward."""
    dz = dout * slope(z, name) if name != "none" else dout
    e32 = np.abs(dout) * 96 * F32 if name != "none" else np.zeros_like(dout)
    e = e32 + np.abs(dz) * BF16
    out = {}
    dx, mag = dz @ w, np.abs(dz) @ np.abs(w)
    err = e @ np.abs(w) + (w.shape[0] + 16) * F32 * mag
    if add is not None:
        dx, err = dx + add, err + F32 * (mag + np.abs(add))
    out["dx"] = dx, (err + np.abs(dx) * BF16) * 1.01 + 2.0 ** -126
    dw, mag = dz.T @ x, np.abs(dz).T @ np.abs(x)
    out["dw"] = dw, (e.T @ np.abs(x) + (x.shape[0] + 16) * F32 * mag + np.abs(dw) * BF16) * 1.01 + 2.0 ** -126
    out["db"] = dz.sum(0), (e32.sum(0) + (x.shape[0] + 16) * F32 * np.abs(dz).sum(0)) * 1.01 + 2.0 ** -126
    return out
