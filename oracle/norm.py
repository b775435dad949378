"""Oracle: the root-mean-square norm with the residual's addition and its
backward, with bounds of what fp32 arithmetic and the documented roundings may
be off.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Plain NumPy in fp64.
"""

import numpy as np

from . import mxfp8

F32 = 2.0 ** -24
BF16 = 2.0 ** -8
TINY = 2.0 ** -126


def stream_sum(x, residual, f32):
    """r in fp64, exactly: the fp32 sum of two values, rounded to bf16 where the stream is bf16."""
    if residual is None:
        return np.asarray(x, np.float64)
    r = np.asarray(residual, np.float32)
    if x is not None:
        r = np.asarray(x, np.float32) + r
    return r.astype(np.float64) if f32 else mxfp8.bf16_to_f64(mxfp8.f64_to_bf16(r.astype(np.float64)))


def _inv(r, eps):
    return 1.0 / np.sqrt((r * r).mean(1, keepdims=True) + eps)


def forward(r, weight, eps):
    """(y, its bound).  A sum of squares is off by 48 roundings at most: a
    thread adds up to 8 chunks, each a tree of 3, 6 steps of a wave, 16 waves,
    the mean and eps, and a square root halves that; the reciprocal root and
    the products are a few more."""
    y = r * _inv(r, eps) * weight
    return y, np.abs(y) * (BF16 + 64 * F32) * 1.01 + TINY


def backward(dy, r, dsum, weight, eps, f32):
    """{"dres", "dx", "dw"}: (value, bound); dres in the stream's type, dx in bf16."""
    n, s = r.shape[1], _inv(r, eps)
    g = dy * weight
    m = s * s * (g * r).mean(1, keepdims=True)
    # the mean's terms cancel: its error is of their magnitudes
    em = s * s * 64 * F32 * np.abs(g * r).mean(1, keepdims=True) + 64 * F32 * np.abs(m)
    d = s * (g - m * r)
    e = s * (np.abs(r) * em + 4 * F32 * (np.abs(g) + np.abs(m * r))) + 64 * F32 * s * (np.abs(g) + np.abs(m * r))
    if dsum is not None:
        d, e = d + dsum, e + F32 * (np.abs(d) + np.abs(dsum))
    out = {"dres": (d, (e + np.abs(d) * (F32 if f32 else BF16)) * 1.01 + TINY),
           "dx": (d, (e + np.abs(d) * BF16) * 1.01 + TINY)}
    t = dy * r * s
    out["dw"] = t.sum(0), np.abs(t).sum(0) * (r.shape[0] + 128) * F32 * 1.01 + TINY
    assert n == dy.shape[1]
    return out
