"""Oracle: the SwiGLU backward and the router's backward from activations kept
in MXFP8.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Plain NumPy in fp64.

The kept codes stand for H' (``mxfp8.dequantize``); the backward is that of
``glue.swiglu`` at H'.  The router's gradient comes from dots[r] = sum_f dA[r, f]
A'[r, f] with dA = w W2^T dout: dots = w <dout, W2 A'> = w dw, so that
dlogits[t, e_j] = w_j (dw_j - sum_i w_i dw_i) = dots_j - w_j sum_i dots_i.
"""

import numpy as np

from . import glue, mxfp8

F32 = 2.0 ** -24


def dots(h_bits, da_bits, F):
    """(dots [R], their bound).  A term's sigmoid, silu and products are off by
    32 roundings, its sum by one for every term it passes."""
    a, _ = glue.swiglu(h_bits, F)
    t = a * mxfp8.bf16_to_f64(da_bits)
    return t.sum(1), np.abs(t).sum(1) * (F + 64) * F32 + 2.0 ** -126


def dlogits(dot, dst_row, expert_ids, weights, num_experts):
    """(dlogits [T, E], its bound) from dots [R]; rows outside count as zero, repeated experts add up."""
    ids = np.asarray(expert_ids, np.int64)
    T, k = ids.shape
    dst = np.asarray(dst_row, np.int64).reshape(T, k)
    ok = (dst >= 0) & (dst < len(dot))
    p = np.where(ok, np.asarray(dot, np.float64)[np.where(ok, dst, 0)], 0.0)
    w = np.asarray(weights, np.float64)
    g = p - w * p.sum(1, keepdims=True)
    e = (np.abs(p) + w * np.abs(p).sum(1, keepdims=True)) * (k + 8) * F32
    out, bound = np.zeros((2, T, num_experts))
    for j in range(k):
        np.add.at(out, (np.arange(T), ids[:, j]), g[:, j])
        np.add.at(bound, (np.arange(T), ids[:, j]), e[:, j])
    return out, bound * 1.01 + 2.0 ** -126
