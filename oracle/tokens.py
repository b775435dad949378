"""Oracle: the whole SwiGLU MoE layer for a few tokens, with the bound of what
a kernel with fp32 sums and one bf16 rounding of w silu(g) u may be off.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Plain NumPy in fp64.

* a token's experts are its k largest logits, equal logits to the lower id;
  a logit of -inf is never chosen, and a token with none left gets its
  residual (or zero);
* out[t] = residual[t] + sum_j W2_e (w[t,j] silu(g) * u), [g; u] = W1_e x[t].
"""

import numpy as np

from . import glue

F32 = 2.0 ** -24     # one fp32 rounding
BF16 = 2.0 ** -8     # one bf16 rounding


def choose(logits, topk):
    """Per token: (expert ids, weights) without the -inf ones."""
    lg = np.asarray(logits, np.float32).astype(np.float64)
    out = []
    for row in lg:
        ids = sorted(range(len(row)), key=lambda e: (-row[e], e))[:topk]
        ids = [e for e in ids if row[e] != -np.inf]
        z = np.array([row[e] for e in ids])
        w = np.exp(z - z.max()) if ids else z
        out.append((ids, w / w.sum() if ids else w))
    return out


def layer(x, logits, w1, w2, topk, residual=None):
    """(out fp64 [T, H], bound fp64 [T, H]) from the values of x [T, H],
    w1 [E, 2F, H], w2 [E, H, F] and residual [T, H].

    The bound counts: every fp32 sum of n products as n + 16 roundings of its
    magnitude sum; silu and its product 32 roundings (exp, sum, division and
    the products, each within a few units) with silu's slope at most 1.1; the
    softmax weight 64 roundings; one bf16 rounding of w silu(g) u; one of the
    result."""
    T, H = x.shape
    F = w2.shape[2]
    out = np.zeros((T, H)) if residual is None else residual.astype(np.float64).copy()
    mag = np.abs(out)
    err = np.zeros((T, H))
    for t, (ids, w) in enumerate(choose(logits, topk)):
        for e, wt in zip(ids, w):
            h = w1[e] @ x[t]
            dh = (H + 16) * F32 * (np.abs(w1[e]) @ np.abs(x[t]))
            g, u, dg, du = h[:F], h[F:], dh[:F], dh[F:]
            a = wt * glue.silu(g) * u
            da = wt * (1.1 * dg * (np.abs(u) + du) + np.abs(glue.silu(g)) * du)
            da = (da + np.abs(a) * 96 * F32) * (1 + BF16) + np.abs(a) * BF16
            out[t] += w2[e] @ a
            m = np.abs(w2[e]) @ (np.abs(a) + da)
            mag[t] += m
            err[t] += np.abs(w2[e]) @ da + (F + 16) * F32 * m
    return out, err + 80 * F32 * mag + np.abs(out) * BF16 + 2.0 ** -126
