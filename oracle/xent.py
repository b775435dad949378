"""Oracle: softmax cross entropy of a product's rows, with its gradient, with
bounds of what fp32 sums and the documented roundings may be off.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Plain NumPy in fp64.
"""

import numpy as np

F32 = 2.0 ** -24
LOG = np.log(2.0) * 2.0 ** -11 * 1.001
BF16 = 2.0 ** -8
TINY = 2.0 ** -126


def run(x, w, targets, row_weight=None):
    """{"loss", "lse", "dx", "dw"}: (value, bound) for x [M, K], w [V, K], targets [M] (outside [0, V): left out).

    Bounds: a logit is an fp32 sum of K products, off by K + 16 roundings of
    their magnitudes; an exponential of a difference d by |d| + 16 roundings,
    which against e^d is 17 at most, and a sum of positive terms by a few more:
    128 roundings of the logarithm's argument in all.  For dz, log2 of exp(z - m)
    is kept in steps of 2^-10, half a step of which is a factor of 2^(2^-11), down
    to 2^-63.9 of the strip's largest, 32 or 64 words that lie in one aligned group
    of 64, and zero below; dz is then rounded to bf16, and summed in fp32.  What is
    below fp32's normal range may be lost on the way."""
    M, V = len(x), len(w)
    t = np.asarray(targets, np.int64)
    live = (t >= 0) & (t < V)
    at = np.where(live, t, 0)
    g = np.where(live, 1.0 if row_weight is None else np.asarray(row_weight, np.float64), 0.0)[:, None]
    rows = np.arange(M)
    # rows that are left out may hold anything; their lse is not looked at where it is not finite
    with np.errstate(invalid="ignore", over="ignore"):
        z, ez = x @ w.T, (x.shape[1] + 16) * F32 * (np.abs(x) @ np.abs(w).T)
        top = z.max(1, keepdims=True)
        p = np.exp(z - top)
        lse = top + np.log(p.sum(1, keepdims=True))
        p = np.exp(z - lse)
        elz = (p * ez).sum(1, keepdims=True) + 128 * F32 + 4 * F32 * (np.abs(lse) + np.abs(top))
        loss = np.where(live, lse[:, 0] - z[rows, at], 0.0)
        eloss = np.where(live, elz[:, 0] + ez[rows, at] + F32 * np.abs(loss), 0.0)
    out = {"loss": (loss, eloss * 1.01 + TINY), "lse": (lse[:, 0], elz[:, 0] * 1.01 + TINY)}
    xl = np.where(live[:, None], x, 0.0)
    p, ep = (np.where(live[:, None], a, 0.0) for a in (p, ez + elz))
    groups = np.pad(p, ((0, 0), (0, -V % 64))).reshape(M, -1, 64).max(2)
    e = np.abs(g) * (p * (ep + LOG + 64 * F32 * (1 + np.abs(np.where(live[:, None], z - lse, 0.0)))) +
                     groups.repeat(64, 1)[:, :V] * 2.0 ** -63.9) + (1 + np.abs(g)) * TINY
    dz = p
    dz[rows[live], t[live]] -= 1.0
    dz = dz * g
    e = e + BF16 * (np.abs(dz) + e)
    e[rows, at] += 4 * F32 * np.abs(g[:, 0])     # the target's 1 is subtracted in fp32
    for name, a, b, n in (("dx", dz, w, V), ("dw", dz.T, xl, M)):
        v, mag = a @ b, np.abs(a) @ np.abs(b)
        err = (e if name == "dx" else e.T) @ np.abs(b) + (n + 16) * F32 * mag
        out[name] = v, (err + np.abs(v) * BF16) * 1.01 + TINY
    return out
