"""GPU parity: the dense product with its epilogue, and its backward, against
the fp64 oracle (oracle/linear.py), whose bounds count the roundings."""

import math

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
import workloads
from mxfp8_block_scaled_07_amd import moe
from oracle import linear as ol
from oracle import mxfp8 as mx

from gpu_util import DEV, dev, host

pytestmark = pytest.mark.gpu

BF, F32 = mxa.MX_OUT_BF16, mxa.MX_OUT_F32
val = lambda a: mx.bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)  # noqa: E731


def within(got, want, bound, what):
    err = np.abs(val(got) - want)
    print(what, "max err/bound", float((err / bound).max()) if err.size else 0.0, flush=True)
    assert (err <= bound).all(), (what, np.argwhere(~(err <= bound))[:5])


def padded(shape, dtype):
    """A tensor with a guard row behind it."""
    t = torch.full((shape[0] + 1,) + tuple(shape[1:]), 77.0, dtype=dtype, device=DEV)
    return t


class Case:
    def __init__(self, M, N, K, act="none", bias=True, residual=True, keep_z=True, f32=False, seed=0):
        g = np.random.default_rng([seed, M, N, K])
        self.M, self.N, self.K, self.act, self.f32 = M, N, K, act, f32
        self.x = workloads.normal_bf16(g, (M, K), 1.0, 0.002)
        self.w = workloads.normal_bf16(g, (N, K), K ** -0.5)
        self.bias = g.standard_normal(N).astype(np.float32) if bias else None
        self.res = workloads.normal_bf16(g, (M, N), 1.0) if residual else None
        self.dout = workloads.normal_bf16(g, (M, N), 1.0) if not f32 else g.standard_normal((M, N)).astype(np.float32)
        self.zin = workloads.normal_bf16(g, (M, N), 2.0)
        self.add = workloads.normal_bf16(g, (M, K), 1.0) if residual else None
        self.keep_z = keep_z
        d = lambda a: None if a is None else dev(a)  # noqa: E731
        self.d = {k: d(getattr(self, k)) for k in ("x", "w", "bias", "res", "dout", "zin", "add")}

    def fwd(self, stream=None, out=None):
        M, N, K = self.M, self.N, self.K
        wsb = mxa.mx_bf16_linear_workspace_size(M, N, K)
        if not hasattr(self, "ws"):
            # all ones: NaN wherever the product would use what it has not written
            self.ws = torch.full((wsb + 64,), 0xFF, dtype=torch.uint8, device=DEV)
            self.out = padded((M, N), torch.float32 if self.f32 else torch.bfloat16)
            self.z = padded((M, N), torch.bfloat16) if self.keep_z else None
        mxa.mx_bf16_linear(self.d["x"], self.d["w"], self.d["bias"], self.d["res"], M, N, K, ol.ACTS.index(self.act),
                           self.z, self.out if out is None else out, F32 if self.f32 else BF, self.ws, wsb, stream)
        return wsb

    def bwd(self, stream=None):
        M, N, K, act = self.M, self.N, self.K, ol.ACTS.index(self.act)
        wsb = mxa.mx_bf16_linear_bwd_workspace_size(M, N, K, act)
        if not hasattr(self, "bws"):
            self.bws = torch.full((wsb + 64,), 0xFF, dtype=torch.uint8, device=DEV)
            self.dx, self.dw = padded((M, K), torch.bfloat16), padded((N, K), torch.bfloat16)
            self.db = torch.full((N + 1,), 77.0, device=DEV)
        mxa.mx_bf16_linear_bwd(self.d["dout"], F32 if self.f32 else BF, self.d["zin"] if act else None, self.d["x"],
                               self.d["w"], self.d["add"], M, N, K, act, self.dx, self.dw, self.db, self.bws, wsb, stream)
        return wsb

    def check_fwd(self):
        wsb = self.fwd()
        torch.cuda.synchronize()
        assert (self.out[self.M] == 77).all() and (self.ws[wsb:] == 0xFF).all()
        y, yb, z, zb = ol.forward(val(self.x), val(self.w), self.bias, None if self.res is None else val(self.res),
                                  self.act, self.f32)
        within(host(self.out[:self.M]), y, yb, "out")
        if self.keep_z:
            assert (self.z[self.M] == 77).all()
            within(host(self.z[:self.M]), z, zb, "z")

    def check_bwd(self):
        wsb = self.bwd()
        torch.cuda.synchronize()
        assert (self.dx[self.M] == 77).all() and (self.dw[self.N] == 77).all() and self.db[self.N] == 77
        assert (self.bws[wsb:] == 0xFF).all()
        want = ol.backward(val(self.dout), val(self.zin), val(self.x), val(self.w),
                           None if self.add is None else val(self.add), self.act)
        within(host(self.dx[:self.M]), *want["dx"], "dx")
        within(host(self.dw[:self.N]), *want["dw"], "dw")
        within(host(self.db[:self.N]), *want["db"], "db")


# rows of the streaming form (its 1, 2 and 4 token tiles), one past it, ragged tiles of each size, split contractions,
# columns that are not a multiple of 8, one column
SIZES = [(1, 8, 32), (1, 100, 96), (5, 64, 160), (16, 33, 544), (17, 48, 256), (64, 200, 2048), (65, 64, 64),
         (66, 1, 32), (100, 7, 352), (200, 130, 96), (257, 300, 224), (1000, 60, 2048), (300, 1000, 4096),
         (3000, 200, 320), (70, 2100, 1536), (4100, 3900, 96), (2500, 2700, 1120),
         # few rows: several items per workgroup, k past the registers; short contractions over several blocks;
         # whole rounds of tiles before a split one; the narrow tiles of a gate and of its weight gradient
         (3, 8209, 640), (16, 4500, 9248), (9, 40, 16416), (9000, 520, 64), (8191, 40, 2048), (4100, 4300, 1088),
         (8200, 64, 4096)]


@pytest.mark.parametrize("size", SIZES)
def test_forward(size):
    i = SIZES.index(size)
    c = Case(*size, act=ol.ACTS[i % 5], bias=i % 3 != 1, residual=i % 4 < 2, keep_z=i % 2 == 0, f32=i % 3 == 2)
    c.check_fwd()
    first = host(c.out).copy()
    c.out.fill_(77.0)
    c.fwd()
    torch.cuda.synchronize()
    assert np.array_equal(host(c.out), first)


@pytest.mark.parametrize("size", SIZES)
def test_backward(size):
    i = SIZES.index(size)
    c = Case(*size, act=ol.ACTS[i % 5], residual=i % 2 == 0, f32=i % 3 == 2)
    c.check_bwd()
    first = [host(t).copy() for t in (c.dx, c.dw, c.db)]
    for t in (c.dx, c.dw, c.db):
        t.fill_(77.0)
    c.bwd()
    torch.cuda.synchronize()
    for a, b in zip(first, (c.dx, c.dw, c.db)):
        assert np.array_equal(a, host(b))


@pytest.mark.parametrize("act", ol.ACTS)
def test_activations_over_their_range(act):
    """x = one column times w = 1: z runs over bf16 values far into both tails, fp32 out and the slope's db."""
    zs = np.concatenate([np.linspace(-30, 30, 4000), [0.0, 1e-30, -1e-30, 2.0 ** -100, -88.0, 88.0, 1e4, -1e4, 1e30, -1e30]])
    z = workloads.f32_to_bf16_bits(zs.astype(np.float32))
    n = z.size
    x = np.zeros((n, 32), np.uint16)
    x[:, 0] = z
    w = np.zeros((8, 32), np.uint16)
    w[0, 0] = 0x3F80
    out = torch.empty((n, 8), device=DEV)
    ws = torch.empty(max(16, mxa.mx_bf16_linear_workspace_size(n, 8, 32)), dtype=torch.uint8, device=DEV)
    mxa.mx_bf16_linear(dev(x), dev(w), None, None, n, 8, 32, ol.ACTS.index(act), None, out, F32, ws, ws.numel())
    torch.cuda.synchronize()
    v = mx.bf16_to_f64(z)
    with np.errstate(over="ignore", invalid="ignore"):
        want = ol.act(v, act)
        slope = ol.slope(v, act)
    if act == "gelu_tanh":
        want = np.where(np.abs(v) > 1e3, np.maximum(v, 0), want)
        slope = np.where(np.abs(v) > 1e3, v > 0, slope)
    err = np.abs(host(out)[:, 0] - want)
    assert (err <= 40 * 2.0 ** -24 * np.abs(v) + 2.0 ** -126).all(), np.argwhere(~(err <= 40 * 2.0 ** -24 * np.abs(v) + 2.0 ** -126))[:5]
    # the slope, one row at a time through dbias: dout is the unit column of each row
    rows = list(range(0, 4000, 400)) + list(range(4000, n))
    for r in rows:
        zt = torch.full((1, 8), 0.0, dtype=torch.bfloat16, device=DEV)
        zt[0, 0] = float(v[r])
        db = torch.empty(8, device=DEV)
        dx = torch.empty((1, 32), dtype=torch.bfloat16, device=DEV)
        bw = torch.empty(mxa.mx_bf16_linear_bwd_workspace_size(1, 8, 32, 1), dtype=torch.uint8, device=DEV)
        mxa.mx_bf16_linear_bwd(torch.ones((1, 8), device=DEV), F32, zt, None, dev(w), None, 1, 8, 32,
                               ol.ACTS.index(act), dx, None, db, bw, bw.numel())
        assert abs(float(db[0]) - float(slope[r])) <= 96 * 2.0 ** -24, (r, v[r], float(db[0]), slope[r])


def test_gradient_against_differences_of_the_kernel():
    """d sum(dout out) / dx[m, k] against a central difference of the fp32 forward: with steps of 2^-4 and weights of
    about 0.1 the third-order term is below 1e-5 and fp32 noise below 1e-4 of a gradient of about 1; dx itself is
    rounded to bf16 (2^-8 of it) from a dz of bf16 (2^-8 of its terms, which add up to about 0.004)."""
    c = Case(70, 96, 96, act="silu", residual=False, f32=True, keep_z=True)
    c.fwd()
    c.d["zin"] = c.z[:70].contiguous()
    c.bwd()
    dx = c.dx[:70].double()
    g = np.random.default_rng(3)
    for _ in range(12):
        m, k = int(g.integers(70)), int(g.integers(96))
        x0 = c.d["x"].clone()
        out = []
        base = float(c.d["x"].view(torch.bfloat16)[m, k])
        lo, hi = (float(torch.tensor(base + s * 2.0 ** -4).bfloat16()) for s in (-1, 1))
        for v in (lo, hi):
            c.d["x"].view(torch.bfloat16)[m, k] = v
            c.fwd()
            out.append((c.out[:70].double() * torch.from_numpy(c.dout).to(DEV).double()).sum())
        c.d["x"].copy_(x0)
        diff = float((out[1] - out[0]) / (hi - lo))
        assert abs(diff - float(dx[m, k])) < 0.015 * max(1.0, abs(diff)), (m, k, diff, float(dx[m, k]))


def test_parts_of_the_backward_alone():
    c = Case(130, 72, 160, act="gelu")
    c.bwd()
    torch.cuda.synchronize()
    wsb = mxa.mx_bf16_linear_bwd_workspace_size(130, 72, 160, 2)
    for part in ("dx", "dw", "db"):
        t = torch.zeros_like(getattr(c, part))
        mxa.mx_bf16_linear_bwd(c.d["dout"], BF, c.d["zin"], c.d["x"] if part == "dw" else None,
                               c.d["w"] if part == "dx" else None, c.d["add"] if part == "dx" else None, 130, 72, 160, 2,
                               t if part == "dx" else None, t if part == "dw" else None, t if part == "db" else None,
                               c.bws, wsb)
        torch.cuda.synchronize()
        n = {"dx": 130, "dw": 72, "db": 72}[part]
        assert torch.equal(t[:n], getattr(c, part)[:n]), part


def test_results_over_their_addends():
    c = Case(90, 64, 64, act="relu")
    c.fwd()
    c.bwd()
    want_out, want_dx = host(c.out[:90]), host(c.dx[:90])
    c.fwd(out=c.d["res"])
    wsb = mxa.mx_bf16_linear_bwd_workspace_size(90, 64, 64, 1)
    mxa.mx_bf16_linear_bwd(c.d["dout"], BF, c.d["zin"], c.d["x"], c.d["w"], c.d["add"], 90, 64, 64, 1, c.d["add"], None,
                           None, c.bws, wsb)
    torch.cuda.synchronize()
    assert np.array_equal(host(c.d["res"]), want_out) and np.array_equal(host(c.d["add"]), want_dx)


def test_no_rows():
    w = dev(np.zeros((40, 64), np.uint16))
    dw, db = torch.full((40, 64), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((40,), 7.0, device=DEV)
    e = torch.empty(16, device=DEV)
    mxa.mx_bf16_linear(e, w, None, None, 0, 40, 64, 0, None, e, F32, None, 0)
    mxa.mx_bf16_linear_bwd(e, F32, e, e, w, None, 0, 40, 64, 4, e, dw, db, None, 0)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("size", [(40, 96, 256), (200, 130, 512), (300, 520, 64)])
def test_nan_and_inf_stay_in_their_row(size):
    M, N, K = size
    c = Case(M, N, K, act="silu", residual=False)
    c.x[7, 3], c.x[30, K - 1] = 0x7FC0, 0x7F80
    c.d["x"] = dev(c.x)
    c.fwd()
    torch.cuda.synchronize()
    got = val(host(c.out[:M]))
    keep = np.ones(M, bool)
    keep[[7, 30]] = False
    assert np.isnan(got[7]).all() and not np.isfinite(got[30]).any() or np.isnan(got[7]).all()
    assert np.isfinite(got[keep]).all()
    c.x[7, 3] = c.x[30, K - 1] = 0
    y, yb, _, _ = ol.forward(val(c.x), val(c.w), c.bias, None, "silu", False)
    assert (np.abs(got - y)[keep] <= yb[keep]).all()


@pytest.mark.parametrize("size", [(9, 64, 512), (500, 72, 1024), (600, 520, 96)])
def test_captured_replays_on_another_stream(size):
    c = Case(*size, act="gelu_tanh")
    c.fwd()
    c.bwd()
    torch.cuda.synchronize()
    names = ("out", "z", "dx", "dw", "db")
    want = {n: host(getattr(c, n)).copy() for n in names}

    def both():
        c.fwd()
        c.bwd()

    g = moe.capture(both)
    other = Case(*size, act="gelu_tanh", seed=5)
    s = torch.cuda.Stream()
    for _ in range(3):
        for n in names:
            getattr(c, n).fill_(3.0)
        other.fwd()
        other.bwd()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        for n in names:
            a = host(getattr(c, n))
            k = -1 if n == "db" else slice(None, -1)
            assert np.array_equal(a[:-1], want[n][:-1]), (n, k)


TAILS = workloads.f32_to_bf16_bits(np.concatenate([np.linspace(-40, 40, 6001), -np.logspace(-30, 30, 183),
                                                   np.logspace(-30, 30, 184)]).astype(np.float32))


def tail_terms(v, act):
    """(act, its error in units of 2^-24 of itself, the terms of its slope added up, their error, the slope) in fp64.

    gelu: its exponential of -v^2 / 2 is off by 1.5 v^2 units and its own 2, the factor that makes it the tail by 6,
    the products by a few.  The sigmoids' 2^x: the product of its argument t is off by 2 |t|, the functions by a few
    units; gelu_tanh's t itself by 7 |t|, in each of its factors.  Past |t| = 200 (v^2 = 400) all of them are 0 or 1."""
    a, erfc = np.abs(v), np.vectorize(math.erfc, otypes=[np.float64])
    if act == "gelu":
        cdf, pdf = 0.5 * erfc(-v / math.sqrt(2)), np.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        k = 16 + 2 * np.minimum(v * v, 400)
        return v * cdf, k, cdf + a * pdf, k, cdf + v * pdf
    if act in ("silu", "gelu_tanh"):
        c = 2 * math.sqrt(2 / math.pi)
        t, dt = (v, np.ones_like(v)) if act == "silu" else (c * (v + 0.044715 * v ** 3), c * (1 + 3 * 0.044715 * v * v))
        s, m = 1 / (1 + np.exp(-t)), 1 / (1 + np.exp(t))
        b = np.minimum(np.abs(t), 200)
        k = (16 + 4 * b, 24 + 4 * b) if act == "silu" else (16 + 10 * b, 32 + 20 * b)
        with np.errstate(invalid="ignore"):
            p = np.where(s * m == 0, 0, v * s * m * dt)
        return v * s, k[0], s + np.abs(p), k[1], s + p
    one = np.ones_like(v) if act == "none" else (v > 0).astype(np.float64)
    return v * one, 0 * v, one, 0 * v, one


@pytest.mark.parametrize("act", ol.ACTS)
def test_activations_and_slopes_relative_to_their_value(act):
    """Far into the tails, where the value is far below its argument, an fp32 result still has most of its bits; what
    the hardware's 2^x flushes (below 2^-126) is all that may be lost beside that."""
    v = mx.bf16_to_f64(TAILS)
    n = v.size // 8 * 8
    v = v[:n]
    with np.errstate(over="ignore"):
        want, units, terms, slope_units, slope = tail_terms(v, act)
    least = 2.0 ** -125 * (1 + np.minimum(np.abs(v), 200)) ** 3
    x, w = np.zeros((n, 32), np.uint16), np.zeros((8, 32), np.uint16)
    x[:, 0], w[0, 0] = TAILS[:n], 0x3F80
    out = torch.empty((n, 8), device=DEV)
    wsb = mxa.mx_bf16_linear_workspace_size(n, 8, 32)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=DEV)
    mxa.mx_bf16_linear(dev(x), dev(w), None, None, n, 8, 32, ol.ACTS.index(act), None, out, F32, ws, wsb)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        err, bound = np.abs(host(out)[:, 0] - want), units * 2.0 ** -24 * np.abs(want) + least
    assert (err <= bound).all(), [(v[i], want[i], host(out)[i, 0]) for i in np.flatnonzero(~(err <= bound))[:5]]
    if act == "none":
        return
    # a row of n columns: dbias is the slope of each
    z, db = dev(TAILS[None, :n]), torch.empty(n, device=DEV)
    wsb = mxa.mx_bf16_linear_bwd_workspace_size(1, n, 32, ol.ACTS.index(act))
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    mxa.mx_bf16_linear_bwd(torch.ones((1, n), device=DEV), F32, z, None, None, None, 1, n, 32, ol.ACTS.index(act), None,
                           None, db, ws, wsb)
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        err, bound = np.abs(host(db) - slope), np.where(terms == 0, 0, slope_units * 2.0 ** -24 * terms) + least
    assert (err <= bound).all(), [(v[i], slope[i], host(db)[i]) for i in np.flatnonzero(~(err <= bound))[:5]]


@pytest.mark.parametrize("size", [(9, 96, 512), (40, 96, 256), (200, 130, 512), (300, 520, 64)])
def test_infinite_rows_are_not_finite(size):
    """x = inf gives z = +-inf in every column: silu(inf) = inf, silu(-inf) = NaN; a NaN row is NaN; the others stay."""
    M, N, K = size
    c = Case(M, N, K, act="silu", residual=False)
    c.x[7, 3], c.x[5, K - 1] = 0x7FC0, 0x7F80
    c.d["x"] = dev(c.x)
    c.fwd()
    torch.cuda.synchronize()
    got = val(host(c.out[:M]))
    assert np.isnan(got[7]).all()
    assert not np.isfinite(got[5]).any()
    c.x[7, 3] = c.x[5, K - 1] = 0
    y, yb, _, _ = ol.forward(val(c.x), val(c.w), c.bias, None, "silu", False)
    keep = np.delete(np.arange(M), [5, 7])
    assert (np.abs(got - y)[keep] <= yb[keep]).all()
