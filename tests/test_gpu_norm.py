"""GPU parity: the root-mean-square norm with the residual's addition, and its
backward, against the fp64 oracle (oracle/norm.py), whose bounds count the
roundings; its MX output against the quantize of its bf16 rows, byte for byte."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
import workloads
from mxfp8_block_scaled_07_amd import moe
from oracle import mxfp8 as mx
from oracle import norm

from gpu_util import DEV, dev, host, srows

pytestmark = pytest.mark.gpu

BF, F32 = mxa.MX_OUT_BF16, mxa.MX_OUT_F32
val = lambda a: mx.bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)  # noqa: E731


def within(got, want, bound, what):
    err = np.abs(val(got) - want)
    print(what, "max err/bound", float((err / bound).max()) if err.size else 0.0, flush=True)
    assert (err <= bound).all(), (what, np.argwhere(~(err <= bound))[:5])


def guarded(R, C, dtype):
    """R rows and a guard row behind them."""
    return torch.full((R + 1, C), 77, dtype=dtype, device=DEV)


class Case:
    def __init__(self, R, C, f32=False, x=True, residual=True, weight=True, eps=1e-6, seed=0):
        g = np.random.default_rng([seed, R, C])
        bits = lambda std: workloads.normal_bf16(g, (R, C), std, 0.002)  # noqa: E731
        stream = (lambda std: (g.standard_normal((R, C)) * std).astype(np.float32)) if f32 else bits
        self.R, self.C, self.f32, self.eps = R, C, f32, eps
        self.x = bits(1.0) if x else None
        self.res = stream(2.0) if residual else None
        self.w = (1 + 0.2 * g.standard_normal(C)).astype(np.float32) if weight else None
        self.dy, self.ds = bits(0.5), stream(0.5)
        self.wv = np.ones(C) if self.w is None else self.w.astype(np.float64)
        self.kind, self.dtype = (F32, torch.float32) if f32 else (BF, torch.bfloat16)
        d = lambda a: None if a is None else dev(a)  # noqa: E731
        self.d = {k: d(getattr(self, k)) for k in ("x", "res", "w", "dy", "ds")}

    def r(self):
        v = lambda a: None if a is None else val(a)  # noqa: E731
        return norm.stream_sum(v(self.x), v(self.res), self.f32)

    def fwd(self, s=None, y=None, q=None, sc=None, stream=None):
        mxa.mx_rmsnorm(self.d["x"], self.d["res"], self.kind, self.d["w"], self.R, self.C, self.eps, s, y, q, sc, stream)

    def check_fwd(self):
        R, C = self.R, self.C
        s, y, q = guarded(R, C, self.dtype), guarded(R, C, torch.bfloat16), guarded(R, C, torch.uint8)
        sc = torch.full(mxa.scale_shape(R, C), 77, dtype=torch.uint8, device=DEV)
        self.fwd(s, y, q, sc)
        torch.cuda.synchronize()
        for t in (s, y, q):
            assert (t[R] == 77).all()
        r = self.r()
        assert np.array_equal(val(host(s[:R])), r)
        within(host(y[:R]), *norm.forward(r, self.wv, self.eps), "y")
        want_q, want_s = mx.quantize_rowwise(host(y[:R]))
        assert np.array_equal(host(q[:R]), want_q) and np.array_equal(srows(sc, C), want_s)
        # each output by itself
        s1, y1, q1, sc1 = (torch.full_like(t, 5) for t in (s, y, q, sc))
        self.fwd(s=s1)
        self.fwd(y=y1)
        self.fwd(q=q1, sc=sc1)
        torch.cuda.synchronize()
        assert torch.equal(s1[:R], s[:R]) and torch.equal(y1[:R], y[:R]) and torch.equal(q1[:R], q[:R]) and torch.equal(sc1, sc)

    def bwd(self, total, dres, dx, dw, ds="own", stream=None):
        wsb = mxa.mx_rmsnorm_bwd_workspace_size(self.R, self.C) if dw is not None else 0
        ws = torch.full((wsb + 64,), 0xFF, dtype=torch.uint8, device=DEV)   # NaN where it is read unwritten
        mxa.mx_rmsnorm_bwd(self.d["dy"], total, self.d["ds"] if isinstance(ds, str) else ds, self.kind, self.d["w"], self.R,
                           self.C, self.eps, dres, dx, dw, ws, wsb, stream)
        return ws, wsb

    def total(self):
        r = self.r()
        return dev(r.astype(np.float32) if self.f32 else mx.f64_to_bf16(r))

    def check_bwd(self):
        R, C = self.R, self.C
        dres, dx, dw = guarded(R, C, self.dtype), guarded(R, C, torch.bfloat16), torch.full((C + 1,), 77.0, device=DEV)
        total = self.total()
        ws, wsb = self.bwd(total, dres, dx, dw)
        torch.cuda.synchronize()
        assert (dres[R] == 77).all() and (dx[R] == 77).all() and dw[C] == 77 and (ws[wsb:] == 0xFF).all()
        want = norm.backward(val(self.dy), self.r(), val(self.ds), self.wv, self.eps, self.f32)
        for k, t in (("dres", dres[:R]), ("dx", dx[:R]), ("dw", dw[:C])):
            within(host(t), *want[k], k)
        # each output by itself, and without a gradient of the sum
        dres1, dx1, dw1 = torch.empty_like(dres), torch.empty_like(dx), torch.empty_like(dw)
        self.bwd(total, dres1, None, None)
        self.bwd(total, None, dx1, None)
        self.bwd(total, None, None, dw1)
        torch.cuda.synchronize()
        assert torch.equal(dres1[:R], dres[:R]) and torch.equal(dx1[:R], dx[:R]) and torch.equal(dw1[:C], dw[:C])
        self.bwd(total, dres1, None, None, ds=None)
        torch.cuda.synchronize()
        lone = norm.backward(val(self.dy), self.r(), None, self.wv, self.eps, self.f32)
        within(host(dres1[:R]), *lone["dres"], "dres alone")


# one row and one block; a part of a panel; each number of threads and chunks per row; ragged bands of rows
SIZES = [(1, 32), (3, 64), (5, 160), (1, 1024), (7, 544), (70, 96), (33, 1056), (2, 2080), (300, 2048), (129, 4128),
         (1, 7168), (40, 8192), (5, 8224), (3, 20000), (2, 40032), (2, 65536), (3000, 32), (2500, 512)]


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_forward(R, C, f32):
    Case(R, C, f32).check_fwd()


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_backward(R, C, f32):
    Case(R, C, f32).check_bwd()


@pytest.mark.parametrize("kw", [dict(residual=False), dict(x=False), dict(x=False, f32=True), dict(residual=False, f32=True),
                                dict(weight=False), dict(eps=10.0), dict(weight=False, residual=False)])
def test_what_may_be_left_out(kw):
    c = Case(50, 288, **kw)
    c.check_fwd()
    c.check_bwd()


@pytest.mark.parametrize("f32", [False, True])
def test_in_place(f32):
    c = Case(40, 2080, f32)
    s, y = guarded(40, 2080, c.dtype), guarded(40, 2080, torch.bfloat16)
    c.fwd(s, y)
    total, dres, dw = c.total(), torch.empty_like(s), torch.empty(2080, device=DEV)
    c.bwd(total, dres, None, dw)
    mine, y2, ds, dw2 = c.d["res"].clone(), torch.empty_like(y), c.d["ds"].clone(), torch.empty_like(dw)
    c.d["res"] = mine
    c.fwd(mine, y2)
    c.bwd(total, ds, None, dw2, ds=ds)
    torch.cuda.synchronize()
    assert torch.equal(mine.view(c.dtype), s[:40]) and torch.equal(y2[:40], y[:40])
    assert torch.equal(ds.view(c.dtype), dres[:40]) and torch.equal(dw2, dw)


def test_rows_of_zeros_infinities_and_nan():
    """A row's values reach its own outputs alone: zero rows give zeros, others are what they are without their neighbours."""
    R, C = 37, 416
    c = Case(R, C, residual=False)
    c.x[3] = 0
    plain = Case(R, C, residual=False)
    plain.x[3] = 0
    for t in (c, plain):
        t.d["x"] = dev(t.x)
    special = [5, 11, 12]
    c.x[5, 17], c.x[11, 0], c.x[12, 415] = 0x7FC0, 0x7F80, 0xFF80   # NaN, inf, -inf
    c.d["x"] = dev(c.x)
    y, yp = guarded(R, C, torch.bfloat16), guarded(R, C, torch.bfloat16)
    c.fwd(y=y)
    plain.fwd(y=yp)
    dres, dp = torch.empty_like(y), torch.empty_like(y)
    c.bwd(dev(c.x), dres, None, None)
    plain.bwd(dev(plain.x), dp, None, None)
    torch.cuda.synchronize()
    keep = [r for r in range(R) if r not in special]
    assert torch.equal(y[keep], yp[keep]) and torch.equal(dres[keep], dp[keep])
    assert (y[3] == 0).all() and torch.isnan(y[5]).all() and torch.isnan(y[11, 0]) and torch.isnan(y[12, 415])
    assert (y[11, 1:] == 0).all()                       # 1 / sqrt(inf) = 0
    assert torch.isnan(dres[5]).all()


def test_a_row_past_the_squares_range():
    """|r| = 2^70: the squares add up to infinity, y is zero; |r| = 2^60: they do not."""
    x = torch.ones(3, 64, dtype=torch.bfloat16, device=DEV)
    x[0], x[1] = -2.0 ** 70, -2.0 ** 60
    total, y, _, _ = mxa.rmsnorm(x)
    torch.cuda.synchronize()
    assert torch.equal(total, x) and not y[0].any() and (y[1] == -1).all() and (y[2] == 1).all()


def test_no_rows():
    c = Case(1, 64)
    dw = torch.full((64,), 7.0, device=DEV)
    mxa.mx_rmsnorm_bwd(c.d["dy"], c.total(), None, BF, None, 0, 64, 1e-6, None, None, dw, None, 0)
    torch.cuda.synchronize()
    assert (dw == 0).all()
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    s, y, q, sc = mxa.rmsnorm(e, rowwise=True)
    assert y.shape == (0, 64) and q.shape == (0, 64)
    dres, dx, dw = mxa.rmsnorm_bwd(e, e)
    assert dres.shape == (0, 64) and (dw == 0).all()


def test_many_rows_past_32_bits():
    """Offsets past 2^32 bytes: the last rows of a tensor of 4.3 GB are those of a small call."""
    R, C = (1 << 31) // 8192 + 5, 8192
    x = torch.zeros(R, C, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    last = torch.randn(8, C, device=DEV, generator=g).to(torch.bfloat16)
    x[-8:] = last
    _, y, q, sc = mxa.rmsnorm(x, rowwise=True)
    _, ys, qs, ss = mxa.rmsnorm(last, rowwise=True)
    torch.cuda.synchronize()
    # (another split of the row's sum over threads: the last bit of s may differ)
    assert (y[-8:].float() - ys.float()).abs().max() <= 2.0 ** -8 * ys.float().abs().max() and not y[:-8].any()
    want_q, want_s = mx.quantize_rowwise(host(y[-8:]))
    assert np.array_equal(host(q[-8:]), want_q) and np.array_equal(host(sc[:, -8:]).transpose(1, 0, 2).reshape(8, -1), want_s)
    del y, q, sc
    dres, _, dw = mxa.rmsnorm_bwd(x, x)
    torch.cuda.synchronize()
    want = norm.backward(val(host(last)), val(host(last)), None, np.ones(C), 1e-6, False)
    within(host(dres[-8:]), *want["dres"], "dres")
    within(host(dw), want["dw"][0], want["dw"][1] * 4, "dw")   # (up to 128 rows more per thread, all of them zero)


def test_graph_and_streams():
    """Captured calls replay to the eager bits; a call on another stream gives them too."""
    c = Case(300, 7168)
    R, C = 300, 7168
    outs = lambda: (guarded(R, C, torch.bfloat16), guarded(R, C, torch.bfloat16), torch.zeros(C, device=DEV))  # noqa: E731
    want, got = outs(), outs()
    total, wsb = c.total(), mxa.mx_rmsnorm_bwd_workspace_size(R, C)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)

    def both(o, stream=None):
        mxa.mx_rmsnorm(c.d["x"], c.d["res"], BF, c.d["w"], R, C, 1e-6, None, o[0], None, None, stream)
        mxa.mx_rmsnorm_bwd(c.d["dy"], total, c.d["ds"], BF, c.d["w"], R, C, 1e-6, o[1], None, o[2], ws, wsb, stream)

    both(want)
    g = moe.capture(lambda: both(got))
    for _ in range(3):
        for t in got:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        both(want)
        assert all(torch.equal(a[:R], b[:R]) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = outs()
    torch.cuda.synchronize()
    both(other, s.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a[:R], b[:R]) for a, b in zip(other, want))


def test_helpers():
    c = Case(90, 352, f32=True)
    bfx = c.d["x"].view(torch.bfloat16)
    s, y, q, sc = mxa.rmsnorm(bfx, c.d["w"], c.d["res"], rowwise=True)
    dres, dx, dw = mxa.rmsnorm_bwd(c.d["dy"].view(torch.bfloat16), s, c.d["w"], c.d["ds"])
    torch.cuda.synchronize()
    r = c.r()
    assert np.array_equal(host(s), r.astype(np.float32))
    within(host(y), *norm.forward(r, c.wv, 1e-6), "y")
    want = norm.backward(val(c.dy), r, val(c.ds), c.wv, 1e-6, True)
    for k, t in (("dres", dres), ("dx", dx), ("dw", dw)):
        within(host(t), *want[k], k)
    b = mxa.rmsnorm(bfx)
    assert b[0] is bfx and b[2] is None
    d = mxa.rmsnorm_bwd(y, bfx, want_dweight=False)
    assert d[0] is d[1] and d[2] is None
