"""GPU parity: softmax cross entropy over a vocabulary with its gradient,
against the fp64 oracle (oracle/xent.py), whose bounds count the roundings."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
import workloads
from mxfp8_block_scaled_07_amd import moe
from oracle import mxfp8 as mx
from oracle import xent

from gpu_util import DEV, dev, host

pytestmark = pytest.mark.gpu

val = lambda a: mx.bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)  # noqa: E731


def within(got, want, bound, what):
    err = np.abs(val(got) - want)
    print(what, "max err/bound", float((err / bound).max()) if err.size else 0.0, flush=True)
    assert (err <= bound).all(), (what, np.argwhere(~(err <= bound))[:5])


class Case:
    def __init__(self, M, V, K, ignored=0.2, weighted=True, std=3.0, seed=0):
        g = np.random.default_rng([seed, M, V, K])
        self.M, self.V, self.K = M, V, K
        self.x = workloads.normal_bf16(g, (M, K), 1.0, 0.002)
        self.w = workloads.normal_bf16(g, (V, K), std * K ** -0.5)
        self.t = g.integers(0, V, M).astype(np.int32)
        out = g.random(M) < ignored
        self.t[out] = g.choice(np.array([-1, -100, V, V + 7, 2 ** 31 - 1, -2 ** 31]), out.sum()).astype(np.int32)
        self.rw = (g.random(M) * 2).astype(np.float32) if weighted else None
        self.put()

    def put(self):
        self.d = [None if a is None else dev(a) for a in (self.x, self.w, self.t, self.rw)]

    def outs(self):
        M, V, K = self.M, self.V, self.K
        f = lambda *s: torch.full(s, 77.0, device=DEV)  # noqa: E731
        b = lambda *s: torch.full(s, 77.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        return [f(M + 1), f(M + 1), b(M + 1, K), b(V + 1, K)]

    def call(self, loss=None, lse=None, dx=None, dw=None, stream=None, ws=None):
        grad = dx is not None or dw is not None
        wsb = mxa.mx_bf16_xent_workspace_size(self.M, self.V, self.K, grad)
        if ws is None:
            ws = torch.full((wsb + 64,), 0xFF, dtype=torch.uint8, device=DEV)   # NaN where it is read unwritten
        mxa.mx_bf16_xent(*self.d, self.M, self.V, self.K, loss, lse, dx, dw, ws, wsb, stream)
        return ws, wsb

    def check(self):
        o = self.outs()
        ws, wsb = self.call(*o)
        torch.cuda.synchronize()
        assert (ws[wsb:] == 0xFF).all()
        want = xent.run(val(self.x), val(self.w), self.t, self.rw)
        for name, t, n in zip(("loss", "lse", "dx", "dw"), o, (self.M, self.M, self.M, self.V)):
            assert (t[n:] == 77).all(), name
            within(host(t[:n]), *want[name], name)
        # the loss alone, and each gradient by itself
        alone = self.outs()
        self.call(alone[0], alone[1])
        ws, wsb = self.call(alone[0], None)
        self.call(None, None, alone[2])
        self.call(None, None, None, alone[3])
        torch.cuda.synchronize()
        for name, t, n in zip(("loss", "lse"), alone, (self.M, self.M)):
            within(host(t[:n]), *want[name], name + " alone")
        assert torch.equal(alone[2], o[2]) and torch.equal(alone[3], o[3])
        return want


# one row and one word; the few-row form and past it; each tile shape; split contractions; words that are no multiple
# of 8, of a strip or of a tile
SIZES = [(1, 1, 32), (1, 1000, 64), (2, 33, 32), (5, 100, 96), (16, 4099, 160), (17, 500, 64), (31, 64, 2048),
         (64, 2000, 256), (65, 129, 512), (100, 3001, 96), (257, 1000, 64), (300, 4100, 320), (1000, 777, 128),
         (40, 20011, 64), (2000, 40, 64), (513, 2049, 544), (8, 70, 8224), (3000, 3, 32)]


@pytest.mark.parametrize("M,V,K", SIZES)
def test_sizes(M, V, K):
    Case(M, V, K).check()


def test_tiles_of_256():
    """Enough tiles for the largest shape, ragged on all sides."""
    Case(2100, 8200, 64).check()


@pytest.mark.parametrize("M,V,K", [(2050, 6100, 2080), (4100, 1030, 4128), (1030, 4100, 4128)])
def test_long_contractions_in_tiles_of_256(M, V, K):
    """The three products, whole tiles and split ones, contractions that end inside a step."""
    Case(M, V, K).check()


@pytest.mark.parametrize("kw", [dict(ignored=0.0, weighted=False), dict(ignored=1.0), dict(std=0.0), dict(std=40.0),
                                dict(ignored=0.0, std=12.0)])
def test_inputs(kw):
    """No row left out or all of them; equal logits; rows whose softmax is one word's."""
    c = Case(150, 1003, 96, **kw)
    c.check()
    if kw.get("ignored") == 1.0:
        o = c.outs()
        c.call(*o)
        torch.cuda.synchronize()
        assert not o[0][:150].any() and not o[2][:150].any() and not o[3][:1003].any()


def test_a_certain_target():
    """The target far above the others: a loss near zero is not lost to rounding, its gradient is bounded by it."""
    c = Case(40, 300, 64, ignored=0.0, weighted=False)
    for i in range(0, 40, 2):
        c.w[c.t[i]] = mx.f64_to_bf16(mx.bf16_to_f64(c.x[i]) * 0.25)   # a logit of about 16 above the others
    c.put()
    c.check()


def test_what_left_out_rows_hold_does_not_matter():
    c = Case(90, 700, 64)
    o = c.outs()
    c.call(*o)
    gone = np.flatnonzero((c.t < 0) | (c.t >= c.V))
    assert len(gone) > 5
    c.x[gone[0]], c.x[gone[1], 3], c.x[gone[2]] = 0x7FC0, 0x7F80, 0xFF80   # NaN, inf, -inf
    c.rw[gone[3]] = np.nan
    c.put()
    n = c.outs()
    c.call(*n)
    torch.cuda.synchronize()
    live = np.setdiff1d(np.arange(90), gone)
    assert torch.equal(n[0], o[0]) and torch.equal(n[1][live], o[1][live])
    assert torch.equal(n[2], o[2]) and torch.equal(n[3], o[3])


def test_nan_and_infinite_rows_stay_in_their_rows():
    c = Case(90, 700, 64, ignored=0.0)
    o = c.outs()
    c.call(*o)
    c.x[7, 5], c.x[33] = 0x7FC0, 0x7F80
    c.put()
    n = c.outs()
    c.call(*n)
    torch.cuda.synchronize()
    rest = [i for i in range(90) if i not in (7, 33)]
    assert torch.equal(n[0][rest], o[0][rest]) and torch.equal(n[2][rest], o[2][rest])
    assert torch.isnan(n[0][[7, 33]]).all() and torch.isnan(n[2][[7, 33]]).all() and torch.isnan(n[3][:700]).all()


def test_differences():
    """The gradient against differences of the loss along a direction that bf16 holds exactly: x + h v, v of +-1 and 0."""
    M, V, K = 64, 500, 64
    c = Case(M, V, K, weighted=False, std=1.0)
    c.x = mx.f64_to_bf16(np.round(mx.bf16_to_f64(c.x) * 16) / 16)
    g = np.random.default_rng(5)
    v, h = g.integers(-1, 2, (M, K)).astype(np.float64), 1.0 / 16
    c.put()
    o = c.outs()
    c.call(*o)
    base = mx.bf16_to_f64(c.x)
    sums = []
    for s in (h, -h):
        c.x = mx.f64_to_bf16(np.clip(base + s * v, -7.9, 7.9))
        c.put()
        n = c.outs()
        c.call(n[0])
        torch.cuda.synchronize()
        sums.append(host(n[0])[:M].astype(np.float64))
    inside = (np.abs(base) < 7.8).all(1)
    num, got = (sums[0] - sums[1]) / (2 * h), (val(host(o[2][:M])) * v).sum(1)
    # the third derivative along v: of a log-sum of exponentials at most the cube of the logits' spread
    spread = np.abs(v @ mx.bf16_to_f64(c.w).T).max(1)
    bound = h * h / 6 * 8 * spread ** 3 + (2.0 ** -8 * 3 * np.abs(val(host(o[2][:M]))) @ np.ones(K)) + 2.0 ** -14
    assert (np.abs(num - got)[inside] <= bound[inside]).all()


def test_chunks_of_rows():
    """More rows than the workspace holds at once: rows as their chunks' own calls give them, dw their sum."""
    M, V, K = 2100, 1000000, 32
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(M, K, device=DEV, generator=g).to(torch.bfloat16)
    w = (torch.randn(V, K, device=DEV, generator=g) * 0.5).to(torch.bfloat16)
    t = torch.randint(-20, V, (M,), device=DEV, generator=g, dtype=torch.int32)
    rw = torch.rand(M, device=DEV, generator=g)
    loss, lse, dx, dw = mxa.bf16_xent(x, w, t, rw, want_grad=True)
    total, size = torch.zeros(V, K, device=DEV), torch.zeros(V, K, device=DEV)
    for r in (slice(0, 768), slice(768, 1536), slice(1536, 2100)):
        a = mxa.bf16_xent(x[r], w, t[r], rw[r], want_grad=True)
        assert torch.equal(a[0], loss[r]) and torch.equal(a[1], lse[r]) and torch.equal(a[2], dx[r])
        total += a[3].float()
        size += a[3].float().abs()
    # each part was rounded to bf16, and so is the sum
    assert ((dw.float() - total).abs() <= 2.0 ** -8 * 1.01 * (size + dw.float().abs()) + 2.0 ** -100).all()
    assert dw.any() and dx.any()


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.ones(300, 64, dtype=torch.bfloat16, device=DEV)
    t = torch.empty(0, dtype=torch.int32, device=DEV)
    loss, lse, dx, dw = mxa.bf16_xent(x, w, t, want_grad=True)
    assert loss.shape == (0,) and dx.shape == (0, 64) and not dw.any()
    dw = torch.full((301, 64), 7, dtype=torch.bfloat16, device=DEV)
    some = torch.zeros(64, dtype=torch.int32, device=DEV)
    mxa.mx_bf16_xent(w, w, some, None, 0, 300, 64, None, None, None, dw, None, 0)
    torch.cuda.synchronize()
    assert not dw[:300].any() and (dw[300] == 7).all()


def test_repeats_graph_and_streams():
    """The same bits again, from a replayed capture with eager work between, and from another stream."""
    c = Case(300, 4100, 320)
    want, got = c.outs(), c.outs()
    ws, _ = c.call(*want)
    graph = moe.capture(lambda: c.call(*got, ws=ws))
    for _ in range(3):
        for t in got:
            t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        c.call(*want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    s, other = torch.cuda.Stream(), c.outs()
    torch.cuda.synchronize()
    ws2, wsb = torch.empty_like(ws), 0
    torch.cuda.synchronize()
    c.call(*other, stream=s.cuda_stream, ws=ws2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))


def test_helper():
    c = Case(77, 410, 96)
    x, w = (t.view(torch.bfloat16) for t in c.d[:2])
    loss, lse, dx, dw = mxa.bf16_xent(x, w, c.d[2], c.d[3], want_grad=True)
    l2, s2, a, b = mxa.bf16_xent(x, w, c.d[2])
    torch.cuda.synchronize()
    want = xent.run(val(c.x), val(c.w), c.t, c.rw)
    for name, t in zip(("loss", "lse", "dx", "dw", "loss", "lse"), (loss, lse, dx, dw, l2, s2)):
        within(host(t), *want[name], name)
    assert a is None and b is None


@pytest.mark.parametrize("M,V", [(1, 64), (96, 640), (300, 4099), (2100, 8192)])
def test_improbable_words_keep_their_gradient(M, V):
    """Words of up to 31.5 nats below the most probable of their 64, and of 40 nats between the 64s: a word's row of dw
    is a sum of terms of one sign, so it is off by a rounding of dz and one of itself to bf16 (2^-8 each, ln 2 2^-11 of
    the kept logarithm beside them), however improbable the word."""
    K = 32
    c = Case(M, V, K, ignored=0.0)
    one, at = mx.f64_to_bf16(np.array(1.0)), np.arange(V)
    c.x[:, 0] = one
    c.w[:] = 0
    c.w[:, 0] = mx.f64_to_bf16(-0.5 * (at % 64) - 8.0 * (at // 64 % 6))
    c.t[:] = 0
    c.rw = c.rw + np.float32(0.01)
    c.put()
    want = c.check()["dw"]
    o = c.outs()
    c.call(*o)
    torch.cuda.synchronize()
    got = val(host(o[3][:V]))[1:, 0]
    err = np.abs(got / want[0][1:, 0] - 1)
    print("relative error", float(err.max()), "at word", 1 + int(err.argmax()), flush=True)
    assert (err < 2 * 2.0 ** -8 + 2.0 ** -11).all() and (want[1][1:, 0] < 0.01 * want[0][1:, 0]).all()


def test_words_past_what_is_kept_are_zero():
    """The documented floor: exp(z - m) of 2^-63.9 and more below its strip's largest has no gradient, nothing else does."""
    M, V, K = 70, 320, 32
    c = Case(M, V, K, ignored=0.0, weighted=False)
    c.x[:, 0] = mx.f64_to_bf16(np.array(1.0))
    c.w[:] = 0
    c.w[:, 0] = mx.f64_to_bf16(np.where(np.arange(V) % 32 == 5, 0.0, np.where(np.arange(V) % 2, -44.0, -45.0)))
    c.t[:] = 5
    c.put()
    want = c.check()["dw"][0][:, 0]
    o = c.outs()
    c.call(*o)
    torch.cuda.synchronize()
    got = val(host(o[3][:V]))[:, 0]
    low = c.w[:, 0] == mx.f64_to_bf16(np.array(-45.0))
    assert not got[low].any() and (np.abs(got / want - 1)[~low] < 0.01).all()


@pytest.mark.parametrize("M,chunk", [(8500, 4352), (9000, 4608)])
def test_chunks_of_rows_without_a_gradient(M, chunk):
    """More rows than the strips' sums of the workspace hold: each chunk's rows as a call on them alone gives them."""
    V, K = 1000000, 32
    assert mxa.mx_bf16_xent_workspace_size(M, V, K, False) == mxa.mx_bf16_xent_workspace_size(chunk, V, K, False)
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn(M, K, device=DEV, generator=g).to(torch.bfloat16)
    w = (torch.randn(V, K, device=DEV, generator=g) * 0.5).to(torch.bfloat16)
    t = torch.randint(-20000, V, (M,), device=DEV, generator=g, dtype=torch.int32)
    loss, lse, dx, dw = mxa.bf16_xent(x, w, t)
    for r in (slice(0, chunk), slice(chunk, M)):
        a = mxa.bf16_xent(x[r], w, t[r])
        assert torch.equal(a[0], loss[r]) and torch.equal(a[1], lse[r])
    out = t < 0
    assert out.any() and not loss[out].any() and (loss[~out] > 0).all() and dx is None and dw is None
    # rows on both sides of the border in fp64: a logit is off by K + 16 roundings of its terms, the logarithm's argument
    # by 128, the largest logit's sum with it by a few of either
    for i in (0, chunk - 1, chunk, M - 1):
        z, mag = (a.double() @ b.double().T for a, b in ((x[i], w), (x[i].abs(), w.abs())))
        want = torch.logsumexp(z, 0)
        assert (lse[i] - want).abs() <= 2.0 ** -24 * ((K + 16) * mag.max() + 128 + 8 * want.abs()), i
        if t[i] >= 0:
            assert (loss[i] - (want - z[t[i]])).abs() <= 2.0 ** -24 * (2 * (K + 16) * mag.max() + 128 + 16 * want.abs()), i


def test_row_weights_of_any_size_and_sign():
    c = Case(90, 700, 64, ignored=0.1)
    c.rw = np.resize(np.array([-2.0, 0.0, 1e-20, 1e20, 1.0, -1e-3], np.float32), 90)
    c.put()
    c.check()
    o = c.outs()
    c.call(*o)
    torch.cuda.synchronize()
    assert not o[2][:90][torch.from_numpy(c.rw == 0).to(DEV)].any()


@pytest.mark.parametrize("M,V", [(3, 40), (70, 1000), (2100, 8200)])
def test_logits_near_the_range_of_fp32(M, V):
    """One word of 2^100 and all others of -2^100: their differences overflow to exponentials of exactly zero."""
    K, top = 32, V // 2
    c = Case(M, V, K, ignored=0.0, weighted=False)
    c.x[:], c.w[:] = 0, 0
    c.x[:, 0] = mx.f64_to_bf16(np.array(2.0 ** 50))
    c.w[:, 0] = mx.f64_to_bf16(np.where(np.arange(V) == top, 2.0 ** 50, -2.0 ** 50))
    c.t[:] = np.arange(M) % 2 * (V - 1 - top) + top         # the word itself, the last word
    c.put()
    o = c.outs()
    c.call(*o)
    torch.cuda.synchronize()
    odd = np.arange(M) % 2
    assert (host(o[1])[:M] == 2.0 ** 100).all() and np.array_equal(host(o[0])[:M], (odd * 2.0 ** 101).astype(np.float32))
    dx, dw = np.zeros((M, K)), np.zeros((V, K))
    dx[:, 0] = odd * 2.0 ** 51
    dw[top, 0], dw[V - 1, 0] = odd.sum() * 2.0 ** 50, -odd.sum() * 2.0 ** 50
    assert np.array_equal(val(host(o[2][:M])), dx)
    assert np.array_equal(val(host(o[3][:V])), mx.bf16_to_f64(mx.f64_to_bf16(dw)))
