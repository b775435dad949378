"""GPU parity: the AdamW step over many tensors against the fp64 oracle
(oracle/adamw.py).

fp32 results within 16 fp32 roundings of the magnitudes they are sums of (the
constants, the division, the root and the products are each within a few).
Stochastically rounded results are the oracle's own code wherever the fp64
value is clear of its threshold (fp32 roundings move it by far less than the
2^-14 of a step that is set aside), and one of the two neighbours elsewhere."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
import workloads
from mxfp8_block_scaled_07_amd import moe
from oracle import adamw as oa
from oracle import mxfp8 as mx

from gpu_util import DEV, dev, host

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24
HYPER = dict(b1=0.9, b2=0.999, eps=1e-8, wd=0.1)


class Set:
    """Tensors at 32-element starts of flat buffers, with a canary in every gap."""

    def __init__(self, sizes, p32, g32, bits, copy, seed=0, gstd=1e-3):
        g = np.random.default_rng([seed, len(sizes), sum(sizes)])
        self.sizes, self.p32, self.g32, self.s8, self.seed = sizes, p32, g32, bits == 8, (9 << 33) + 77 + seed
        self.at, end = [], 0
        for n in sizes:
            self.at.append(end)
            end += -(-n // 32) * 32 + 32
        self.end = end
        self.p = (g.standard_normal(end) * 0.02).astype(np.float32)
        self.g = (g.standard_normal(end) * gstd).astype(np.float32)
        if not p32:
            self.p = workloads.f32_to_bf16_bits(self.p)
        if not g32:
            self.g = workloads.f32_to_bf16_bits(self.g)
        m = g.standard_normal(end) * 2e-4
        r = np.abs(g.standard_normal(end)) * 1e-3
        m[::97] = r[::97] = 0.0
        self.m, self.v, self.ms, self.vs = m.astype(np.float32), (r * r).astype(np.float32), None, None
        if self.s8:
            self.ms, self.vs = oa.scale_bytes(m)[0], oa.scale_bytes(r)[0]
            self.m, _ = oa.encode(m, np.full(end, 32768.0), self.ms, False)
            self.v, _ = oa.encode(r, np.full(end, 32768.0), self.vs, True)
        names = ("p", "g", "m", "v") + (("ms", "vs") if self.s8 else ())
        self.d = {k: dev(getattr(self, k).copy()) for k in names}
        self.d["copy"] = torch.full((end,), 7.0, dtype=torch.bfloat16, device=DEV) if copy else None
        self.lr = torch.tensor([1e-3], device=DEV)
        self.step = torch.tensor([0], dtype=torch.int32, device=DEV)
        self.scale = torch.tensor([0.5], device=DEV)
        rows = []
        for n, a in zip(sizes, self.at):
            b = slice(a // 32, a // 32 + -(-n // 32))
            t = {k: None if x is None else (x[b] if k in ("ms", "vs") else x[a:a + n]) for k, x in self.d.items()}
            rows.append((t["p"], t["g"], t["m"], t["v"], t.get("ms"), t.get("vs"), t["copy"]))
        self.table = mxa.adamw_table(rows)

    def launch(self, stream=None):
        f, b = mxa.MX_OUT_F32, mxa.MX_OUT_BF16
        mxa.mx_adamw(self.table, len(self.sizes), f if self.p32 else b, f if self.g32 else b, 8 if self.s8 else 32,
                     self.lr, self.step, self.scale, HYPER["b1"], HYPER["b2"], HYPER["eps"], HYPER["wd"], self.seed,
                     stream)

    def read(self):
        return {k: host(x) for k, x in self.d.items() if x is not None}

    def check(self, old, got, step):
        live = np.zeros(self.end, bool)
        blocks = np.zeros(self.end // 32, bool)
        unsure = 0
        wide = lambda a: mx.bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)  # noqa: E731
        for i, (n, a) in enumerate(zip(self.sizes, self.at)):
            w, blk = slice(a, a + n), slice(a // 32, a // 32 + -(-n // 32))
            live[w], blocks[blk] = True, True
            if n == 0:
                continue
            m, v = old["m"][w], old["v"][w]
            if self.s8:
                m, v = oa.decode(m, old["ms"][blk]), oa.decode(v, old["vs"][blk]) ** 2
            (p2, m2, v2), (pm, mm) = oa.update(wide(old["p"][w]), wide(old["g"][w]), m.astype(np.float64),
                                               v.astype(np.float64), step, float(np.float32(1e-3)), 0.5, **HYPER)
            h = oa.bits(self.seed, step, i, n)
            if self.s8:
                for name, val, u, root in (("m", m2, h >> np.uint64(16), False), ("v", np.sqrt(v2), h & np.uint64(0xFFFF), True)):
                    by, top = oa.scale_bytes(val)
                    mant = np.frexp(top)[0]
                    clear = np.abs(mant - 0.875) > 2.0 ** -20      # the scale is not a matter of rounding
                    gb = got[name + "s"][blk]
                    assert np.array_equal(gb[clear], by[clear]), (i, name)
                    codes, near = oa.encode(val, u.astype(np.float64), gb, root)
                    gc = got[name][w]
                    ok = (gc == codes) | near
                    # m cancels: its fp32 error is in roundings of its terms, which may reach 2^-14 of a small code's step
                    err = 8 * F32 * (mm if name == "m" else val)
                    step_at = np.maximum(np.abs(oa.decode(gc, gb)) / 16, 2.0 ** -9 * np.repeat(2.0 ** (gb - 127.0), 32)[:n])
                    ok |= err > 2.0 ** -14 * step_at
                    assert ok.all(), (i, name, np.argwhere(~ok)[:5])
                    # at most a code's step away: an eighth of the value, or 2^-9 of the scale below the normal codes;
                    # and the fp32 value's own error (where m cancels to 0 in fp64, fp32 leaves a rounding of its
                    # terms, of either sign, which a large u rounds up to a whole smallest code: 2^-9 + err)
                    least = 2.0 ** -9 * np.repeat(2.0 ** (gb - 127.0), 32)[:n]
                    assert (np.abs(oa.decode(gc, gb) - val) <= np.maximum(np.abs(val) / 8 * 1.001, least) + err).all()
                    unsure += int(near.sum())
            else:
                assert (np.abs(got["m"][w] - m2) <= 16 * F32 * mm + 2.0 ** -140).all(), i
                assert (np.abs(got["v"][w] - v2) <= 16 * F32 * v2 + 2.0 ** -140).all(), i
            if self.p32:
                assert (np.abs(got["p"][w] - p2) <= 32 * F32 * pm).all(), (i, np.max(np.abs(got["p"][w] - p2) / pm) / F32)
                if "copy" in got:
                    assert np.array_equal(got["copy"][w], workloads.f32_to_bf16_bits(got["p"][w]))
            else:
                u = oa.mix(h ^ np.uint64(oa.GOLD)) >> np.uint64(16)
                bits, near = oa.round_bf16(p2, u.astype(np.float64))
                # 32 fp32 roundings of the terms against 2^-12 of a bf16 step of the result
                near |= 32 * F32 * pm > 2.0 ** -12 * 2.0 ** -8 * np.abs(p2)
                assert ((got["p"][w] == bits) | near).all(), i
                d = np.abs(mx.bf16_to_f64(got["p"][w]) - p2)
                assert (d <= 2.0 ** -7 * 1.001 * np.abs(p2) + 32 * F32 * pm).all()
                if "copy" in got:
                    assert np.array_equal(got["copy"][w], got["p"][w])
        for k in ("p", "g", "m", "v", "copy"):
            if k in got:
                assert np.array_equal(got[k][~live], old[k][~live]), k
        if self.s8:
            for k in ("ms", "vs"):
                assert np.array_equal(got[k][~blocks], old[k][~blocks]), k
        assert np.array_equal(got["g"], old["g"])
        print("elements", int(live.sum()), "near a threshold", unsure)


RAGGED = [1, 31, 32, 33, 0, 1023, 1024, 1025, 100003, 7]


@pytest.mark.parametrize("p32,g32,bits,copy", [(True, True, 32, False), (True, False, 8, True), (False, False, 8, False),
                                               (False, True, 32, True), (True, True, 8, False), (False, False, 32, False)])
def test_step(p32, g32, bits, copy):
    s = Set(RAGGED, p32, g32, bits, copy)
    for t in (1, 2, 500):
        s.step.fill_(t)
        old = s.read()
        s.launch()
        torch.cuda.synchronize()
        s.check(old, s.read(), t)


@pytest.mark.parametrize("bits", [8, 32])
def test_more_tensors_than_one_launch_takes(bits):
    g = np.random.default_rng(5)
    s = Set([int(n) for n in g.integers(1, 5000, 117)], True, False, bits, True)
    s.step.fill_(3)
    old = s.read()
    s.launch()
    torch.cuda.synchronize()
    s.check(old, s.read(), 3)


def test_one_large_tensor():
    s = Set([40_000_003], True, False, 8, False)      # several passes per block
    s.step.fill_(10)
    old = s.read()
    s.launch()
    torch.cuda.synchronize()
    s.check(old, s.read(), 10)


def test_repeated_step_gives_the_same_bits_on_another_stream():
    a, b = Set(RAGGED, False, False, 8, True), Set(RAGGED, False, False, 8, True)
    a.step.fill_(4)
    b.step.fill_(4)
    a.launch()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b.launch(st.cuda_stream)
    torch.cuda.synchronize()
    x, y = a.read(), b.read()
    for k in x:
        assert np.array_equal(x[k], y[k]), k


def test_zero_state_and_zero_gradient():
    s = Set([1000], True, True, 8, False)
    for k in ("m", "v", "ms", "vs", "g"):
        s.d[k].zero_()
    s.step.fill_(1)
    old = s.read()
    s.launch()
    torch.cuda.synchronize()
    got = s.read()
    assert (got["m"][:1000] & 0x7F == 0).all() and (got["v"][:1000] == 0).all() and (got["vs"][:32] == 0).all()
    s.check(old, got, 1)


def test_extreme_gradients():
    s = Set([256], True, True, 8, False)
    s.d["g"][:256] = torch.tensor([0.0, 1e-30, 1e-12, 1.0, 1e4, 1e18, -1e15, 2.0] * 32, device=DEV)
    s.step.fill_(1)
    s.launch()
    torch.cuda.synchronize()
    got = s.read()
    p = got["p"][:256]
    assert np.isfinite(p).all()
    # every positive root keeps a code: the next step divides by more than eps
    g = host(s.d["g"])[:256]
    assert (got["v"][:256][np.abs(g) > 1e-15] > 0).all()
    s.d["g"].zero_()
    before = p
    s.launch()
    torch.cuda.synchronize()
    assert (np.abs(s.read()["p"][:256] - before) <= 2 * 1e-3 * 12 + 1e-3 * np.abs(before)).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_nonfinite_gradients_stay_in_their_elements(bits):
    s = Set([96], True, True, bits, False)
    s.d["g"][40] = float("nan")
    s.d["g"][41] = float("inf")
    s.step.fill_(2)
    s.launch()
    torch.cuda.synchronize()
    got = s.read()
    bad = np.zeros(96, bool)
    bad[[40, 41]] = True
    m = oa.decode(got["m"], got["ms"])[:96] if bits == 8 else got["m"][:96]
    assert np.array_equal(np.isfinite(got["p"][:96]), ~bad) and np.array_equal(np.isfinite(m), ~bad)


def test_root_decays_without_bias():
    """With no gradient the root shrinks by sqrt(b2) a step, on average: after 1000 steps by 0.999^500.  A step's
    rounding has a variance of at most 0.0005 / 8 of the root's square (it moves by 0.0005 of itself, a code's step is at
    most an eighth), so an element is off by 25% at most in standard deviation and the mean of 65536 by 0.1%."""
    n = 65536
    s = Set([n], True, True, 8, False)
    s.d["g"].zero_()
    start = oa.decode(host(s.d["v"])[:n], host(s.d["vs"])[:n // 32])
    keep = start > 2e-4
    for t in range(1, 1001):
        s.step.fill_(t)
        s.launch()
    torch.cuda.synchronize()
    end = oa.decode(host(s.d["v"])[:n], host(s.d["vs"])[:n // 32])
    ratio = end[keep].sum() / start[keep].sum()
    print("decayed to", ratio, "of", 0.999 ** 500)
    assert abs(ratio / 0.999 ** 500 - 1) < 0.006


def test_captured_step_follows_step_and_lr():
    a, b = (Set([5000, 33], True, False, 8, True, seed=1) for _ in range(2))

    def one(s):
        s.step.add_(1)
        s.launch()

    ref = []
    g = None
    for _ in range(2):                                 # what capture runs first, eagerly
        one(b)
    for r in range(3):
        b.lr.fill_(1e-3 * (r + 1))
        one(b)
        torch.cuda.synchronize()
        ref.append(b.read())
    g = moe.capture(lambda: one(a))
    for r in range(3):
        a.lr.fill_(1e-3 * (r + 1))
        g.replay()
        torch.cuda.synchronize()
        got = a.read()
        for k in ref[r]:
            assert np.array_equal(got[k], ref[r][k]), (r, k)
        one(b)                                          # eager work between the replays


def test_the_class_under_another_default_type():
    """Its states and its lr are fp32 whatever torch makes by default."""
    p, g = (torch.linspace(-1, 1, 1000, dtype=torch.float32, device=DEV) for _ in range(2))
    want = p.clone()
    moe.Adamw([(want, g, None)], lr=0.25).step()
    torch.set_default_dtype(torch.bfloat16)
    try:
        opt = moe.Adamw([(p, g, None)], lr=0.25)
        assert opt.lr.dtype == torch.float32 and all(t.dtype == torch.float32 for t in opt.states[0][:2])
        opt.step()
    finally:
        torch.set_default_dtype(torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(p, want)


def test_a_refused_step_is_not_counted():
    p = torch.ones(64, device=DEV)
    opt = moe.Adamw([(p, torch.ones(64, device=DEV), None)])
    opt.step()
    opt.betas = (0.9, 1.5)
    with pytest.raises(mxa.MXError):
        opt.step()
    torch.cuda.synchronize()
    assert int(opt.count) == 1
