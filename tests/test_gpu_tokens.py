"""GPU parity: the whole MoE layer for a few tokens (MXFP8 and bf16 weights)
against the fp64 oracle (oracle/tokens.py), whose bound counts the kernel's
roundings."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
import workloads
from mxfp8_block_scaled_07_amd import moe
from oracle import mxfp8 as mx
from oracle import tokens as ot

from gpu_util import DEV, dev, host, spanels

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, T, H, F, E, k, mxw, residual, seed=0, w_std=None):
        g = np.random.default_rng([seed, T, H, F, E, k])
        self.T, self.H, self.F, self.E, self.k, self.mxw = T, H, F, E, k, mxw
        std = H ** -0.5 if w_std is None else w_std
        self.x = workloads.normal_bf16(g, (T, H), 1.0, 0.01)
        self.logits = g.standard_normal((T, E)).astype(np.float32)
        w1 = workloads.normal_bf16(g, (E, 2 * F, H), std)
        w2 = workloads.normal_bf16(g, (E, H, F), F ** -0.5)
        self.res = workloads.normal_bf16(g, (T, H), 1.0) if residual else None
        if mxw:
            q1, s1 = mx.quantize_rowwise(w1.reshape(E * 2 * F, H))
            q2, s2 = mx.quantize_rowwise(w2.reshape(E * H, F))
            self.w = [dev(q1), dev(spanels(s1)), dev(q2), dev(spanels(s2))]
            self.w1, self.w2 = mx.mx_values(q1, s1).reshape(E, 2 * F, H), mx.mx_values(q2, s2).reshape(E, H, F)
        else:
            self.w = [dev(w1), dev(w2)]
            self.w1, self.w2 = mx.bf16_to_f64(w1), mx.bf16_to_f64(w2)
        self.wsb = mxa.mx_moe_tokens_workspace_size(T, k, E, F)
        # all ones: NaN wherever the layer would use what it has not written
        self.ws = torch.full((self.wsb + 64,), 0xFF, dtype=torch.uint8, device=DEV)
        self.out = torch.full((T + 1, H), 77.0, dtype=torch.bfloat16, device=DEV)

    def upload(self):
        self.dx, self.dl = dev(self.x), dev(self.logits)
        self.dr = dev(self.res) if self.res is not None else None

    def launch(self, stream=None, out=None):
        fn = mxa.mx_moe_tokens if self.mxw else mxa.mx_bf16_moe_tokens
        fn(self.dx, self.dl, self.T, self.k, self.E, self.H, self.F, *self.w, self.dr,
           self.out if out is None else out, self.ws, self.wsb, stream)

    def run(self):
        self.upload()
        self.launch()
        torch.cuda.synchronize()
        assert (self.out[self.T] == 77.0).all() and (self.ws[self.wsb:] == 0xFF).all()
        return host(self.out[:self.T])

    def check(self, got, rows=slice(None)):
        with np.errstate(invalid="ignore"):
            want, bound = ot.layer(mx.bf16_to_f64(self.x), self.logits, self.w1, self.w2, self.k,
                                   None if self.res is None else mx.bf16_to_f64(self.res))
        err = np.abs(mx.bf16_to_f64(got) - want)[rows]
        print("max err/bound", float((err / bound[rows]).max()) if err.size else 0.0)
        assert (err <= bound[rows]).all(), np.argwhere(~(err <= bound[rows]))[:5]


SIZES = [(40, 160, 96, 12, 3), (7, 96, 160, 9, 1), (1, 256, 192, 4, 2), (1, 64, 32, 1, 1), (5, 96, 64, 7, 3), (16, 160, 96, 16, 4), (17, 544, 160, 9, 3),
         (33, 512, 288, 64, 8), (64, 224, 64, 3, 3), (64, 256, 640, 300, 5), (20, 64, 32, 1024, 64), (2, 2048, 1408, 8, 2),
         # many tokens of one expert where few tiles of them fit the registers, rows longer than the registers hold
         (50, 2560, 64, 3, 2), (37, 4128, 96, 2, 1), (21, 8480, 64, 3, 2), (3, 16672, 32, 4, 2)]


@pytest.mark.parametrize("mxw", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_layer(size, mxw):
    print(size, mxw, flush=True)
    c = Case(*size, mxw, residual=size[0] % 2 == 1)
    first = c.run()
    c.check(first)
    c.out.fill_(77.0)
    assert np.array_equal(c.run(), first)


@pytest.mark.parametrize("mxw", [True, False])
def test_masked_and_tied_logits(mxw):
    c = Case(24, 128, 64, 70, 4, mxw, residual=True)
    low = np.finfo(np.float32).min
    c.logits[0, :] = -np.inf                 # padding
    c.logits[1, 2:] = -np.inf                # fewer left than topk
    c.logits[2, :] = low                     # the type's lowest value, all tied: the lowest ids
    c.logits[3, 5:] = low
    c.logits[4, :] = 0.0
    c.logits[4, ::2] = -0.0                  # -0 ties with +0
    c.logits[5, 65:] = c.logits[5, 0] + 3    # ties above 64 experts
    c.logits[6, 1] = 3e38                    # one weight of 1
    c.logits[-1, :] = -np.inf
    got = c.run()
    c.check(got)
    assert np.array_equal(got[0], c.res[0]) and np.array_equal(got[-1], c.res[-1])


def test_all_padding_reads_nothing():
    c = Case(3, 64, 32, 4, 2, True, residual=False)
    c.logits[:] = -np.inf
    assert (c.run() == 0).all()


def test_every_token_on_the_same_expert():
    c = Case(64, 96, 96, 5, 1, True, residual=False)
    c.logits[:] = 0.0
    c.logits[:, 3] = 1.0
    c.check(c.run())


@pytest.mark.parametrize("mxw", [True, False])
def test_nan_stays_in_its_row(mxw):
    c = Case(40, 96, 64, 6, 2, mxw, residual=True)
    c.logits[7, 3] = np.nan
    c.x[20, 5] = 0x7FC0
    c.x[21, 95] = 0x7F80                     # inf
    got = c.run()
    bad = [7, 20, 21]
    assert np.isnan(mx.bf16_to_f64(got[7])).all() and np.isnan(mx.bf16_to_f64(got[20])).all()
    c.logits[7, 3] = 0.0
    c.x[20, 5] = c.x[21, 95] = 0
    c.check(got, [t for t in range(40) if t not in bad])


def test_out_over_residual_and_other_stream():
    c = Case(9, 160, 96, 8, 2, True, residual=True)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.launch(out=c.dr)
    torch.cuda.current_stream().wait_stream(s)
    assert np.array_equal(host(c.dr), want)


def test_no_tokens():
    c = Case(1, 64, 32, 4, 2, True, residual=False)
    c.upload()
    c.T = 0
    c.launch()
    torch.cuda.synchronize()
    assert (c.out == 77.0).all()


def test_two_captured_graphs_replay_as_eager():
    cs = [Case(n, 256, 128, 16, 4, n == 6, residual=True, seed=n) for n in (6, 30)]
    want, graphs = [], []
    for c in cs:
        want.append(c.run())
        graphs.append(moe.capture(c.launch))
    for _ in range(3):
        for c in cs:
            c.out.fill_(77.0)
            c.launch(out=torch.empty_like(c.out))       # eager work between the replays
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, w in zip(cs, want):
            assert np.array_equal(host(c.out[:c.T]), w)


@pytest.mark.parametrize("mxw", [True, False])
@pytest.mark.parametrize("E", [6, 70, 300])
def test_nan_logits_of_either_sign(E, mxw):
    """A NaN makes its token's row NaN whatever its sign and payload, beside enough other logits, masked ones, +inf and
    more NaNs than topk."""
    c = Case(20, 96, 64, E, 2, mxw, residual=True)
    bits = c.logits.view(np.uint32)
    bad = []
    for i, nan in enumerate((0xFFC00000, 0xFFFFFFFF, 0x7FC00000, 0x7FFFFFFF, 0xFF800001, 0x7F800001)):
        bits[2 * i, E - 1 - i % 3] = nan
        bad.append(2 * i)
    c.logits[13, :] = -np.inf
    bits[13, 1] = 0xFFC00000
    c.logits[15, 0] = np.inf
    bits[15, 2] = 0xFFFFFFFF
    bits[17, :] = 0xFFC00000
    bad += [13, 15, 17]
    got = c.run()
    assert np.isnan(mx.bf16_to_f64(got[bad])).all()
    c.logits[bad] = 0.0
    c.check(got, [t for t in range(20) if t not in bad])


@pytest.mark.parametrize("mxw", [True, False])
def test_an_infinite_token_is_not_finite(mxw):
    """g is +-inf in every row of W1: silu(-inf) = -inf / inf is NaN, and NaN times any weight."""
    c = Case(40, 96, 64, 6, 2, mxw, residual=True)
    c.x[21, 95] = 0x7F80
    got = c.run()
    assert not np.isfinite(mx.bf16_to_f64(got[21])).any()
    c.x[21, 95] = 0
    c.check(got, [t for t in range(40) if t != 21])
