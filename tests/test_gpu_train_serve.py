"""The layer with its gate trained by AdamW and then served: the gate product,
the layer's forward and backward, the gate's backward, the AdamW step on all
weights and the few-token layer on the MXFP8 weights a step leaves, together."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
import workloads
from mxfp8_block_scaled_07_amd import moe
from oracle import adamw as oa
from oracle import linear as ol
from oracle import mxfp8 as mx
from oracle import tokens as ot

from gpu_util import DEV, dev, host, srows

pytestmark = pytest.mark.gpu

T, H, F, E, K = 200, 160, 96, 12, 3


class Trained:
    def __init__(self, state_bits):
        g = np.random.default_rng(8)
        self.x, self.dout = workloads.normal_bf16(g, (T, H), 1.0), workloads.normal_bf16(g, (T, H), 0.1)
        self.w = {"wg": g.standard_normal((E, H)) * H ** -0.5, "w1": g.standard_normal((E, 2 * F, H)) * H ** -0.5,
                  "w2": g.standard_normal((E, H, F)) * F ** -0.5}
        self.master = {k: dev(v.astype(np.float32)) for k, v in self.w.items()}
        self.weights = {k: v.to(torch.bfloat16) for k, v in self.master.items()}
        self.bg = torch.linspace(-0.2, 0.2, E, device=DEV)
        self.dx, self.dd = dev(self.x), dev(self.dout)
        self.b = moe.GatedLayerBuffers(T, H, F, E, K)
        grads = {"wg": self.b.dwg, "w1": self.b.dw1, "w2": self.b.dw2}
        self.opt = moe.Adamw([(self.master[k], grads[k], self.weights[k]) for k in self.w], state_bits, lr=2e-3, seed=3)
        self.bias = moe.Adamw([(self.bg, self.b.dbg, None)], 32, lr=2e-3, weight_decay=0.0)

    def step(self):
        moe.gated_layer_step(self.b, self.dx, self.weights["wg"], self.bg, self.weights["w1"], self.weights["w2"], self.dd)
        self.opt.step()
        self.bias.step()

    def state(self):
        t = {k: host(v).copy() for k, v in self.weights.items()}
        t.update({"m_" + k: host(v).copy() for k, v in self.master.items()})
        t.update(out=host(self.b.out).copy(), dx=host(self.b.dx).copy(), bg=host(self.bg).copy(),
                 states=[host(x).copy() for s in self.opt.states for x in s if x is not None])
        return t


def same(a, b):
    for k in a:
        if k == "states":
            assert all(np.array_equal(x, y) for x, y in zip(a[k], b[k])), k
        else:
            assert np.array_equal(a[k], b[k]), k


@pytest.mark.parametrize("bits", [8, 32])
def test_each_part_of_a_step(bits):
    t = Trained(bits)
    old = {k: host(v).copy() for k, v in t.weights.items()}
    master = {k: host(v).astype(np.float64) for k, v in t.master.items()}
    bg = host(t.bg).astype(np.float64)
    t.step()
    torch.cuda.synchronize()
    b = t.b
    x, wg = mx.bf16_to_f64(t.x), mx.bf16_to_f64(old["wg"])
    want, bound, _, _ = ol.forward(x, wg, bg, None, "none", True)
    assert (np.abs(host(b.logits) - want) <= bound).all()
    # the gate's backward adds to the layer's own gradient of x, which the layer alone gives again
    lone = moe.LayerBuffers(T, H, F, E, K)
    w1, w2 = dev(old["w1"]), dev(old["w2"])
    moe.layer_step(lone, t.dx, w1, w2, b.logits, t.dd)
    torch.cuda.synchronize()
    assert np.array_equal(host(lone.out), host(b.out)) and np.array_equal(host(lone.dlogits), host(b.dlogits))
    got = ol.backward(host(b.dlogits).astype(np.float64), None, x, wg, mx.bf16_to_f64(host(lone.dx)), "none")
    for k, v in (("dx", mx.bf16_to_f64(host(b.dx))), ("dw", mx.bf16_to_f64(host(b.dwg))), ("db", host(b.dbg))):
        assert (np.abs(v - got[k][0]) <= got[k][1]).all(), k
    # AdamW's first step from zero states: m = 0.1 g, v = 0.001 g^2 whatever the states' type
    for k, grad in (("wg", b.dwg), ("w1", b.dw1), ("w2", b.dw2)):
        gr = mx.bf16_to_f64(host(grad)).ravel()
        lr = float(np.float32(2e-3))
        (p, _, _), (pm, _) = oa.update(master[k].ravel(), gr, 0 * gr, 0 * gr, 1, lr, 1.0, 0.9, 0.999, 1e-8, 0.01)
        new = host(t.master[k]).ravel()
        assert (np.abs(new - p) <= 32 * 2.0 ** -24 * pm).all(), k
        assert np.array_equal(host(t.weights[k]).ravel(), workloads.f32_to_bf16_bits(new)), k
    assert int(t.opt.count) == 1 and int(t.bias.count) == 1


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_steps_are_the_eager_ones(bits):
    eager, graph = Trained(bits), Trained(bits)
    for _ in range(2):
        eager.step()                      # what the capture runs first
    g = moe.capture(graph.step)
    for _ in range(3):
        eager.step()                      # eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        same(eager.state(), graph.state())


def test_the_trained_layer_serves_its_tokens():
    t = Trained(8)
    for _ in range(4):
        t.step()
    b, n = t.b, 40
    # the MXFP8 weights are those of the last step's forward: quantize the new ones as a step does
    mxa.mx_quantize(t.weights["w1"], E, 2 * F, H, None, 2 * F, b.w1q, b.w1s, b.w1tq, b.w1ts)
    mxa.mx_quantize(t.weights["w2"], E, H, F, None, H, b.w2q, b.w2s, b.w2tq, b.w2ts)
    tb = moe.TokenBuffers(n, H, F, E, K)
    x = t.dx[:n].contiguous()
    moe.token_step(tb, x, t.weights["wg"], t.bg, (b.w1q, b.w1s), (b.w2q, b.w2s), residual=x)
    torch.cuda.synchronize()
    xv = mx.bf16_to_f64(t.x[:n])
    logits = host(tb.logits)
    want, bound, _, _ = ol.forward(xv, mx.bf16_to_f64(host(t.weights["wg"])), host(t.bg).astype(np.float64), None, "none", True)
    assert (np.abs(logits - want) <= bound).all()
    w1 = mx.mx_values(host(b.w1q).reshape(-1, H), srows(b.w1s, H)).reshape(E, 2 * F, H)
    w2 = mx.mx_values(host(b.w2q).reshape(-1, F), srows(b.w2s, F)).reshape(E, H, F)
    out, bound = ot.layer(xv, logits, w1, w2, K, xv)
    assert (np.abs(mx.bf16_to_f64(host(tb.out)) - out) <= bound).all()
    # bf16 weights, and the allocating helpers, give the same calls' results
    moe.token_step(tb, x, t.weights["wg"], t.bg, t.weights["w1"], t.weights["w2"], residual=x)
    lg, _ = mxa.bf16_linear(x, t.weights["wg"], t.bg, out_dtype=mxa.MX_OUT_F32)
    helper = mxa.moe_tokens(x, lg, K, t.weights["w1"], t.weights["w2"], residual=x)
    helper_mx = mxa.moe_tokens(x, lg, K, (b.w1q, b.w1s), (b.w2q, b.w2s), residual=x)
    torch.cuda.synchronize()
    assert torch.equal(helper, tb.out)
    got = np.abs(mx.bf16_to_f64(host(helper_mx)) - out)
    assert (got <= bound).all()


def test_helpers():
    g = np.random.default_rng(2)
    x, w = dev(workloads.normal_bf16(g, (90, 64), 1.0)).view(torch.bfloat16), dev(workloads.normal_bf16(g, (24, 64), 0.1)).view(torch.bfloat16)
    dout = dev(g.standard_normal((90, 24)).astype(np.float32))
    out, z = mxa.bf16_linear(x, w, act=mxa.MX_ACT_GELU, want_z=True)
    dx, dw, db = mxa.bf16_linear_bwd(dout, x, w, z, mxa.MX_ACT_GELU)
    torch.cuda.synchronize()
    y, yb, zz, zb = ol.forward(mx.bf16_to_f64(host(x)), mx.bf16_to_f64(host(w)), None, None, "gelu", False)
    assert (np.abs(mx.bf16_to_f64(host(out)) - y) <= yb).all() and (np.abs(mx.bf16_to_f64(host(z)) - zz) <= zb).all()
    want = ol.backward(host(dout).astype(np.float64), mx.bf16_to_f64(host(z)), mx.bf16_to_f64(host(x)),
                       mx.bf16_to_f64(host(w)), None, "gelu")
    for k, v in (("dx", mx.bf16_to_f64(host(dx))), ("dw", mx.bf16_to_f64(host(dw))), ("db", host(db))):
        assert (np.abs(v - want[k][0]) <= want[k][1]).all(), k
    e = x[:0]
    assert mxa.bf16_linear(e, w)[0].shape == (0, 24)
    dx, dw, db = mxa.bf16_linear_bwd(dout[:0], e, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_helpers_on_another_stream():
    """Workspaces are freed as the helpers return: what they allocate belongs to the call's stream, so that later
    allocations of the current stream do not get them while the kernels still run."""
    g = np.random.default_rng(3)
    x = dev(workloads.normal_bf16(g, (300, 2048), 1.0)).view(torch.bfloat16)
    w = dev(workloads.normal_bf16(g, (64, 2048), 0.1)).view(torch.bfloat16)
    dout = dev(g.standard_normal((300, 64)).astype(np.float32))
    want = [mxa.bf16_linear(x, w)[0], *mxa.bf16_linear_bwd(dout, x, w)]
    p, grad = torch.ones(3000, device=x.device), torch.ones(3000, device=x.device)
    opt = moe.Adamw([(p, grad, None)], lr=0.5, weight_decay=0.0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = [mxa.bf16_linear(x, w, stream=s.cuda_stream)[0], *mxa.bf16_linear_bwd(dout, x, w, stream=s.cuda_stream)]
        junk = [torch.full((1 << 20,), float("nan"), device=x.device) for _ in range(8)]
        opt.step(s.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
    # the gradient is constant, so each step moves by lr m / sqrt(v) = lr; the largest rounding in it is that of
    # 1 - beta2 = 1e-3 from an fp32 beta2, 2^-25 / 1e-3 < 2^-15 relative, with a few of 2^-24 beside it
    assert (p - (1 - 5 * 0.5)).abs().max() <= 5 * 0.5 * 2.0 ** -14 and int(opt.count) == 5
