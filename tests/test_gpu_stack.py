"""A stack of layers from the residual stream to the loss: the norm, the layer
with its activations kept in MXFP8 and the cross entropy run together, trained
by AdamW, captured, and scoring tokens."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
from mxfp8_block_scaled_07_amd import moe

from gpu_util import DEV

pytestmark = pytest.mark.gpu

bf = torch.bfloat16


def model(T, H, F, E, V, L, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    layers = [[1 + n(H, std=0.1), n(E, H, std=H ** -0.5).to(bf), n(E, std=0.1), n(E, 2 * F, H, std=H ** -0.5).to(bf),
               n(E, H, F, std=F ** -0.5).to(bf)] for _ in range(L)]
    t = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    t[::9] = -1
    return n(T, H).to(bf), layers, 1 + n(H, std=0.1), n(V, H, std=2 * H ** -0.5).to(bf), t, torch.rand(T, generator=g, device=DEV)


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


def test_a_step_is_its_parts():
    """Forward: bit for bit the layer that keeps bf16.  Backward: bit for bit that layer's, run on the values the kept
    codes stand for; the router's gradient near the one from the down product's rows."""
    T, H, F, E, k, V, L = 200, 160, 96, 12, 3, 700, 2
    x, layers, norm, wv, t, rw = model(T, H, F, E, V, L)
    b = moe.StackBuffers(T, H, F, E, k, V, L)
    moe.stack_step(b, x, layers, norm, wv, t, rw)
    torch.cuda.synchronize()
    out, total, refs = None, x, []
    for n, wg, bg, w1, w2 in layers:
        if out is None:
            total, y, xq, xs = mxa.rmsnorm(total, n, rowwise=True)
        else:
            total, y, xq, xs = mxa.rmsnorm(out, n, total, rowwise=True)
        r = moe.LayerBuffers(T, H, F, E, k)
        logits, _ = mxa.bf16_linear(y, wg, bg, out_dtype=mxa.MX_OUT_F32)
        for s in moe.LAYER_STAGES[:9]:
            moe.run_layer_stage(s, r, y, w1, w2, logits, None)
        assert torch.equal(r.xq, xq) and torch.equal(r.xs, xs)
        refs.append((r, y, total))
        out = r.out.clone()
    total, y, _, _ = mxa.rmsnorm(out, norm, total)
    loss, lse, dx, dwv = mxa.bf16_xent(y, wv, t, rw, want_grad=True)
    dsum, _, dn = mxa.rmsnorm_bwd(dx, total, norm)
    torch.cuda.synchronize()
    assert torch.equal(loss, b.loss) and torch.equal(lse, b.lse) and torch.equal(dwv, b.dwv) and torch.equal(dn, b.dnorm)
    assert not loss[::9].any()
    for kept, (n, wg, bg, w1, w2), (r, y, s) in reversed(list(zip(b.kept, layers, refs))):
        cap = r.cap
        kq, ks, _, _ = mxa.quantize(r.h)
        live = torch.zeros(cap, dtype=torch.bool, device=DEV)
        live[:int(r.off[-1])] = True
        assert torch.equal(kq[live], kept.hq[live]) and torch.equal(kept.sum, s) and torch.equal(kept.ids, r.ids)
        r.h = mxa.dequantize(kq, ks)                       # what the kept codes stand for
        xv = mxa.dequantize(r.xq, r.xs)
        moe.run_layer_stage("swiglu", r, xv, w1, w2, None, dsum)
        for stage in moe.LAYER_STAGES[9:]:
            moe.run_layer_stage(stage, r, xv, w1, w2, None, dsum)
        dots = mxa.swiglu_bwd_kept(kq, ks, r.da, False, False, False)[6]
        dl = mxa.router_bwd_dots(dots, r.dst, r.ids, r.weights, E)
        assert torch.equal(kept.dw2, r.dw2) and torch.equal(kept.dw1, r.dw1)
        # both estimate the same sum from operands rounded to E4M3: two of them (dY, W2^T) and A' on this side, A and W2
        # on the other, each off by 2^-4 at most, 0.03 root mean square; five independent ones give 0.07
        assert rel(dl, r.dlogits) < 4 * 0.07
        dx, dwg, dbg = mxa.bf16_linear_bwd(dl, y, wg, dx_add=r.dx)
        assert torch.equal(kept.dwg, dwg) and torch.equal(kept.dbg, dbg)
        dsum, _, dn = mxa.rmsnorm_bwd(dx, s, n, dsum)
        assert torch.equal(kept.dnorm, dn)
    assert torch.equal(b.dsum, dsum)


def test_against_autograd():
    """fp64 autograd of the same network; every expert is chosen, so that no choice can differ.  The operands of six
    products a layer are E4M3, off by 0.03 root mean square each: a gradient passes through at most three of them per
    layer on its way, with two operands each."""
    T, H, F, E, V, L = 96, 128, 64, 4, 300, 2
    x, layers, norm, wv, t, rw = model(T, H, F, E, V, L, seed=3)
    b = moe.StackBuffers(T, H, F, E, E, V, L)
    moe.stack_step(b, x, layers, norm, wv, t, rw)
    torch.cuda.synchronize()
    d = lambda v: v.double().requires_grad_()  # noqa: E731
    rms = lambda v, w: v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    s = x0 = d(x)
    ws = [[d(v) for v in layer] for layer in layers]
    nv, wvd = d(norm), d(wv)
    for n, wg, bg, w1, w2 in ws:
        y = rms(s, n)
        p = torch.softmax(y @ wg.t() + bg, 1)
        out = 0
        for e in range(E):
            h = y @ w1[e].t()
            out = out + p[:, e:e + 1] * ((torch.nn.functional.silu(h[:, :F]) * h[:, F:]) @ w2[e].t())
        s = s + out
    z = rms(s, nv) @ wvd.t()
    live = t >= 0
    loss = torch.where(live, torch.logsumexp(z, 1) - z.gather(1, t.long().clamp_min(0).unsqueeze(1)).squeeze(1), 0.0)
    (loss * rw).sum().backward()
    noise = 0.03 * (2 * 3 * L) ** 0.5                     # 0.10
    assert rel(b.loss, loss.detach()) < noise
    assert rel(b.dwv, wvd.grad) < 2 * noise and rel(b.dnorm, nv.grad) < 2 * noise and rel(b.dsum, x0.grad) < 2 * noise
    for kept, (n, wg, bg, w1, w2) in zip(b.kept, ws):
        for name, got, want in (("norm", kept.dnorm, n), ("wg", kept.dwg, wg), ("bg", kept.dbg, bg), ("w1", kept.dw1, w1),
                                ("w2", kept.dw2, w2)):
            print(name, rel(got, want.grad), flush=True)
            assert rel(got, want.grad) < 3 * noise, name


@pytest.mark.parametrize("T", [1, 37])
def test_a_batch_without_targets(T):
    """Every target masked: no loss, and gradients that are exactly zero."""
    x, layers, norm, wv, t, _ = model(T, 128, 64, 4, 300, 2, seed=4)
    b = moe.StackBuffers(T, 128, 64, 4, 2, 300, 2)
    moe.stack_step(b, x, layers, norm, wv, torch.full_like(t, -1))
    torch.cuda.synchronize()
    assert torch.isfinite(b.lse).all() and not b.loss.any()
    for grad in (b.dsum, b.dwv, b.dnorm):
        assert not grad.any()
    for kept in b.kept:
        for grad in (kept.dnorm, kept.dwg, kept.dbg, kept.dw1, kept.dw2):
            assert not grad.any()


def test_two_stacks_at_once():
    """Steps on two streams, each with its own buffers, give what each gives alone."""
    T, H, F, E, k, V, L = 200, 256, 128, 8, 2, 3000, 2
    made = [model(T, H, F, E, V, L, seed=s) for s in (11, 12)]
    want, got = ([moe.StackBuffers(T, H, F, E, k, V, L) for _ in made] for _ in range(2))
    streams = [torch.cuda.Stream() for _ in made]
    for b, (x, layers, norm, wv, t, rw) in zip(want, made):
        moe.stack_step(b, x, layers, norm, wv, t, rw)
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s, (x, layers, norm, wv, t, rw) in zip(got, streams, made):
            moe.stack_step(b, x, layers, norm, wv, t, rw, s.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for name in ("loss", "lse", "dsum", "dwv", "dnorm"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        for p, q in zip(a.kept, b.kept):
            assert all(torch.equal(getattr(p, n), getattr(q, n)) for n in ("dnorm", "dwg", "dbg", "dw1", "dw2"))


def trained(seed=5):
    T, H, F, E, k, V, L = 120, 128, 64, 6, 2, 260, 2
    x, layers, norm, wv, t, rw = model(T, H, F, E, V, L, seed)
    b = moe.StackBuffers(T, H, F, E, k, V, L)
    master = [[w.float() if w.dtype == bf else w for w in layer] for layer in layers]
    head = wv.float()
    big = [(m[i], g, layer[i]) for m, layer, kept in zip(master, layers, b.kept)
           for i, g in ((1, kept.dwg), (3, kept.dw1), (4, kept.dw2))] + [(head, b.dwv, wv)]
    small = [(layer[i], g, None) for layer, kept in zip(layers, b.kept) for i, g in ((0, kept.dnorm), (2, kept.dbg))] + [(norm, b.dnorm, None)]
    opts = moe.Adamw(big, 8, lr=1e-3), moe.Adamw(small, 32, lr=1e-3, weight_decay=0.0)

    def step():
        moe.stack_step(b, x, layers, norm, wv, t, rw)
        for o in opts:
            o.step()

    def state():
        return [b.loss, b.dsum, wv, norm, head] + [w for layer in layers for w in layer] + [s for o in opts for st in o.states for s in st if s is not None]

    return step, state


def test_captured_steps_are_the_eager_ones():
    (eager, se), (graph, sg) = trained(), trained()
    for _ in range(2):
        eager()                               # what the capture runs first
    g = moe.capture(graph)
    for _ in range(3):
        eager()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(se(), sg()))


@pytest.mark.parametrize("mx", [True, False])
def test_scoring_of_a_few_tokens(mx):
    """Against fp64 on the same weights.  Activations are rounded to bf16 five times a layer and once in the head, 2^-9
    root mean square each; a logit of unit size moves by about 0.008, the loss by twice that: 0.08 is five times it."""
    T, H, F, E, k, V, L = 33, 128, 64, 8, 8, 900, 2
    x, layers, norm, wv, t, _ = model(T, H, F, E, V, L, seed=7)
    b = moe.TokenStackBuffers(T, H, F, E, k, V)
    served, exact = [], []
    for n, wg, bg, w1, w2 in layers:
        if mx:
            q1, q2 = mxa.quantize(w1)[:2], mxa.quantize(w2)[:2]
            served.append((n, wg, bg, q1, q2))
            exact.append((n, wg, bg, mxa.dequantize(*q1), mxa.dequantize(*q2)))
        else:
            served.append((n, wg, bg, w1, w2))
            exact.append((n, wg, bg, w1, w2))
    moe.token_stack_step(b, x, served, norm, wv, t)
    torch.cuda.synchronize()
    s = x.double()
    rms = lambda v, w: v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w.double()  # noqa: E731
    for n, wg, bg, w1, w2 in exact:
        y = rms(s, n)
        p, out = torch.softmax(y @ wg.double().t() + bg.double(), 1), 0
        for e in range(E):
            h = y @ w1[e].double().t()
            out = out + p[:, e:e + 1] * ((torch.nn.functional.silu(h[:, :F]) * h[:, F:]) @ w2[e].double().t())
        s = s + out
    z = rms(s, norm) @ wv.double().t()
    want = torch.where(t >= 0, torch.logsumexp(z, 1) - z.gather(1, t.long().clamp_min(0).unsqueeze(1)).squeeze(1), 0.0)
    assert (b.loss.double() - want).abs().max() < 0.08 and (b.lse.double() - torch.logsumexp(z, 1)).abs().max() < 0.08
    assert not b.loss[t < 0].any()


def test_layers_that_do_not_fit():
    b = moe.StackBuffers(32, 64, 32, 2, 1, 40, 2)
    with pytest.raises(ValueError, match="layers"):
        moe.stack_step(b, None, [()], None, None, None)


def test_what_a_layer_keeps():
    """Codes of 33 / 32 bytes an element for the tokens and the gate/up product; no rows of the down product."""
    T, H, F, E, k = 256, 512, 256, 4, 2
    kept = moe.LayerKept(T, H, F, E, k)
    cap = -(-(T * k + 31 * E) // 32) * 32
    size = lambda *ts: sum(t.numel() * t.element_size() for t in ts)  # noqa: E731
    assert size(kept.xq, kept.xs, kept.hq, kept.hs) == (T * H + cap * 2 * F) * 33 // 32
    assert size(kept.sum, kept.ids, kept.weights, kept.off, kept.dst, kept.src) == 2 * T * H + 4 * (3 * T * k + E + 1 + cap)
