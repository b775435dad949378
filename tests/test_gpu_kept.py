"""GPU parity: the SwiGLU forward that keeps its input in MXFP8, the backward
from the kept codes, the router's backward from its dots, and the columnwise
requantize, against the oracle (oracle/kept.py, oracle/glue.py,
oracle/mxfp8.py).  MX bytes are those of the bf16 values that the calls on bf16
inputs write out, bit for bit; those values pass the glue's rule."""

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
import workloads
from mxfp8_block_scaled_07_amd import moe
from oracle import glue, kept, routing, tolerance
from oracle import mxfp8 as mx

from gpu_util import DEV, dev, host, spanels, srows

pytestmark = pytest.mark.gpu


def same_mx(vals, rq=None, rs=None, cq=None, cs=None):
    """MX bytes of bf16 values: mx_quantize's, and the oracle's where the values are finite (which it asks for)."""
    bits = host(vals)
    R, C = bits.shape
    finite = ((bits & 0x7F80) != 0x7F80).all()
    got = mxa.quantize(vals, rq is not None, cq is not None)
    torch.cuda.synchronize()
    if rq is not None:
        assert torch.equal(rq, got[0]) and torch.equal(rs, got[1])
        if finite:
            q, s = mx.quantize_rowwise(bits)
            assert np.array_equal(host(rq), q) and np.array_equal(srows(rs, C), s)
    if cq is not None:
        assert torch.equal(cq, got[2]) and torch.equal(cs, got[3])
        if finite:
            q, s = mx.quantize_colwise(bits)
            assert np.array_equal(host(cq), q) and np.array_equal(srows(cs, R), s)


def near(got, exact, S):
    """The glue's rule; values of at least (2 - 2^-8) 2^127 round to infinity in bf16, which the rule, made for finite
    results, would call infinitely far off."""
    bits, over = host(got), np.abs(exact) >= (2 - 2.0 ** -8) * 2.0 ** 127
    assert np.array_equal(bits[over], np.where(exact[over] > 0, 0x7F80, 0xFF80))
    res = tolerance.check_bf16_elementwise(bits[~over], exact[~over], S[~over])
    assert res["ok"], res


def h_input(g, rows, F, pad=()):
    h = workloads.normal_bf16(g, (rows, 2 * F), 2.0, outlier_p=0.002)
    special = mx.f64_to_bf16(np.array([-1e30, 1e30, -200.0, 200.0, 1e-40, -1e-40, 0.0, -0.0, -1.2785]))
    h.ravel()[g.integers(0, h.size, special.size * 4)] = np.tile(special, 4)
    h[list(pad)] = 0
    return h


# whole tiles; ragged rows; F with panels that the two halves share, one block, one tile, several
SIZES = [(256, 128), (224, 96), (32, 32), (1056, 160), (96, 2048), (64, 1408), (160, 224), (128, 64)]


@pytest.mark.parametrize("rows,F", SIZES + [(1, 32), (77, 96), (131, 288)])
def test_keep(rows, F):
    g = np.random.default_rng([rows, F])
    h = h_input(g, rows, F, range(rows - rows // 8, rows))
    hd = dev(h)
    rq, rs, kq, ks = (torch.full(s, 0x55, dtype=torch.uint8, device=DEV) for s in (
        (rows + 1, F), mxa.scale_shape(rows, F), (rows + 1, 2 * F), mxa.scale_shape(rows, 2 * F)))
    mxa.mx_swiglu_keep(hd, rows, F, rq, rs, kq, ks)
    a, _, _, _, _ = mxa.swiglu_quantize(hd, colwise=False, want_bf16=True)
    torch.cuda.synchronize()
    near(a, *glue.swiglu(h, F))
    same_mx(a, rq[:rows], rs)
    same_mx(hd, kq[:rows], ks)
    assert (rq[rows] == 0x55).all() and (kq[rows] == 0x55).all()


def kept_input(rows, F, seed=0):
    g = np.random.default_rng([seed, rows, F])
    q, s = mx.quantize_rowwise(h_input(g, rows, F, range(rows - rows // 8, rows)))
    da = workloads.normal_bf16(g, (rows, F), 0.1, 0.002)
    da[rows - rows // 8:] = 0
    return q, s, da


def check_bwd(rows, F, colwise):
    q, s, da = kept_input(rows, F)
    kq, ks, dd = dev(q), dev(spanels(s)), dev(da).view(torch.bfloat16)
    guard = lambda *sh: torch.full(sh, 0x55, dtype=torch.uint8, device=DEV)  # noqa: E731
    row = guard(rows + 1, 2 * F), guard(*mxa.scale_shape(rows, 2 * F))
    col = (guard(2 * F + 1, rows), guard(*mxa.scale_shape(2 * F, rows))) if colwise else (None, None)
    a = (guard(F + 1, rows), guard(*mxa.scale_shape(F, rows))) if colwise else (None, None)
    dots = torch.full((rows + 1,), 7.0, device=DEV)
    wsb = mxa.mx_swiglu_bwd_kept_workspace_size(rows, F)
    ws = torch.full((wsb + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    mxa.mx_swiglu_bwd_kept(kq, ks, dd, rows, F, *row, *col, *a, dots, ws, wsb)
    # the calls on bf16 inputs write their bf16 values out
    hb = mx.dequantize(q, s)
    hd = dev(hb)
    dh, _, _, _, _ = mxa.swiglu_bwd_quantize(hd, dev(da), colwise=False, want_bf16=True)
    ab, _, _, _, _ = mxa.swiglu_quantize(hd, colwise=False, want_bf16=True)
    torch.cuda.synchronize()
    near(dh, *glue.swiglu_bwd(hb, da, F))
    near(ab, *glue.swiglu(hb, F))
    same_mx(dh, row[0][:rows], row[1])
    want, bound = kept.dots(hb, da, F)
    # (a row with a term that fp32 cannot hold, or that with others may sum past it, is not finite)
    a64, _ = glue.swiglu(hb, F)
    held = np.abs(a64).max(1) < 2.0 ** 127
    held &= np.abs(a64 * mx.bf16_to_f64(da)).sum(1) < 2.0 ** 127
    err = np.abs(host(dots)[:rows] - want)[held]
    print("dots max err/bound", float((err / bound[held]).max(initial=0)), "rows", int(held.sum()), flush=True)
    assert (err <= bound[held]).all() and held.sum() > rows // 2 - 1 and dots[rows] == 7 and (ws[wsb:] == 0xFF).all() and (row[0][rows] == 0x55).all()
    if colwise:
        same_mx(dh, cq=col[0][:2 * F], cs=col[1])
        same_mx(ab, cq=a[0][:F], cs=a[1])
        assert (col[0][2 * F] == 0x55).all() and (a[0][F] == 0x55).all()
    # each output by itself
    one = mxa.swiglu_bwd_kept(kq, ks, dd, True, False, False, False)[:2]
    assert torch.equal(one[0], row[0][:rows]) and torch.equal(one[1], row[1])
    assert torch.equal(mxa.swiglu_bwd_kept(kq, ks, dd, False, False, False)[6], dots[:rows])
    if colwise:
        one = mxa.swiglu_bwd_kept(kq, ks, dd, False, True, False, False)[2:4]
        assert torch.equal(one[0], col[0][:2 * F]) and torch.equal(one[1], col[1])
        one = mxa.swiglu_bwd_kept(kq, ks, dd, False, False, True, False)[4:6]
        assert torch.equal(one[0], a[0][:F]) and torch.equal(one[1], a[1])


@pytest.mark.parametrize("rows,F", SIZES)
def test_backward(rows, F):
    check_bwd(rows, F, True)


@pytest.mark.parametrize("rows,F", [(1, 32), (77, 96), (131, 288), (5, 1408)])
def test_backward_of_odd_rows(rows, F):
    check_bwd(rows, F, False)


def test_nan_scales_and_codes():
    """A block of scale 255 and a NaN code decode as mx_dequantize decodes them; other blocks' bytes do not change."""
    q, s, da = kept_input(64, 96)
    clean = mxa.swiglu_bwd_kept(dev(q), dev(spanels(s)), dev(da).view(torch.bfloat16))
    s[3, 1], q[9, 40] = 255, 0x7F
    kq, ks, dd = dev(q), dev(spanels(s)), dev(da).view(torch.bfloat16)
    hd = mxa.dequantize(kq, ks)
    got = mxa.swiglu_bwd_kept(kq, ks, dd)
    want = mxa.swiglu_bwd_quantize(hd, dd)[1:] + mxa.swiglu_quantize(hd, rowwise=False)[3:]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:6], want))
    rows = [r for r in range(64) if r not in (3, 9)]
    assert torch.equal(got[0][rows], clean[0][rows]) and torch.equal(got[6][rows], clean[6][rows])
    assert torch.isnan(got[6][3]) and torch.isnan(got[6][9])


@pytest.mark.parametrize("rows,cols,out", [(100, 64, None), (64, 160, 128), (33, 352, None), (300, 1024, 416), (1, 32, 32)])
@pytest.mark.parametrize("gathered", [True, False])
def test_requantize(rows, cols, out, gathered):
    g = np.random.default_rng([rows, cols])
    x = workloads.normal_bf16(g, (rows, cols), 1.0, 0.01)
    q, s = mx.quantize_rowwise(x)
    out = -(-rows // 32) * 32 if out is None else out
    idx = None
    if gathered:
        idx = g.integers(0, rows, out)
        idx[::7], idx[3::11] = -1, rows + 5
    cq = torch.full((cols + 1, out), 0x55, dtype=torch.uint8, device=DEV)
    cs = torch.full(mxa.scale_shape(cols, out), 0x55, dtype=torch.uint8, device=DEV)
    mxa.mx_requantize(dev(q), dev(spanels(s)), rows, cols, None if idx is None else dev(idx), out, cq, cs)
    torch.cuda.synchronize()
    if idx is not None:
        idx = np.where(idx >= rows, -1, idx)
    wq, wsc = mx.quantize_colwise(mx.dequantize(q, s), rows_out=out, gather=idx)
    assert np.array_equal(host(cq[:cols]), wq) and np.array_equal(srows(cs, out), wsc) and (cq[cols] == 0x55).all()
    one = mxa.requantize(dev(q), dev(spanels(s)), out, None if idx is None else dev(idx))
    torch.cuda.synchronize()
    assert torch.equal(one[0], cq[:cols]) and torch.equal(one[1], cs)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 3), (130, 64, 8), (9, 100, 64), (40, 1000, 7)])
def test_router(T, E, k):
    g = np.random.default_rng([T, E, k])
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    if T > 4:
        ids[2] = ids[2, 0]                                # a repeated expert adds its terms
        ids[3, 0] = E + 3                                 # no such expert: no entry
    rows = T * k + 17
    dst = g.permutation(rows)[:T * k]
    if T > 4:
        dst[::5], dst[1::9] = -1, rows + 2
    w = g.random((T, k)).astype(np.float32)
    w /= w.sum(1, keepdims=True)
    dot = g.standard_normal(rows).astype(np.float32)
    dl = torch.full((T + 1, E), 7.0, device=DEV)
    mxa.mx_router_bwd_dots(dev(dot), rows, dev(dst.astype(np.int32)), dev(ids.astype(np.int32)), dev(w), T, E, k, dl)
    torch.cuda.synchronize()
    padded = np.where(ids < E, ids, E)
    want, bound = kept.dlogits(dot, dst, padded, w, E + 1)
    off = np.abs(host(dl)[:T] - want[:, :E]) > bound[:, :E]
    assert not off.any() and (dl[T] == 7).all(), np.argwhere(off)[:5]
    one = mxa.router_bwd_dots(dev(dot), dev(dst.astype(np.int32)), dev(ids.astype(np.int32)), dev(w), E)
    torch.cuda.synchronize()
    assert torch.equal(one, dl[:T])


def test_router_of_no_rows():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
    f = torch.float32
    assert (mxa.router_bwd_dots(z(0, dt=f), z(6) - 1, z(3, 2), z(3, 2, dt=f), 4) == 0).all()
    assert mxa.router_bwd_dots(z(4, dt=f), z(0), z(0, 2), z(0, 2, dt=f), 4).shape == (0, 4)


def test_graph_and_streams():
    """A captured chain of keep, backward and requantize replays to the eager bytes; another stream gives them too."""
    T, E, k, F, H = 90, 6, 2, 160, 96
    g = np.random.default_rng(4)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    cap = workloads.capacity(T, k, E)
    _, _, dst, src = routing.route(ids, E, cap)
    h = h_input(g, cap, F)
    h[src < 0] = 0
    q, s = mx.quantize_rowwise(workloads.normal_bf16(g, (T, H), 1.0))
    w = g.random((T, k)).astype(np.float32)
    hd, da = dev(h), dev(workloads.normal_bf16(g, (cap, F), 0.1)).view(torch.bfloat16)
    xq, xs, dstd, srcd, idd, wd = dev(q), dev(spanels(s)), dev(dst), dev(src), dev(ids), dev(w)
    u8 = lambda *sh: torch.zeros(sh, dtype=torch.uint8, device=DEV)  # noqa: E731
    pair = lambda r, c: (u8(r, c), u8(*mxa.scale_shape(r, c)))  # noqa: E731
    wsb = mxa.mx_swiglu_bwd_kept_workspace_size(cap, F)

    def buffers():
        return (*pair(cap, F), *pair(cap, 2 * F), *pair(cap, 2 * F), *pair(2 * F, cap), *pair(F, cap), *pair(H, cap),
                torch.zeros(cap, device=DEV), torch.zeros(T, E, device=DEV), u8(wsb))

    def chain(b, stream=None):
        mxa.mx_swiglu_keep(hd, cap, F, *b[:4], stream)
        mxa.mx_swiglu_bwd_kept(b[2], b[3], da, cap, F, *b[4:10], b[12], b[14], wsb, stream)
        mxa.mx_router_bwd_dots(b[12], cap, dstd, idd, wd, T, E, k, b[13], stream)
        mxa.mx_requantize(xq, xs, T, H, srcd, cap, b[10], b[11], stream)

    want, got = buffers(), buffers()
    chain(want)
    graph = moe.capture(lambda: chain(got))
    for _ in range(3):
        for t in got:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        chain(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    st, other = torch.cuda.Stream(), buffers()
    torch.cuda.synchronize()
    chain(other, st.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))


def test_codes_past_32_bits():
    """Rows whose codes lie past 2^32 bytes give what they give by themselves."""
    F = 4096
    rows = (1 << 32) // (2 * F) + 64
    q, s, da = kept_input(64, F)
    s[:] = np.where((q.reshape(64, -1, 32) & 0x7F).max(2) > 0, s, 0)
    kq, ks = torch.zeros(rows, 2 * F, dtype=torch.uint8, device=DEV), torch.zeros(mxa.scale_shape(rows, 2 * F), dtype=torch.uint8, device=DEV)
    dd = torch.zeros(rows, F, dtype=torch.bfloat16, device=DEV)
    kq[-64:], ks[:, -64:], dd[-64:] = dev(q), dev(spanels(s)), dev(da).view(torch.bfloat16)
    got = mxa.swiglu_bwd_kept(kq, ks, dd)
    one = mxa.swiglu_bwd_kept(dev(q), dev(spanels(s)), dev(da).view(torch.bfloat16))
    torch.cuda.synchronize()
    assert torch.equal(got[0][-64:], one[0]) and torch.equal(got[1][:, -64:], one[1]) and torch.equal(got[6][-64:], one[6])
    assert torch.equal(got[2][:, -64:], one[2]) and torch.equal(got[4][:, -64:], one[4])
    assert not got[0][:-64].any() and not got[6][:-64].any()
    del got
    rq, rs = mxa.swiglu_keep(mxa.dequantize(kq, ks))[2:]
    torch.cuda.synchronize()
    assert torch.equal(rq[-64:], mxa.swiglu_keep(mxa.dequantize(dev(q), dev(spanels(s))))[2]) and not rq[:-64].any()


@pytest.mark.parametrize("rows,F", [(4001, 160), (2100, 1056), (2085, 256)])
def test_keep_of_many_workgroups(rows, F):
    """More than one run of 256 workgroups, the last one partial; panels of both halves, and of one."""
    assert rows * F // 8 > 256 * 256 and rows * F // 8 % (256 * 256)
    g = np.random.default_rng([rows, F])
    hd = dev(h_input(g, rows, F, range(rows - rows // 8, rows)))
    guard = lambda *sh: torch.full(sh, 0x55, dtype=torch.uint8, device=DEV)  # noqa: E731
    rq, rs, kq, ks = guard(rows + 1, F), guard(*mxa.scale_shape(rows, F)), guard(rows + 1, 2 * F), guard(*mxa.scale_shape(rows, 2 * F))
    mxa.mx_swiglu_keep(hd, rows, F, rq, rs, kq, ks)
    a = mxa.swiglu_quantize(hd, colwise=False, want_bf16=True)[0]
    torch.cuda.synchronize()
    same_mx(a, rq[:rows], rs)
    same_mx(hd, kq[:rows], ks)
    assert (rq[rows] == 0x55).all() and (kq[rows] == 0x55).all()


# four column tiles to a workgroup (from 4096 tiles on): a last group of two, one, four and three, the last column tile
# partial or whole, the last row tile partial
@pytest.mark.parametrize("rows,cols,out", [(3000, 672, 90016), (2000, 640, 105056), (90000, 928, 66016), (7, 352, 175040)])
@pytest.mark.parametrize("gathered", [True, False])
def test_requantize_of_many_tiles(rows, cols, out, gathered):
    assert -(-out // 128) * -(-cols // 128) >= 4096
    if not gathered:
        rows = out - 40 if cols != 640 else out     # (rows past the last are zeros)
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x = torch.randn(rows, cols, device=DEV, generator=g).mul_(torch.randn(rows, cols // 32, device=DEV, generator=g)
                                                              .exp_().repeat_interleave(32, 1)).to(torch.bfloat16)
    q, s = mxa.quantize(x)[:2]
    q[5, 40], q[rows - 1, cols - 1] = 0x7F, 0xFF                              # NaN codes
    s[(cols - 1) // 128, 3, (cols // 32 - 1) % 4] = 255                       # a block of NaN: the last of row 3
    idx = None
    if gathered:
        idx = torch.randint(0, rows, (out,), device=DEV, generator=g, dtype=torch.int32)
        idx[::7], idx[3::11], idx[-1] = -1, rows + 5, rows - 1
    cq = torch.full((cols + 1, out), 0x55, dtype=torch.uint8, device=DEV)
    cs = torch.full(mxa.scale_shape(cols, out), 0x55, dtype=torch.uint8, device=DEV)
    mxa.mx_requantize(q, s, rows, cols, idx, out, cq, cs)
    want = mxa.quantize(mxa.dequantize(q, s), False, True, out, idx)[2:]
    torch.cuda.synchronize()
    assert torch.equal(cq[:cols], want[0]) and torch.equal(cs, want[1]) and (cq[cols] == 0x55).all()
    # a sample of columns against the oracle, where no NaN is near
    clean = mxa.quantize(x)[:2]
    mxa.mx_requantize(*clean, rows, cols, idx, out, cq, cs)
    torch.cuda.synchronize()
    at = np.unique([0, 31, 32, 127, 128, 200, 257, cols - 33, cols - 1])
    d = host(mxa.dequantize(*clean)[:, torch.from_numpy(at).to(DEV)].contiguous())
    i = None if idx is None else np.where(host(idx) >= rows, -1, host(idx))
    wq, wsc = mx.quantize_colwise(d, rows_out=out, gather=i)
    assert np.array_equal(host(cq)[at], wq) and np.array_equal(srows(cs, out)[at], wsc)
