"""Pins of the AdamW oracle: torch.optim.AdamW in fp64, the random bits, and the state format."""

import numpy as np
import torch

from oracle import adamw, mxfp8


def test_update_is_torchs():
    g = np.random.default_rng(0)
    p = torch.tensor(g.standard_normal(50), requires_grad=True)
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.3)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        grad = g.standard_normal(50)
        p.grad = torch.tensor(grad * 0.25)
        opt.step()
        (q, m, v), _ = adamw.update(q, grad, m, v, t, 0.01, 0.25, 0.8, 0.95, 1e-6, 0.3)
        assert np.allclose(p.detach().numpy(), q, rtol=1e-13, atol=1e-15)


def test_bits_are_uniform_and_differ():
    n = 1 << 18
    h = adamw.bits(1234567890123, 7, 3, n)
    for half in (h >> np.uint64(16), h & np.uint64(0xFFFF)):
        u = half.astype(np.float64) / 65536
        # mean and spread of n uniform values, each within 6 of its standard deviations
        assert abs(u.mean() - 0.5) < 6 * (1 / 12 / n) ** 0.5
        assert abs(u.var() - 1 / 12) < 6 * (1 / 180 / n) ** 0.5
        assert abs(np.mean((u[1:] - 0.5) * (u[:-1] - 0.5))) < 6 / 12 / n ** 0.5
    hi, lo = (h >> np.uint64(16)).astype(float), (h & np.uint64(0xFFFF)).astype(float)
    assert abs(np.corrcoef(hi, lo)[0, 1]) < 6 / n ** 0.5
    assert len(np.unique(adamw.mix(np.arange(1 << 16)))) == 1 << 16
    for other in (adamw.bits(1234567890124, 7, 3, n), adamw.bits(1234567890123, 8, 3, n),
                  adamw.bits(1234567890123, 7, 4, n), adamw.bits(1234567890123 + (1 << 40), 7, 3, n)):
        assert np.mean(other == h) < 1e-3


def test_state_format():
    x = np.zeros(40)
    x[:4] = [1.75, -0.5, 2.0 ** -9 * 2.0 ** -8, 3e-9]
    x[33] = -1.7500001
    b, top = adamw.scale_bytes(x)
    assert b.tolist() == [127 - 8, 127 - 7] and top.tolist() == [1.75, 1.7500001]
    codes, _ = adamw.encode(x, np.zeros(40), b, False)
    assert mxfp8.e4m3_decode(codes)[:4].tolist() == [448.0, -128.0, 2.0 ** -9, 0.0]
    codes, _ = adamw.encode(np.abs(x), np.zeros(40), b, True)
    assert mxfp8.e4m3_decode(codes)[3] == 2.0 ** -9      # a positive root is never zero
    up, _ = adamw.encode(x, np.full(40, 65535.0), b, False)
    assert mxfp8.e4m3_decode(up)[0] == 448.0             # representable values stay
    bits, _ = adamw.round_bf16(np.array([1.0, 1.0 + 2.0 ** -8, -3.0]), np.array([65535, 32768, 0]))
    assert mxfp8.bf16_to_f64(bits).tolist() == [1.0, 1.0 + 2.0 ** -7, -3.0]
