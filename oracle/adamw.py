"""Oracle: the AdamW step with fp32 states or states in MX blocks.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Plain NumPy: fp64 for
the update, integers for the random bits.

The random bits of an element are a 32-bit mix of (seed, step, tensor index,
element); a state is rounded up when the fraction of its code step plus its 16
random bits reach 1.
"""

import numpy as np

from . import mxfp8

MASK = 0xFFFFFFFF
GOLD = 0x9E3779B1


def mix(x):
    """Bijective mix of 32-bit values (uint64 arrays)."""
    x = np.asarray(x, np.uint64) & MASK
    x ^= x >> np.uint64(16)
    x = x * np.uint64(0x6A09E667) & np.uint64(MASK)
    x ^= x >> np.uint64(15)
    x = x * np.uint64(0xBB67AE85) & np.uint64(MASK)
    return x ^ (x >> np.uint64(16))


def bits(seed, step, tensor, n):
    """The 32 random bits of each of n elements."""
    k = mix((seed & MASK) ^ GOLD)
    k = mix(k ^ np.uint64(seed >> 32))
    k = mix(k ^ np.uint64(step))
    k = mix(k ^ np.uint64(tensor))
    i = np.arange(n, dtype=np.uint64)
    return mix((k + i * np.uint64(GOLD)) & np.uint64(MASK))


def update(p, g, m, v, step, lr, scale, b1, b2, eps, wd):
    """One step in fp64: (p, m, v) and the magnitudes their fp32 roundings go by."""
    g = g * scale
    m2 = b1 * m + (1 - b1) * g
    v2 = b2 * v + (1 - b2) * g * g
    den = np.sqrt(v2 / (1 - b2 ** step)) + eps
    move = lr / (1 - b1 ** step) / den
    p2 = p * (1 - lr * wd) - move * m2
    mm = np.abs(b1 * m) + np.abs((1 - b1) * g)
    return (p2, m2, v2), (np.abs(p) * (1 + abs(lr * wd)) + move * mm, mm)


def scale_bytes(x):
    """Scale byte of each block of 32 (the last may be short): the smallest power of two with amax / 2^s <= 448."""
    x = np.abs(np.asarray(x, np.float64))
    b = np.zeros(-(-x.size // 32) * 32)
    b[:x.size] = np.where(np.isfinite(x), x, 0)
    top = b.reshape(-1, 32).max(1)
    mant, ex = np.frexp(top)                       # top = mant 2^ex, mant in [1/2, 1)
    e = np.where(top > 0, ex - 9 + (mant > 0.875), -127)
    return (np.clip(e, -127, 127) + 127).astype(np.uint8), top


def encode(x, u16, bytes_, root):
    """(codes, where the rounding is too near to call in fp32) of x in blocks with the given scale bytes."""
    n = x.size
    y = np.abs(x) / np.repeat(2.0 ** (bytes_.astype(np.float64) - 127), 32)[:n]
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -20))), -6) - 3)
    r = y / step + u16 / 65536.0
    val = np.floor(r) * step
    if root:
        val = np.where((x > 0) & (val == 0), 2.0 ** -9, val)
    codes = mxfp8.e4m3_encode(val) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return codes, np.abs(r - np.round(r)) < 2.0 ** -14


def decode(codes, bytes_):
    return mxfp8.e4m3_decode(codes) * np.repeat(2.0 ** (bytes_.astype(np.float64) - 127), 32)[:codes.size]


def round_bf16(x, u16):
    """bf16 bits of x rounded up in magnitude with probability the fraction, and where that is too near to call."""
    ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 7)
    r = np.abs(x) / ulp + u16 / 65536.0
    val = np.copysign(np.floor(r) * ulp, x)
    return mxfp8.f64_to_bf16(val), np.abs(r - np.round(r)) < 2.0 ** -12
