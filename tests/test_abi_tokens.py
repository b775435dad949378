"""The few-token layer's refusals, before any launch."""

import ctypes

import pytest

import mxfp8_block_scaled_07_amd as mxa
from test_abi import P, Q, lib  # noqa: F401

BIG = 1 << 40


def call(lib, T=4, k=2, E=8, H=64, F=32, x=P, logits=P, w1=P, s1=P, w2=P, s2=P, res=None, out=P, ws=P, wsb=BIG):  # noqa: F811
    a = lib.mx_moe_tokens(x, logits, T, k, E, H, F, w1, s1, w2, s2, res, out, ws, wsb, None)
    b = lib.mx_bf16_moe_tokens(x, logits, T, k, E, H, F, w1, w2, res, out, ws, wsb, None)
    return a, b


@pytest.mark.parametrize("bad", [dict(x=None), dict(logits=None), dict(w1=None), dict(w2=None), dict(out=None),
                                 dict(ws=None), dict(T=-1), dict(k=0), dict(E=0), dict(k=9), dict(H=48), dict(F=33),
                                 dict(H=0), dict(F=0), dict(x=Q), dict(w1=Q), dict(w2=Q), dict(ws=Q),
                                 dict(logits=ctypes.c_void_p(18)), dict(out=ctypes.c_void_p(17)),
                                 dict(res=ctypes.c_void_p(17)), dict(wsb=100)])
def test_invalid(lib, bad):  # noqa: F811
    assert call(lib, **bad) == (mxa.MX_EINVAL, mxa.MX_EINVAL)


def test_scales_are_needed(lib):  # noqa: F811
    assert call(lib, s1=None)[0] == mxa.MX_EINVAL and call(lib, s2=None)[0] == mxa.MX_EINVAL
    assert call(lib, s2=ctypes.c_void_p(18))[0] == mxa.MX_EINVAL


@pytest.mark.parametrize("big", [dict(T=65), dict(E=1025), dict(E=1024, k=65), dict(H=1 << 24), dict(F=1 << 24),
                                 dict(H=1 << 17, F=1 << 13)])
def test_unsupported(lib, big):  # noqa: F811
    assert call(lib, **big) == (mxa.MX_EUNSUPPORTED, mxa.MX_EUNSUPPORTED)


def test_sizes(lib):  # noqa: F811
    n = lib.mx_moe_tokens_workspace_size
    assert n(64, 8, 64, 2048) >= 64 * 8 * 2048 * 2
    assert n(65, 8, 64, 2048) == 0 and n(1, 65, 100, 32) == 0 and n(1, 0, 4, 32) == 0
    need = n(4, 2, 8, 32)
    assert call(lib, wsb=need - 1) == (mxa.MX_EINVAL, mxa.MX_EINVAL)
    assert call(lib, T=0, wsb=0) == (mxa.MX_OK, mxa.MX_OK)


def test_no_workspace_for_what_is_refused(lib):  # noqa: F811
    n = lib.mx_moe_tokens_workspace_size
    assert n(64, 8, 1024, 2048) > 0 and n(64, 4, 4, 2048) > 0
    assert n(64, 8, 1025, 2048) == 0 and n(64, 5, 4, 2048) == 0 and n(64, 2, 8, 1 << 24) == 0
    assert n(64, 2, 8, 33) == 0
    assert n(64, 64, 64, 1 << 18) == 0                  # w silu(g) u of 2^31 bytes
    assert call(lib, T=64, k=64, E=64, H=32, F=1 << 18) == (mxa.MX_EUNSUPPORTED, mxa.MX_EUNSUPPORTED)
