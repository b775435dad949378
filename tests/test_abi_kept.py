"""The refusals of the kept activations' calls, before any launch."""

import ctypes

import pytest

import mxfp8_block_scaled_07_amd as mxa
from test_abi import P, lib  # noqa: F401

BIG = 1 << 50
A8, A4, A2 = (ctypes.c_void_p(n) for n in (24, 20, 18))


def keep(lib, h=P, R=64, F=96, q=P, s=P, kq=P, ks=P):  # noqa: F811
    return lib.mx_swiglu_keep(h, R, F, q, s, kq, ks, None)


def bwd(lib, kq=P, ks=P, da=P, R=64, F=160, q=P, s=P, cq=P, cs=P, aq=P, as_=P, dots=P, ws=P, wsb=BIG):  # noqa: F811
    return lib.mx_swiglu_bwd_kept(kq, ks, da, R, F, q, s, cq, cs, aq, as_, dots, ws, wsb, None)


def router(lib, dots=P, R=64, dst=P, ids=P, w=P, T=5, E=8, k=2, dl=P):  # noqa: F811
    return lib.mx_router_bwd_dots(dots, R, dst, ids, w, T, E, k, dl, None)


def requant(lib, q=P, s=P, R=5, C=64, g=None, out=64, cq=P, cs=P):  # noqa: F811
    return lib.mx_requantize(q, s, R, C, g, out, cq, cs, None)


@pytest.mark.parametrize("bad", [dict(h=None), dict(q=None), dict(s=None), dict(kq=None), dict(ks=None), dict(R=-1), dict(F=0),
                                 dict(F=40), dict(F=-32), dict(h=A8), dict(q=A4), dict(kq=A4), dict(s=A2), dict(ks=A2)])
def test_keep_invalid(lib, bad):  # noqa: F811
    assert keep(lib, **bad) == mxa.MX_EINVAL


@pytest.mark.parametrize("bad", [dict(kq=None), dict(ks=None), dict(da=None), dict(R=-1), dict(F=0), dict(F=40), dict(R=40),
                                 dict(R=40, cq=None, cs=None), dict(q=None), dict(s=None), dict(cq=None), dict(cs=None),
                                 dict(aq=None), dict(as_=None), dict(kq=A4), dict(ks=A2), dict(da=A8), dict(q=A4), dict(s=A2),
                                 dict(cq=A8), dict(cs=A2), dict(aq=A8), dict(as_=A2), dict(dots=A2), dict(ws=A8), dict(ws=None),
                                 dict(wsb=64 * 2 * 4 - 1),
                                 dict(q=None, s=None, cq=None, cs=None, aq=None, as_=None, dots=None)])
def test_backward_invalid(lib, bad):  # noqa: F811
    assert bwd(lib, **bad) == mxa.MX_EINVAL


@pytest.mark.parametrize("bad", [dict(dots=None), dict(dst=None), dict(ids=None), dict(w=None), dict(dl=None), dict(R=-1),
                                 dict(T=-1), dict(E=0), dict(k=0), dict(k=65)])
def test_router_invalid(lib, bad):  # noqa: F811
    assert router(lib, **bad) == mxa.MX_EINVAL


@pytest.mark.parametrize("bad", [dict(q=None), dict(s=None), dict(cq=None), dict(cs=None), dict(R=-1), dict(C=0), dict(C=40),
                                 dict(out=-32), dict(out=40), dict(q=A4), dict(s=A2), dict(cq=A8), dict(cs=A2), dict(g=A2)])
def test_requantize_invalid(lib, bad):  # noqa: F811
    assert requant(lib, **bad) == mxa.MX_EINVAL


def test_sizes(lib):  # noqa: F811
    assert keep(lib, R=0) == mxa.MX_OK and bwd(lib, R=0) == mxa.MX_OK and router(lib, T=0) == mxa.MX_OK
    assert requant(lib, out=0) == mxa.MX_OK
    n = lib.mx_swiglu_bwd_kept_workspace_size
    assert n(64, 128) == 0 and n(64, 160) == 64 * 2 * 4 and n(64, 1408) == 64 * 11 * 4
    for bad in ((0, 160), (-1, 160), (64, 0), (64, 40), (64, (1 << 22) + 32)):
        assert n(*bad) == 0
    assert bwd(lib, F=(1 << 22) + 32) == mxa.MX_EUNSUPPORTED and keep(lib, F=(1 << 22) + 32) == mxa.MX_EUNSUPPORTED
    assert keep(lib, R=1 << 28, F=128) == mxa.MX_EUNSUPPORTED and keep(lib, R=1 << 62, F=32) == mxa.MX_EUNSUPPORTED
