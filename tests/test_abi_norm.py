"""The norm's refusals, before any launch."""

import ctypes

import pytest

import mxfp8_block_scaled_07_amd as mxa
from test_abi import P, lib  # noqa: F401

BIG = 1 << 50
A8, A4, A2 = (ctypes.c_void_p(n) for n in (24, 20, 18))


def fwd(lib, x=P, res=P, dt=0, w=P, R=5, C=64, eps=1e-6, s=P, y=P, q=P, sc=P):  # noqa: F811
    return lib.mx_rmsnorm(x, res, dt, w, R, C, eps, s, y, q, sc, None)


def bwd(lib, dy=P, s=P, ds=P, dt=0, w=P, R=5, C=64, eps=1e-6, dres=P, dx=P, dw=P, ws=P, wsb=BIG):  # noqa: F811
    return lib.mx_rmsnorm_bwd(dy, s, ds, dt, w, R, C, eps, dres, dx, dw, ws, wsb, None)


BOTH = [dict(dt=2), dict(dt=-1), dict(R=-1), dict(C=0), dict(C=-32), dict(C=48), dict(eps=0.0), dict(eps=-1.0),
        dict(eps=float("nan")), dict(eps=float("inf")), dict(w=A2)]


@pytest.mark.parametrize("bad", BOTH + [dict(x=None, res=None), dict(q=None), dict(sc=None), dict(x=A8), dict(res=A8),
                                        dict(s=A8), dict(y=A8), dict(q=A4), dict(sc=A2),
                                        dict(s=None, y=None, q=None, sc=None)])
def test_forward_invalid(lib, bad):  # noqa: F811
    assert fwd(lib, **bad) == mxa.MX_EINVAL


@pytest.mark.parametrize("bad", BOTH + [dict(dy=None), dict(s=None), dict(dres=None, dx=None, dw=None), dict(dy=A8),
                                        dict(s=A8), dict(ds=A8), dict(dres=A8), dict(dx=A8), dict(dw=A2), dict(ws=A8),
                                        dict(ws=None), dict(wsb=0)])
def test_backward_invalid(lib, bad):  # noqa: F811
    assert bwd(lib, **bad) == mxa.MX_EINVAL


def test_sizes(lib):  # noqa: F811
    for f in (fwd, bwd):
        assert f(lib, C=65568) == mxa.MX_EUNSUPPORTED and f(lib, R=1 << 31) == mxa.MX_EUNSUPPORTED
    assert fwd(lib, R=0) == mxa.MX_OK and bwd(lib, R=0, dw=None) == mxa.MX_OK
    n = lib.mx_rmsnorm_bwd_workspace_size
    assert n(5, 64) % (4 * 64) == 0 and n(5, 64) > 0
    assert bwd(lib, wsb=n(5, 64) - 1) == mxa.MX_EINVAL
    for bad in ((0, 64), (-1, 64), (5, 0), (5, 48), (5, 65568), (1 << 31, 64)):
        assert n(*bad) == 0
