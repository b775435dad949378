"""The dense product's refusals, before any launch."""

import ctypes

import pytest

import mxfp8_block_scaled_07_amd as mxa
from test_abi import P, Q, lib  # noqa: F401

BIG = 1 << 50


def fwd(lib, x=P, w=P, bias=None, res=None, M=100, n=64, k=64, act=0, z=None, out=P, dt=0, ws=P, wsb=BIG):  # noqa: F811
    return lib.mx_bf16_linear(x, w, bias, res, M, n, k, act, z, out, dt, ws, wsb, None)


def bwd(lib, dout=P, dt=0, z=P, x=P, w=P, add=None, M=100, n=64, k=64, act=1, dx=P, dw=P, db=P, ws=P, wsb=BIG):  # noqa: F811
    return lib.mx_bf16_linear_bwd(dout, dt, z, x, w, add, M, n, k, act, dx, dw, db, ws, wsb, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(out=None), dict(M=-1), dict(n=0), dict(k=0),
                                 dict(k=40), dict(act=5), dict(act=-1), dict(dt=2), dict(x=Q), dict(w=Q), dict(out=Q),
                                 dict(res=Q), dict(z=Q), dict(ws=Q), dict(bias=ctypes.c_void_p(18))])
def test_forward_invalid(lib, bad):  # noqa: F811
    assert fwd(lib, **bad) == mxa.MX_EINVAL


@pytest.mark.parametrize("bad", [dict(dout=None), dict(z=None), dict(x=None), dict(w=None), dict(M=-1), dict(n=0),
                                 dict(k=33), dict(act=5), dict(dt=7), dict(dout=Q), dict(z=Q), dict(x=Q), dict(w=Q),
                                 dict(add=Q), dict(dx=Q), dict(dw=Q), dict(db=ctypes.c_void_p(18)), dict(ws=Q),
                                 dict(ws=None), dict(wsb=10), dict(dx=None, dw=None, db=None), dict(dx=None, add=P)])
def test_backward_invalid(lib, bad):  # noqa: F811
    assert bwd(lib, **bad) == mxa.MX_EINVAL


def test_sizes(lib):  # noqa: F811
    for f in (fwd, bwd):
        assert f(lib, n=1 << 21) == mxa.MX_EUNSUPPORTED and f(lib, k=1 << 21) == mxa.MX_EUNSUPPORTED
        assert f(lib, M=1 << 31) == mxa.MX_EUNSUPPORTED
    assert fwd(lib, M=0) == mxa.MX_OK
    s = lib.mx_bf16_linear_workspace_size
    assert s(8, 64, 4096) == 0                        # streamed: no workspace
    need = s(100, 64, 8192)
    assert need >= 2 * 100 * 64 * 4                   # split
    assert fwd(lib, k=8192, wsb=need - 1) == mxa.MX_EINVAL and fwd(lib, k=8192, ws=None) == mxa.MX_EINVAL
    b = lib.mx_bf16_linear_bwd_workspace_size
    assert b(100, 64, 64, 1) >= 100 * 64 * 2 and b(0, 64, 64, 1) == 0 and b(100, 64, 64, 9) == 0


def test_a_launch_holds_its_threads(lib):  # noqa: F811
    assert fwd(lib, M=1 << 30, n=1 << 20, k=128) == mxa.MX_EUNSUPPORTED
    assert bwd(lib, M=1 << 30, n=1 << 10, k=1 << 16) == mxa.MX_EUNSUPPORTED
