"""The cross entropy's refusals, before any launch."""

import ctypes

import pytest

import mxfp8_block_scaled_07_amd as mxa
from test_abi import P, lib  # noqa: F401

BIG = 1 << 50
A8, A2 = ctypes.c_void_p(24), ctypes.c_void_p(18)


def xent(lib, x=P, w=P, t=P, rw=P, M=100, V=1000, k=64, loss=P, lse=P, dx=P, dw=P, ws=P, wsb=BIG):  # noqa: F811
    return lib.mx_bf16_xent(x, w, t, rw, M, V, k, loss, lse, dx, dw, ws, wsb, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(t=None), dict(M=-1), dict(V=0), dict(V=-1), dict(k=0), dict(k=40),
                                 dict(loss=None, lse=None, dx=None, dw=None), dict(x=A8), dict(w=A8), dict(dx=A8), dict(dw=A8),
                                 dict(ws=A8), dict(t=A2), dict(rw=A2), dict(loss=A2), dict(lse=A2), dict(ws=None), dict(wsb=100),
                                 dict(dx=None, dw=None, wsb=100)])
def test_invalid(lib, bad):  # noqa: F811
    assert xent(lib, **bad) == mxa.MX_EINVAL


def test_sizes(lib):  # noqa: F811
    for bad in (dict(V=1 << 21), dict(k=1 << 21), dict(M=1 << 31)):
        assert xent(lib, **bad) == mxa.MX_EUNSUPPORTED
    assert xent(lib, M=0, dw=None, ws=None, wsb=0) == mxa.MX_OK
    n = lib.mx_bf16_xent_workspace_size
    for back in (0, 1):
        need = n(100, 1000, 64, back)
        assert need > 0
        kw = {} if back else dict(dx=None, dw=None)
        assert xent(lib, wsb=need - 1, **kw) == mxa.MX_EINVAL
        for bad in ((0, 1000, 64), (-1, 1000, 64), (100, 0, 64), (100, 1000, 0), (100, 1000, 40), (100, 1 << 21, 64),
                    (100, 1000, 1 << 21), (1 << 31, 1000, 64)):
            assert n(*bad, back) == 0


def test_the_workspace_is_bounded(lib):  # noqa: F811
    """Not by the logits: by a chunk of rows of them in two bytes, and dw's sum where there are several chunks."""
    n = lib.mx_bf16_xent_workspace_size
    V, k = 131072, 5120
    assert n(1 << 20, V, k, 1) < 4 * V * k + 3.2 * 2 ** 30
    assert n(4096, V, k, 1) < 2 * 4096 * V + 0.3 * 2 ** 30
    assert n(1 << 20, V, k, 0) < 2.1 * 2 ** 30
    assert n(1 << 30, 8, 32, 1) < 8.5 * 2 ** 30
