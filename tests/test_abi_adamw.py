"""The AdamW step's refusals, before any launch."""

import ctypes

import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
from test_abi import P, Q, lib  # noqa: F401


def call(lib, n=64, count=1, pd=1, gd=1, bits=32, lr=P, step=P, scale=None, b1=0.9, b2=0.999, eps=1e-8, wd=0.1, **t):  # noqa: F811
    f = dict(param=16, grad=16, m=16, v=16, m_scale=16, v_scale=16, copy=None, n=n)
    f.update(t)
    table = (mxa.AdamwTensor * 1)(mxa.AdamwTensor(**f))
    return lib.mx_adamw(table, count, pd, gd, bits, lr, step, scale, b1, b2, eps, wd, 5, None)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(param=None), dict(grad=None), dict(m=None), dict(v=None),
                                 dict(bits=8, m_scale=None), dict(bits=8, v_scale=None), dict(param=8), dict(grad=24),
                                 dict(m=8), dict(v=8), dict(copy=8), dict(pd=2), dict(gd=-1), dict(bits=16),
                                 dict(lr=None), dict(step=None), dict(lr=ctypes.c_void_p(18)), dict(b1=1.0),
                                 dict(b1=-0.1), dict(b2=float("nan")), dict(eps=-1e-9), dict(wd=float("inf")),
                                 dict(count=-1)])
def test_invalid(lib, bad):  # noqa: F811
    assert call(lib, **bad) == mxa.MX_EINVAL


def test_nothing_to_do_and_too_much(lib):  # noqa: F811
    assert call(lib, n=0) == mxa.MX_OK and call(lib, count=0) == mxa.MX_OK
    assert lib.mx_adamw(None, 0, 1, 1, 32, P, P, None, 0.9, 0.9, 0.0, 0.0, 0, None) == mxa.MX_OK
    assert lib.mx_adamw(None, 1, 1, 1, 32, P, P, None, 0.9, 0.9, 0.0, 0.0, 0, None) == mxa.MX_EINVAL
    assert call(lib, n=1 << 41) == mxa.MX_EUNSUPPORTED


def test_one_launch_holds_its_threads(lib):  # noqa: F811
    """48 tensors in turn with 2^34 elements or more are refused before the first of them is updated."""
    assert call(lib, n=1 << 34) == mxa.MX_EUNSUPPORTED
    row = mxa.AdamwTensor(param=16, grad=16, m=16, v=16, n=1 << 33)
    rows = [mxa.AdamwTensor(param=16, grad=16, m=16, v=16, n=0)] * 48 + [row, row]
    table = (mxa.AdamwTensor * 50)(*rows)
    assert lib.mx_adamw(table, 50, 1, 1, 32, P, P, None, 0.9, 0.9, 0.0, 0.0, 0, None) == mxa.MX_EUNSUPPORTED


def test_table():
    p = torch.zeros(40)
    t = mxa.adamw_table([(p, p.clone(), p.clone(), p.clone(), torch.zeros(2, dtype=torch.uint8), None, None)])
    assert t[0].n == 40 and t[0].param == p.data_ptr() and t[0].v_scale is None
    with pytest.raises(ValueError):
        mxa.adamw_table([(p, torch.zeros(39), p, p, None, None, None)])
    with pytest.raises(ValueError):
        mxa.adamw_table([(torch.zeros(8, 5).t(), p, p, p, None, None, None)])
