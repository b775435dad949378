"""The allocating helpers of the few-token layer, the dense product and AdamW refuse arguments that do not fit, before
any call (on the CPU)."""

import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa
from mxfp8_block_scaled_07_amd import moe

bf, u8 = torch.bfloat16, torch.uint8


def tokens(x=None, logits=None, w1=None, w2=None, res=None):
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    return mxa.moe_tokens(z(3, 64) if x is None else x, z(3, 4, dt=torch.float32) if logits is None else logits, 2,
                          z(4, 64, 64) if w1 is None else w1, z(4, 64, 32) if w2 is None else w2, res)


def test_moe_tokens():
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    for bad in (dict(x=z(3, 64, dt=torch.float32)), dict(x=z(64, 3).t()), dict(logits=z(3, 4)), dict(logits=z(2, 4, dt=torch.float32)),
                dict(w1=z(4, 32, 64)), dict(w2=z(4, 32, 64)), dict(res=z(3, 32)), dict(w1=(z(4, 64, 64, dt=u8), z(1, 256, 4, dt=u8))),
                dict(w1=(z(4, 64, 64, dt=u8), z(1, 255, 4, dt=u8)), w2=(z(4, 64, 32, dt=u8), z(1, 256, 4, dt=u8)))):
        with pytest.raises(ValueError):
            tokens(**bad)


def test_bf16_linear():
    x, w = torch.zeros(5, 64, dtype=bf), torch.zeros(8, 64, dtype=bf)
    for bad in (dict(bias=torch.zeros(8, dtype=bf)), dict(bias=torch.zeros(7)), dict(residual=torch.zeros(5, 7, dtype=bf))):
        with pytest.raises(ValueError):
            mxa.bf16_linear(x, w, **bad)
    with pytest.raises(ValueError):
        mxa.bf16_linear(x, torch.zeros(8, 32, dtype=bf))
    d = torch.zeros(5, 8)
    with pytest.raises(ValueError):
        mxa.bf16_linear_bwd(d, x, w, act=mxa.MX_ACT_SILU)
    with pytest.raises(ValueError):
        mxa.bf16_linear_bwd(torch.zeros(5, 7), x, w)
    with pytest.raises(ValueError):
        mxa.bf16_linear_bwd(d, x, w, dx_add=torch.zeros(5, 64))


def test_adamw():
    p, g = torch.zeros(40), torch.zeros(40, dtype=bf)
    with pytest.raises(ValueError):
        mxa.adamw_state(p, 16)
    m, v, ms, vs = mxa.adamw_state(p, 8)
    assert m.dtype == u8 and m.numel() == 40 and ms.numel() == 2 and not vs.any()
    with pytest.raises(ValueError):
        moe.Adamw([(p, g, None), (p.clone(), p.clone(), None)])
    with pytest.raises(ValueError):
        moe.Adamw([(p, g, p.clone())])
    with pytest.raises(ValueError):
        moe.Adamw([(p.double(), g, None)])
    with pytest.raises(ValueError):
        moe.Adamw([(p, g, None)], grad_scale=torch.ones(1, dtype=torch.float64))


def test_host_tensors_are_refused():
    x, w, d, p = torch.zeros(5, 64, dtype=bf), torch.zeros(8, 64, dtype=bf), torch.zeros(5, 8), torch.zeros(40)
    for call in (tokens, lambda: mxa.bf16_linear(x, w), lambda: mxa.bf16_linear_bwd(d, x, w),
                 lambda: moe.Adamw([(p, p.clone(), None)])):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


@pytest.mark.parametrize("other", [torch.bfloat16, torch.float64])
def test_adamw_state_is_fp32_under_another_default_type(other):
    """The kernel reads and writes 4 bytes an element of these states."""
    torch.set_default_dtype(other)
    try:
        m, v, _, _ = mxa.adamw_state(torch.zeros(40, dtype=torch.float32), 32)
    finally:
        torch.set_default_dtype(torch.float32)
    assert m.dtype == v.dtype == torch.float32 and m.numel() == v.numel() == 40


def adam_row(n=40, bits=8, pd=torch.float32, gd=bf, copy=True):
    m, v, ms, vs = mxa.adamw_state(torch.zeros(n), bits)
    return [torch.zeros(n, dtype=pd), torch.zeros(n, dtype=gd), m, v, ms, vs, torch.zeros(n, dtype=bf) if copy else None]


@pytest.mark.parametrize("at,bad", [(0, torch.zeros(40, dtype=torch.float64)), (0, torch.zeros(40, dtype=torch.float16)),
                                    (1, torch.zeros(40, dtype=u8)), (2, torch.zeros(40)), (3, torch.zeros(40)),
                                    (2, torch.zeros(40, dtype=bf)), (4, None), (5, None), (4, torch.zeros(2)),
                                    (5, torch.zeros(2, dtype=bf)), (6, torch.zeros(40)),
                                    (1, torch.zeros(40, dtype=bf, device="meta"))])
def test_adamw_table_refuses_types_and_devices(at, bad):
    row = adam_row()
    mxa.adamw_table([row])
    row[at] = bad
    with pytest.raises(ValueError, match="adamw_table"):
        mxa.adamw_table([row])


@pytest.mark.parametrize("other", [dict(bits=32), dict(pd=bf), dict(gd=torch.float32)])
def test_adamw_table_takes_rows_of_one_kind(other):
    mxa.adamw_table([adam_row(), adam_row(n=0, copy=False)])
    with pytest.raises(ValueError, match="adamw_table"):
        mxa.adamw_table([adam_row(), adam_row(**other)])


def adam_call(table, count=1, pd=mxa.MX_OUT_F32, gd=mxa.MX_OUT_BF16, bits=8, lr=torch.zeros(1),
              step=torch.zeros(1, dtype=torch.int32), scale=None):
    mxa.mx_adamw(table, count, pd, gd, bits, lr, step, scale, 0.9, 0.999, 1e-8, 0.0, 0, 0)


@pytest.mark.parametrize("bad", [dict(pd=mxa.MX_OUT_BF16), dict(gd=mxa.MX_OUT_F32), dict(bits=32), dict(count=2),
                                 dict(lr=torch.zeros(1, dtype=torch.float64)), dict(lr=torch.zeros(0)),
                                 dict(step=torch.zeros(1)), dict(scale=torch.zeros(1, dtype=bf)),
                                 dict(lr=torch.zeros(1, device="meta"))])
def test_mx_adamw_refuses_what_its_table_does_not_hold(bad):
    table = mxa.adamw_table([adam_row()])
    with pytest.raises(ValueError, match="mx_adamw"):
        adam_call(table, **bad)


def test_mx_adamw_refuses_a_table_of_host_tensors():
    with pytest.raises(ValueError, match="not on a GPU"):
        adam_call(mxa.adamw_table([adam_row()]))


def test_adamw_table_refuses_tensors_written_twice():
    """Two blocks would update the same element, in either order."""
    a, b = adam_row(), adam_row()
    mxa.adamw_table([a, b[:1] + a[1:2] + b[2:]])              # a gradient may be shared: it is only read
    flat = torch.zeros(80)
    for i in (0, 2, 3, 4, 5, 6):
        with pytest.raises(ValueError, match="overlap"):
            mxa.adamw_table([a, b[:i] + a[i:i + 1] + b[i + 1:]])
    with pytest.raises(ValueError, match="overlap"):          # partly
        mxa.adamw_table([[flat[:40]] + a[1:], [flat[32:72]] + b[1:]])
    with pytest.raises(ValueError, match="overlap"):          # the gradient is written too
        mxa.adamw_table([a[:1] + [a[6]] + a[2:]])
    with pytest.raises(ValueError, match="overlap"):          # a copy over its fp32 parameter
        mxa.adamw_table([[flat[:40]] + a[1:6] + [flat.view(bf)[:40]]])
    mxa.adamw_table([[flat[:40]] + a[1:], [flat[40:]] + b[1:]])
    f = adam_row(bits=32)                                     # scales beside fp32 states are not touched
    mxa.adamw_table([f[:4] + a[4:5] * 2 + f[6:]])
    p = torch.zeros(40, dtype=bf)                             # a bf16 parameter's copy has its value
    mxa.adamw_table([[p] + a[1:6] + [p]])


@pytest.mark.parametrize("at", [0, 1, 2, 3, 6])
def test_adamw_table_refuses_misaligned_tensors(at):
    """When the table is built, not at each step."""
    row, old = adam_row(), adam_row(n=80)[at]
    row[at] = old[1:41]
    with pytest.raises(ValueError, match="16-byte aligned"):
        mxa.adamw_table([row])
    row[at] = old[32:72]
    mxa.adamw_table([row])
