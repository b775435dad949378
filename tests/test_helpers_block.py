"""The allocating helpers of the norm, the kept activations and the cross entropy refuse arguments that do not fit,
before any call (on the CPU)."""

import pytest
import torch

import mxfp8_block_scaled_07_amd as mxa

bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731


@pytest.mark.parametrize("bad", [dict(x=z(3, 64, dt=f32)), dict(x=z(64, 3).t()), dict(weight=z(64)), dict(weight=z(32, dt=f32)),
                                 dict(residual=z(3, 32)), dict(residual=z(3, 64, dt=torch.float64)),
                                 dict(residual=z(3, 64, dt=torch.float16)), dict(want_bf16=False)])
def test_rmsnorm(bad):
    with pytest.raises(ValueError):
        mxa.rmsnorm(**{**dict(x=z(3, 64)), **bad})


@pytest.mark.parametrize("bad", [dict(dy=z(3, 64, dt=f32)), dict(dy=z(2, 64)), dict(sum=z(3, 64, dt=torch.float64)),
                                 dict(dsum=z(3, 64, dt=f32)), dict(sum=z(3, 64, dt=f32), dsum=z(3, 64)),
                                 dict(weight=z(64)), dict(sum=z(64, 3).t(), dy=z(3, 64))])
def test_rmsnorm_bwd(bad):
    with pytest.raises(ValueError):
        mxa.rmsnorm_bwd(**{**dict(dy=z(3, 64), sum=z(3, 64)), **bad})


def test_swiglu_keep():
    for bad in (z(32, 64, dt=f32), z(64, 32).t()):
        with pytest.raises(ValueError):
            mxa.swiglu_keep(bad)


@pytest.mark.parametrize("bad", [dict(keep_q=z(32, 32, dt=u8)), dict(keep_q=z(32, 64)), dict(keep_s=z(1, 31, 4, dt=u8)),
                                 dict(keep_s=z(32, 2, dt=u8)), dict(da=z(32, 32, dt=f32)), dict(da=z(31, 32))])
def test_swiglu_bwd_kept(bad):
    with pytest.raises(ValueError):
        mxa.swiglu_bwd_kept(**{**dict(keep_q=z(32, 64, dt=u8), keep_s=z(1, 32, 4, dt=u8), da=z(32, 32)), **bad})


@pytest.mark.parametrize("bad", [dict(dots=z(9)), dict(dst_row=z(7, dt=i32)), dict(dst_row=z(6, dt=torch.int64)),
                                 dict(expert_ids=z(2, 3, dt=i32)), dict(expert_ids=z(3, 2, dt=torch.int64)), dict(weights=z(3, 2))])
def test_router_bwd_dots(bad):
    with pytest.raises(ValueError):
        mxa.router_bwd_dots(**{**dict(dots=z(9, dt=f32), dst_row=z(6, dt=i32), expert_ids=z(3, 2, dt=i32),
                                      weights=z(3, 2, dt=f32), num_experts=4), **bad})


@pytest.mark.parametrize("bad", [dict(q=z(32, 64)), dict(s=z(1, 31, 4, dt=u8)), dict(gather=z(32, dt=torch.int64)),
                                 dict(gather=z(32, dt=i32), rows_out=64), dict(q=z(0, 64, dt=u8), s=z(1, 0, 4, dt=u8), rows_out=32)])
def test_requantize(bad):
    with pytest.raises(ValueError):
        mxa.requantize(**{**dict(q=z(32, 64, dt=u8), s=z(1, 32, 4, dt=u8)), **bad})


@pytest.mark.parametrize("bad", [dict(x=z(3, 64, dt=f32)), dict(w=z(9, 32)), dict(w=z(9, 64, dt=f32)), dict(targets=z(3, dt=torch.int64)),
                                 dict(targets=z(2, dt=i32)), dict(row_weight=z(3)), dict(row_weight=z(2, dt=f32))])
def test_bf16_xent(bad):
    with pytest.raises(ValueError):
        mxa.bf16_xent(**{**dict(x=z(3, 64), w=z(9, 64), targets=z(3, dt=i32)), **bad})


def test_host_tensors_are_refused():
    for call in (lambda: mxa.rmsnorm(z(3, 64)), lambda: mxa.rmsnorm_bwd(z(3, 64), z(3, 64)), lambda: mxa.swiglu_keep(z(32, 64)),
                 lambda: mxa.swiglu_bwd_kept(z(32, 64, dt=u8), z(1, 32, 4, dt=u8), z(32, 32)),
                 lambda: mxa.router_bwd_dots(z(9, dt=f32), z(6, dt=i32), z(3, 2, dt=i32), z(3, 2, dt=f32), 4),
                 lambda: mxa.requantize(z(32, 64, dt=u8), z(1, 32, 4, dt=u8)),
                 lambda: mxa.bf16_xent(z(3, 64), z(9, 64), z(3, dt=i32))):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()
