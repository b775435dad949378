"""MI355X (gfx950) MXFP8 Mixture-of-Experts expert path.

Python binding of ``libmxmoe.so`` (declared in ``include/mxmoe.h``).  The
functions named ``mx_*`` mirror the C entry points one to one and only
marshal arguments: torch tensors stand for device buffers (their data
pointers are passed), ``None`` stands for NULL, and the stream defaults to
torch's current stream (``mx_adamw`` also refuses what does not fit a table
that ``adamw_table`` made).  The ``alloc_*``/convenience helpers only allocate
output tensors with torch and then call the same entry points.  Every
computation runs in the HIP kernels; there is no fallback: if the library is
missing or a call fails, an exception is raised.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxmoe.so")

MX_OK, MX_EINVAL, MX_EUNSUPPORTED, MX_EHIP = 0, -1, -2, -3
MX_OUT_BF16, MX_OUT_F32 = 0, 1
MX_ACT_NONE, MX_ACT_RELU, MX_ACT_GELU, MX_ACT_GELU_TANH, MX_ACT_SILU = 0, 1, 2, 3, 4

_lib = None

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_f64 = ctypes.c_double
_SIGNATURES = {
    "mx_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mx_quantize": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp]),
    "mx_dequantize": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp]),
    "mx_permute_workspace_size": (_sz, [_i64, _i32, _i32]),
    "mx_permute": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "mx_permute_noalloc": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mx_ceiling_copy": (ctypes.c_int, [_vp, _vp, _i64, _vp]),
    "mx_ceiling_tile_pattern": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "mx_ceiling_mfma": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp]),
    "mx_grouped_gemm_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "mx_grouped_gemm_dgrad": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "mx_grouped_gemm_wgrad": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "mx_swiglu_quantize": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mx_swiglu_bwd_quantize": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mx_combine": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _vp]),
    "mx_combine_bwd_quantize": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                                               _vp]),
    "mx_route_topk": (ctypes.c_int, [_vp, _i64, _i32, _i32, _vp, _vp, _vp]),
    "mx_router_bwd": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp]),
    "mx_moe_tokens_workspace_size": (_sz, [_i64, _i32, _i32, _i64]),
    "mx_moe_tokens": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                     _vp]),
    "mx_bf16_moe_tokens": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "mx_adamw": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _f64, _f64, _f64, _f64, ctypes.c_uint64,
                                _vp]),
    "mx_bf16_linear_workspace_size": (_sz, [_i64, _i64, _i64]),
    "mx_bf16_linear": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp, _i32, _vp, _sz, _vp]),
    "mx_bf16_linear_bwd_workspace_size": (_sz, [_i64, _i64, _i64, _i32]),
    "mx_bf16_linear_bwd": (ctypes.c_int, [_vp, _i32, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp,
                                          _sz, _vp]),
    "mx_bf16_gather": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp]),
    "mx_bf16_grouped_gemm_fwd": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "mx_bf16_grouped_gemm_dgrad": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "mx_bf16_grouped_gemm_wgrad": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp]),
    "mx_rmsnorm": (ctypes.c_int, [_vp, _vp, _i32, _vp, _i64, _i64, _f64, _vp, _vp, _vp, _vp, _vp]),
    "mx_rmsnorm_bwd_workspace_size": (_sz, [_i64, _i64]),
    "mx_swiglu_keep": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "mx_swiglu_bwd_kept_workspace_size": (_sz, [_i64, _i64]),
    "mx_swiglu_bwd_kept": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "mx_router_bwd_dots": (ctypes.c_int, [_vp, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _vp, _vp]),
    "mx_requantize": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp]),
    "mx_bf16_xent_workspace_size": (_sz, [_i64, _i64, _i64, _i32]),
    "mx_bf16_xent": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "mx_rmsnorm_bwd": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _i64, _i64, _f64, _vp, _vp, _vp, _vp, _sz, _vp]),
}


class AdamwTensor(ctypes.Structure):
    """mx_adamw_tensor_t: one tensor of an AdamW step (device addresses)."""
    _fields_ = [("param", _vp), ("grad", _vp), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp),
                ("copy", _vp), ("n", _i64)]


class MXError(RuntimeError):
    pass


def lib():
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MXError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype, fn.argtypes = res, args
        _lib = h
    return _lib


# (Plain integers: ctypes converts them by the signatures above.  Of a small call's
# time the host's part is the larger; with c_void_p objects and a Stream object per
# call it was 7.8 us where a launch by itself takes 3.4.)
def _p(t):
    return None if t is None else t.data_ptr()


_current = None   # torch's (raw stream of a device, current device)


def _s(stream):
    if stream is not None:
        return int(stream)
    global _current
    if _current is None:
        import torch
        _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    return _current[0](_current[1]())   # torch.cuda.current_stream().cuda_stream


def _check(rc, name):
    if rc != MX_OK:
        raise MXError(f"{name}: {lib().mx_status_string(rc).decode()}")


# --- entry points (same names and argument order as include/mxmoe.h) -------
def mx_quantize(x, batch, rows, cols, gather, rows_out, row_q, row_s, col_q, col_s, stream=None):
    _check(lib().mx_quantize(_p(x), batch, rows, cols, _p(gather), rows_out, _p(row_q), _p(row_s), _p(col_q),
                             _p(col_s), _s(stream)), "mx_quantize")


def mx_dequantize(q, s, rows, cols, y, stream=None):
    _check(lib().mx_dequantize(_p(q), _p(s), rows, cols, _p(y), _s(stream)), "mx_dequantize")


def mx_permute_workspace_size(tokens, topk, num_experts):
    return int(lib().mx_permute_workspace_size(tokens, topk, num_experts))


def mx_permute(q, s, tokens, cols, expert_ids, topk, num_experts, capacity_rows, q_out, s_out, group_offsets,
               dst_row, src_row, workspace, workspace_bytes, stream=None):
    _check(lib().mx_permute(_p(q), _p(s), tokens, cols, _p(expert_ids), topk, num_experts, capacity_rows, _p(q_out),
                            _p(s_out), _p(group_offsets), _p(dst_row), _p(src_row), _p(workspace), workspace_bytes,
                            _s(stream)), "mx_permute")


def mx_permute_noalloc(q, s, tokens, cols, expert_ids, topk, num_experts, capacity_rows, q_out, s_out,
                       group_offsets, dst_row, src_row, stream=None):
    _check(lib().mx_permute_noalloc(_p(q), _p(s), tokens, cols, _p(expert_ids), topk, num_experts, capacity_rows,
                                    _p(q_out), _p(s_out), _p(group_offsets), _p(dst_row), _p(src_row), _s(stream)),
           "mx_permute_noalloc")


def mx_ceiling_copy(src, dst, nbytes, stream=None):
    _check(lib().mx_ceiling_copy(_p(src), _p(dst), nbytes, _s(stream)), "mx_ceiling_copy")


def mx_ceiling_tile_pattern(x, row_out, col_out, rows, cols, stream=None):
    _check(lib().mx_ceiling_tile_pattern(_p(x), _p(row_out), _p(col_out), rows, cols, _s(stream)),
           "mx_ceiling_tile_pattern")


def mx_ceiling_mfma(out, workgroups, iters, random_operands=True, stream=None):
    _check(lib().mx_ceiling_mfma(_p(out), workgroups, iters, int(bool(random_operands)), _s(stream)),
           "mx_ceiling_mfma")


def mx_grouped_gemm_fwd(a_q, a_s, b_q, b_s, group_offsets, num_groups, m_cap, n, k, out, out_dtype, stream=None):
    _check(lib().mx_grouped_gemm_fwd(_p(a_q), _p(a_s), _p(b_q), _p(b_s), _p(group_offsets), num_groups, m_cap, n, k,
                                     _p(out), out_dtype, _s(stream)), "mx_grouped_gemm_fwd")


def mx_grouped_gemm_dgrad(dy_q, dy_s, wt_q, wt_s, group_offsets, num_groups, m_cap, n_out, k_contract, dx,
                          out_dtype, stream=None):
    _check(lib().mx_grouped_gemm_dgrad(_p(dy_q), _p(dy_s), _p(wt_q), _p(wt_s), _p(group_offsets), num_groups, m_cap,
                                       n_out, k_contract, _p(dx), out_dtype, _s(stream)), "mx_grouped_gemm_dgrad")


def mx_grouped_gemm_wgrad(dyt_q, dyt_s, xt_q, xt_s, group_offsets, num_groups, m_cap, n, k, dw, out_dtype,
                          stream=None):
    _check(lib().mx_grouped_gemm_wgrad(_p(dyt_q), _p(dyt_s), _p(xt_q), _p(xt_s), _p(group_offsets), num_groups, m_cap,
                                       n, k, _p(dw), out_dtype, _s(stream)), "mx_grouped_gemm_wgrad")


def mx_swiglu_quantize(h, rows, F, a, row_q, row_s, col_q, col_s, stream=None):
    _check(lib().mx_swiglu_quantize(_p(h), rows, F, _p(a), _p(row_q), _p(row_s), _p(col_q), _p(col_s), _s(stream)),
           "mx_swiglu_quantize")


def mx_swiglu_bwd_quantize(h, da, rows, F, dh, row_q, row_s, col_q, col_s, stream=None):
    _check(lib().mx_swiglu_bwd_quantize(_p(h), _p(da), rows, F, _p(dh), _p(row_q), _p(row_s), _p(col_q), _p(col_s),
                                        _s(stream)), "mx_swiglu_bwd_quantize")


def mx_combine(y, y_rows, H, dst_row, weights, tokens, topk, out, stream=None):
    _check(lib().mx_combine(_p(y), y_rows, H, _p(dst_row), _p(weights), tokens, topk, _p(out), _s(stream)),
           "mx_combine")


def mx_combine_bwd_quantize(dout, weights, dst_row, src_row, tokens, topk, rows, H, dy, row_q, row_s, col_q, col_s,
                            stream=None):
    _check(lib().mx_combine_bwd_quantize(_p(dout), _p(weights), _p(dst_row), _p(src_row), tokens, topk, rows, H,
                                         _p(dy), _p(row_q), _p(row_s), _p(col_q), _p(col_s), _s(stream)),
           "mx_combine_bwd_quantize")


def mx_route_topk(logits, tokens, num_experts, topk, expert_ids, weights, stream=None):
    _check(lib().mx_route_topk(_p(logits), tokens, num_experts, topk, _p(expert_ids), _p(weights), _s(stream)),
           "mx_route_topk")


def mx_router_bwd(dout, y, y_rows, H, dst_row, expert_ids, weights, tokens, num_experts, topk, dw, dlogits,
                  stream=None):
    _check(lib().mx_router_bwd(_p(dout), _p(y), y_rows, H, _p(dst_row), _p(expert_ids), _p(weights), tokens,
                               num_experts, topk, _p(dw), _p(dlogits), _s(stream)), "mx_router_bwd")


def mx_moe_tokens_workspace_size(tokens, topk, num_experts, F):
    return int(lib().mx_moe_tokens_workspace_size(tokens, topk, num_experts, F))


def mx_moe_tokens(x, logits, tokens, topk, num_experts, H, F, w1_q, w1_s, w2_q, w2_s, residual, out, workspace,
                  workspace_bytes, stream=None):
    _check(lib().mx_moe_tokens(_p(x), _p(logits), tokens, topk, num_experts, H, F, _p(w1_q), _p(w1_s), _p(w2_q),
                               _p(w2_s), _p(residual), _p(out), _p(workspace), workspace_bytes, _s(stream)),
           "mx_moe_tokens")


def mx_bf16_moe_tokens(x, logits, tokens, topk, num_experts, H, F, w1, w2, residual, out, workspace,
                       workspace_bytes, stream=None):
    _check(lib().mx_bf16_moe_tokens(_p(x), _p(logits), tokens, topk, num_experts, H, F, _p(w1), _p(w2), _p(residual),
                                    _p(out), _p(workspace), workspace_bytes, _s(stream)), "mx_bf16_moe_tokens")


def mx_bf16_linear_workspace_size(rows, n, k):
    return int(lib().mx_bf16_linear_workspace_size(rows, n, k))


def mx_bf16_linear(x, w, bias, residual, rows, n, k, act, z, out, out_dtype, workspace, workspace_bytes, stream=None):
    _check(lib().mx_bf16_linear(_p(x), _p(w), _p(bias), _p(residual), rows, n, k, act, _p(z), _p(out), out_dtype,
                                _p(workspace), workspace_bytes, _s(stream)), "mx_bf16_linear")


def mx_bf16_linear_bwd_workspace_size(rows, n, k, act):
    return int(lib().mx_bf16_linear_bwd_workspace_size(rows, n, k, act))


def mx_bf16_linear_bwd(dout, dout_dtype, z, x, w, dx_add, rows, n, k, act, dx, dw, dbias, workspace, workspace_bytes,
                       stream=None):
    _check(lib().mx_bf16_linear_bwd(_p(dout), dout_dtype, _p(z), _p(x), _p(w), _p(dx_add), rows, n, k, act, _p(dx),
                                    _p(dw), _p(dbias), _p(workspace), workspace_bytes, _s(stream)),
           "mx_bf16_linear_bwd")


def mx_adamw(tensors, count, param_dtype, grad_dtype, state_bits, lr, step, grad_scale, beta1, beta2, eps,
             weight_decay, seed, stream=None):
    """tensors: an array of AdamwTensor; one from adamw_table is checked against the other arguments."""
    if hasattr(tensors, "kinds"):
        _adamw_fits(tensors, count, (param_dtype, grad_dtype, state_bits), lr, step, grad_scale)
    _check(lib().mx_adamw(tensors, count, param_dtype, grad_dtype, state_bits, _p(lr), _p(step), _p(grad_scale),
                          beta1, beta2, eps, weight_decay, seed, _s(stream)), "mx_adamw")


def mx_bf16_gather(x, batch, rows, cols, gather, rows_out, out_rows, out_cols, stream=None):
    _check(lib().mx_bf16_gather(_p(x), batch, rows, cols, _p(gather), rows_out, _p(out_rows), _p(out_cols),
                                _s(stream)), "mx_bf16_gather")


def mx_bf16_grouped_gemm_fwd(a, b, group_offsets, num_groups, m_cap, n, k, out, out_dtype, stream=None):
    _check(lib().mx_bf16_grouped_gemm_fwd(_p(a), _p(b), _p(group_offsets), num_groups, m_cap, n, k, _p(out),
                                          out_dtype, _s(stream)), "mx_bf16_grouped_gemm_fwd")


def mx_bf16_grouped_gemm_dgrad(dy, wt, group_offsets, num_groups, m_cap, n_out, k_contract, dx, out_dtype,
                               stream=None):
    _check(lib().mx_bf16_grouped_gemm_dgrad(_p(dy), _p(wt), _p(group_offsets), num_groups, m_cap, n_out, k_contract,
                                            _p(dx), out_dtype, _s(stream)), "mx_bf16_grouped_gemm_dgrad")


def mx_bf16_grouped_gemm_wgrad(dyt, xt, group_offsets, num_groups, m_cap, n, k, dw, out_dtype, stream=None):
    _check(lib().mx_bf16_grouped_gemm_wgrad(_p(dyt), _p(xt), _p(group_offsets), num_groups, m_cap, n, k, _p(dw),
                                            out_dtype, _s(stream)), "mx_bf16_grouped_gemm_wgrad")


def mx_rmsnorm(x, residual, stream_dtype, weight, rows, cols, eps, sum, y, row_q, row_s, stream=None):
    _check(lib().mx_rmsnorm(_p(x), _p(residual), stream_dtype, _p(weight), rows, cols, eps, _p(sum), _p(y), _p(row_q),
                            _p(row_s), _s(stream)), "mx_rmsnorm")


def mx_rmsnorm_bwd_workspace_size(rows, cols):
    return int(lib().mx_rmsnorm_bwd_workspace_size(rows, cols))


def mx_rmsnorm_bwd(dy, sum, dsum, stream_dtype, weight, rows, cols, eps, dres, dx, dweight, workspace, workspace_bytes,
                   stream=None):
    _check(lib().mx_rmsnorm_bwd(_p(dy), _p(sum), _p(dsum), stream_dtype, _p(weight), rows, cols, eps, _p(dres), _p(dx),
                                _p(dweight), _p(workspace), workspace_bytes, _s(stream)), "mx_rmsnorm_bwd")


def mx_swiglu_keep(h, rows, F, row_q, row_s, keep_q, keep_s, stream=None):
    _check(lib().mx_swiglu_keep(_p(h), rows, F, _p(row_q), _p(row_s), _p(keep_q), _p(keep_s), _s(stream)),
           "mx_swiglu_keep")


def mx_swiglu_bwd_kept_workspace_size(rows, F):
    return int(lib().mx_swiglu_bwd_kept_workspace_size(rows, F))


def mx_swiglu_bwd_kept(keep_q, keep_s, da, rows, F, row_q, row_s, col_q, col_s, a_col_q, a_col_s, dots, workspace,
                       workspace_bytes, stream=None):
    _check(lib().mx_swiglu_bwd_kept(_p(keep_q), _p(keep_s), _p(da), rows, F, _p(row_q), _p(row_s), _p(col_q),
                                    _p(col_s), _p(a_col_q), _p(a_col_s), _p(dots), _p(workspace), workspace_bytes,
                                    _s(stream)), "mx_swiglu_bwd_kept")


def mx_router_bwd_dots(dots, rows, dst_row, expert_ids, weights, tokens, num_experts, topk, dlogits, stream=None):
    _check(lib().mx_router_bwd_dots(_p(dots), rows, _p(dst_row), _p(expert_ids), _p(weights), tokens, num_experts, topk,
                                    _p(dlogits), _s(stream)), "mx_router_bwd_dots")


def mx_requantize(q, s, rows, cols, gather, rows_out, col_q, col_s, stream=None):
    _check(lib().mx_requantize(_p(q), _p(s), rows, cols, _p(gather), rows_out, _p(col_q), _p(col_s), _s(stream)),
           "mx_requantize")


def mx_bf16_xent_workspace_size(rows, vocab, k, backward):
    return int(lib().mx_bf16_xent_workspace_size(rows, vocab, k, int(bool(backward))))


def mx_bf16_xent(x, w, targets, row_weight, rows, vocab, k, loss, lse, dx, dw, workspace, workspace_bytes, stream=None):
    _check(lib().mx_bf16_xent(_p(x), _p(w), _p(targets), _p(row_weight), rows, vocab, k, _p(loss), _p(lse), _p(dx),
                              _p(dw), _p(workspace), workspace_bytes, _s(stream)), "mx_bf16_xent")


# --- allocating helpers ----------------------------------------------------
def scale_shape(rows, cols):
    """Shape of the scale bytes of an MX tensor with ``rows`` rows (batch
    entries stacked) and ``cols`` columns, in the kernels' panel layout:
    (ceil(cols / 128), rows, 4) -- panel p, row r holds the scale bytes of
    blocks 4p..4p+3 of that row; pad bytes past the last block are zero."""
    return ((cols + 127) // 128, rows, 4)


def quantize(x, rowwise=True, colwise=False, rows_out=None, gather=None, stream=None):
    """x: bf16 (or int16 bit) tensor [rows, cols] or [batch, rows, cols] on the GPU.
    Returns (row_q, row_s, col_q, col_s); unrequested outputs are None."""
    import torch
    if x.dim() == 2:
        batch, rows, cols = 1, x.shape[0], x.shape[1]
    else:
        batch, rows, cols = x.shape
    rows_out = rows if rows_out is None else rows_out
    dev = x.device
    shp = (rows_out, cols) if x.dim() == 2 else (batch, rows_out, cols)
    row_q = torch.empty(shp, dtype=torch.uint8, device=dev) if rowwise else None
    row_s = torch.empty(scale_shape(batch * rows_out, cols), dtype=torch.uint8, device=dev) if rowwise else None
    cshp = (cols, rows_out) if x.dim() == 2 else (batch, cols, rows_out)
    col_q = torch.empty(cshp, dtype=torch.uint8, device=dev) if colwise else None
    col_s = torch.empty(scale_shape(batch * cols, rows_out), dtype=torch.uint8, device=dev) if colwise else None
    mx_quantize(x, batch, rows, cols, gather, rows_out, row_q, row_s, col_q, col_s, stream)
    return row_q, row_s, col_q, col_s


def dequantize(q, s, stream=None):
    """q: codes [..., cols] (leading dims stacked as rows), s: panel-layout scales."""
    import torch
    y = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    mx_dequantize(q, s, q.numel() // q.shape[-1], q.shape[-1], y, stream)
    return y


def permute(q, s, expert_ids, num_experts, capacity_rows=None, stream=None):
    """Returns (q_out, s_out, group_offsets, dst_row, src_row); q/s may be None
    (metadata only)."""
    import torch
    tokens, topk = expert_ids.shape
    dev = expert_ids.device
    cap = -(-(tokens * topk + 31 * num_experts) // 32) * 32 if capacity_rows is None else capacity_rows
    cols = q.shape[1] if q is not None else 0
    q_out = torch.empty((cap, cols), dtype=torch.uint8, device=dev) if q is not None else None
    s_out = torch.empty(scale_shape(cap, cols), dtype=torch.uint8, device=dev) if q is not None else None
    off = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    dst = torch.empty(tokens * topk, dtype=torch.int32, device=dev)
    src = torch.empty(cap, dtype=torch.int32, device=dev)
    wsb = mx_permute_workspace_size(tokens, topk, num_experts)
    ws = torch.empty(max(wsb, 4), dtype=torch.uint8, device=dev)
    mx_permute(q, s, tokens, cols, expert_ids, topk, num_experts, cap, q_out, s_out, off, dst, src, ws, wsb, stream)
    return q_out, s_out, off, dst, src


def _mx_pair(rows, cols, dev, want):
    import torch
    if not want:
        return None, None
    return (torch.empty((rows, cols), dtype=torch.uint8, device=dev),
            torch.empty(scale_shape(rows, cols), dtype=torch.uint8, device=dev))


def swiglu_quantize(h, rowwise=True, colwise=True, want_bf16=False, stream=None):
    """h: bf16 [rows, 2F].  Returns (a_bf16, row_q, row_s, col_q, col_s)."""
    import torch
    rows, F = h.shape[0], h.shape[1] // 2
    a = torch.empty((rows, F), dtype=torch.bfloat16, device=h.device) if want_bf16 else None
    rq, rs = _mx_pair(rows, F, h.device, rowwise)
    cq, cs = _mx_pair(F, rows, h.device, colwise)
    if rows:   # an empty input has nothing to compute (its tensors have no storage)
        mx_swiglu_quantize(h, rows, F, a, rq, rs, cq, cs, stream)
    return a, rq, rs, cq, cs


def swiglu_bwd_quantize(h, da, rowwise=True, colwise=True, want_bf16=False, stream=None):
    """h: bf16 [rows, 2F], da: bf16 [rows, F].  Returns (dh_bf16, row_q, row_s, col_q, col_s)."""
    import torch
    rows, F = h.shape[0], h.shape[1] // 2
    dh = torch.empty((rows, 2 * F), dtype=torch.bfloat16, device=h.device) if want_bf16 else None
    rq, rs = _mx_pair(rows, 2 * F, h.device, rowwise)
    cq, cs = _mx_pair(2 * F, rows, h.device, colwise)
    if rows:
        mx_swiglu_bwd_quantize(h, da, rows, F, dh, rq, rs, cq, cs, stream)
    return dh, rq, rs, cq, cs


def swiglu_keep(h, stream=None):
    """h: bf16 [rows, 2F].  Returns (row_q, row_s, keep_q, keep_s): the rowwise MX of A and of h itself."""
    import torch
    rows, F = h.shape[0], h.shape[1] // 2
    _tensor("h", h, (rows, 2 * F), torch.bfloat16)
    with _on(h.device, stream):
        rq, rs = _mx_pair(rows, F, h.device, True)
        kq, ks = _mx_pair(rows, 2 * F, h.device, True)
        if rows:
            mx_swiglu_keep(h, rows, F, rq, rs, kq, ks, stream)
    return rq, rs, kq, ks


def swiglu_bwd_kept(keep_q, keep_s, da, rowwise=True, colwise=True, a_colwise=True, want_dots=True, stream=None):
    """keep_q, keep_s as swiglu_keep left them, da bf16 [rows, F].  Returns (row_q, row_s, col_q, col_s) of dH, (a_col_q,
    a_col_s) of the rebuilt A and the dots fp32 [rows], None for what is not asked for."""
    import torch
    rows, F, dev = da.shape[0], da.shape[1], da.device
    _tensor("da", da, (rows, F), torch.bfloat16)
    _tensor("keep_q", keep_q, (rows, 2 * F), torch.uint8, dev)
    _tensor("keep_s", keep_s, scale_shape(rows, 2 * F), torch.uint8, dev)
    with _on(dev, stream):
        rq, rs = _mx_pair(rows, 2 * F, dev, rowwise)
        cq, cs = _mx_pair(2 * F, rows, dev, colwise)
        aq, as_ = _mx_pair(F, rows, dev, a_colwise)
        dots = torch.empty(rows, dtype=torch.float32, device=dev) if want_dots else None
        if rows:
            wsb = mx_swiglu_bwd_kept_workspace_size(rows, F) if want_dots else 0
            ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
            mx_swiglu_bwd_kept(keep_q, keep_s, da, rows, F, rq, rs, cq, cs, aq, as_, dots, ws, wsb, stream)
    return rq, rs, cq, cs, aq, as_, dots


def router_bwd_dots(dots, dst_row, expert_ids, weights, num_experts, stream=None):
    """The logits' gradient, fp32 [tokens, num_experts], from the dots of swiglu_bwd_kept."""
    import torch
    T, topk = weights.shape
    dev = dots.device
    _tensor("dots", dots, dots.shape, torch.float32)
    _tensor("dst_row", dst_row, (T * topk,), torch.int32, dev)
    _tensor("expert_ids", expert_ids, (T, topk), torch.int32, dev)
    _tensor("weights", weights, (T, topk), torch.float32, dev)
    with _on(dev, stream):
        dl = torch.empty((T, num_experts), dtype=torch.float32, device=dev)
        if T and not dots.numel():   # (no storage to pass; every pair's row is outside it)
            dl.zero_()
        elif T:
            mx_router_bwd_dots(dots, dots.numel(), dst_row, expert_ids, weights, T, num_experts, topk, dl, stream)
    return dl


def requantize(q, s, rows_out=None, gather=None, stream=None):
    """q, s: rowwise MX [rows, cols].  Returns (col_q, col_s), its columnwise MX of rows_out rows."""
    import torch
    rows, cols = q.shape
    rows_out = (rows if gather is None else gather.numel()) if rows_out is None else rows_out
    _tensor("q", q, (rows, cols), torch.uint8)
    _tensor("s", s, scale_shape(rows, cols), torch.uint8, q.device)
    if gather is not None:
        _tensor("gather", gather, (rows_out,), torch.int32, q.device)
    _need(rows > 0 or not rows_out, "requantize: no rows to take from")
    with _on(q.device, stream):
        cq, cs = _mx_pair(cols, rows_out, q.device, True)
        if rows_out:
            mx_requantize(q, s, rows, cols, gather, rows_out, cq, cs, stream)
    return cq, cs


def combine(y, dst_row, weights, tokens, topk, stream=None):
    """y: bf16 [rows, H] permuted rows; weights fp32 [tokens, topk] or None.  Returns bf16 [tokens, H]."""
    import torch
    out = torch.empty((tokens, y.shape[1]), dtype=torch.bfloat16, device=y.device)
    if tokens:
        mx_combine(y, y.shape[0], y.shape[1], dst_row, weights, tokens, topk, out, stream)
    return out


def combine_bwd_quantize(dout, weights, dst_row, src_row, topk, rows, rowwise=True, colwise=True, want_bf16=False,
                         stream=None):
    """dout: bf16 [tokens, H].  Returns (dy_bf16, row_q, row_s, col_q, col_s) of the permuted gradient [rows, H]."""
    import torch
    tokens, H = dout.shape
    dy = torch.empty((rows, H), dtype=torch.bfloat16, device=dout.device) if want_bf16 else None
    rq, rs = _mx_pair(rows, H, dout.device, rowwise)
    cq, cs = _mx_pair(H, rows, dout.device, colwise)
    if rows:
        mx_combine_bwd_quantize(dout if tokens else None, weights if tokens else None, dst_row if tokens else None,
                                src_row, tokens, topk, rows, H, dy, rq, rs, cq, cs, stream)
    return dy, rq, rs, cq, cs


def route_topk(logits, topk, stream=None):
    """logits: fp32 [tokens, E].  Returns (expert_ids int32 [tokens, topk], weights fp32 [tokens, topk])."""
    import torch
    T, E = logits.shape
    ids = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    if T:
        mx_route_topk(logits, T, E, topk, ids, w, stream)
    return ids, w


def router_bwd(dout, y, dst_row, expert_ids, weights, num_experts, stream=None):
    """Returns (dw fp32 [tokens, topk], dlogits fp32 [tokens, num_experts])."""
    import torch
    T, topk = weights.shape
    dw = torch.empty((T, topk), dtype=torch.float32, device=dout.device)
    dl = torch.empty((T, num_experts), dtype=torch.float32, device=dout.device)
    if T:
        mx_router_bwd(dout, y, y.shape[0], y.shape[1], dst_row, expert_ids, weights, T, num_experts, topk, dw, dl,
                      stream)
    return dw, dl


# --- the layer for a few tokens, the dense product, AdamW ---------------------
def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _tensor(name, t, shape, dtype, device=None):
    """t is a contiguous tensor of this shape and type (bf16 may come as its int16 bits) on the device."""
    import torch
    kinds = (torch.bfloat16, torch.int16) if dtype == torch.bfloat16 else (dtype,)
    _need(tuple(t.shape) == tuple(shape), f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    _need(t.dtype in kinds, f"{name} is {t.dtype}, not {dtype}")
    _need(t.is_contiguous(), f"{name} is not contiguous")
    _need(device is None or t.device == device, f"{name} is on {t.device}, not {device}")


def _on(device, stream):
    """The tensors' device as the current one, and the call's stream as its current stream: what a helper allocates
    inside belongs to that stream, so the memory is not handed out again before the call's kernels have run."""
    import torch
    _need(device.type == "cuda", f"tensors are on {device}, not on a GPU")
    if stream is None:
        return torch.cuda.device(device)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=device))


def moe_tokens(x, logits, topk, w1, w2, residual=None, stream=None):
    """The whole MoE layer for at most 64 tokens: x bf16 [T, H], logits fp32 [T, E]; w1, w2 bf16 [E, 2F, H] and
    [E, H, F], or MX rowwise (codes, scales) pairs of them.  Returns bf16 [T, H]."""
    import torch
    T, H = x.shape
    mxw = isinstance(w1, (tuple, list))
    _need(mxw == isinstance(w2, (tuple, list)), "moe_tokens: w1 and w2 are both bf16 or both (codes, scales)")
    E, F = logits.shape[1], (w2[0] if mxw else w2).shape[2]
    dev, bf = x.device, torch.bfloat16
    _tensor("x", x, (T, H), bf)
    _tensor("logits", logits, (T, E), torch.float32, dev)
    if mxw:
        _tensor("w1 codes", w1[0], (E, 2 * F, H), torch.uint8, dev)
        _tensor("w1 scales", w1[1], scale_shape(E * 2 * F, H), torch.uint8, dev)
        _tensor("w2 codes", w2[0], (E, H, F), torch.uint8, dev)
        _tensor("w2 scales", w2[1], scale_shape(E * H, F), torch.uint8, dev)
    else:
        _tensor("w1", w1, (E, 2 * F, H), bf, dev)
        _tensor("w2", w2, (E, H, F), bf, dev)
    if residual is not None:
        _tensor("residual", residual, (T, H), bf, dev)
    with _on(dev, stream):
        out = torch.empty((T, H), dtype=bf, device=dev)
        if T:
            wsb = mx_moe_tokens_workspace_size(T, topk, E, F)
            ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
            if mxw:
                mx_moe_tokens(x, logits, T, topk, E, H, F, w1[0], w1[1], w2[0], w2[1], residual, out, ws, wsb, stream)
            else:
                mx_bf16_moe_tokens(x, logits, T, topk, E, H, F, w1, w2, residual, out, ws, wsb, stream)
    return out


def bf16_linear(x, w, bias=None, residual=None, act=MX_ACT_NONE, out_dtype=MX_OUT_BF16, want_z=False, stream=None):
    """act(x w^T + bias) + residual: x bf16 [M, K], w bf16 [N, K], bias fp32 [N], residual bf16 [M, N].
    Returns (out, z), z the bf16 pre-activation for the backward or None."""
    import torch
    M, K = x.shape
    N, dev, bf = w.shape[0], x.device, torch.bfloat16
    _tensor("x", x, (M, K), bf)
    _tensor("w", w, (N, K), bf, dev)
    if bias is not None:
        _tensor("bias", bias, (N,), torch.float32, dev)
    if residual is not None:
        _tensor("residual", residual, (M, N), bf, dev)
    with _on(dev, stream):
        out = torch.empty((M, N), dtype=bf if out_dtype == MX_OUT_BF16 else torch.float32, device=dev)
        z = torch.empty((M, N), dtype=bf, device=dev) if want_z else None
        if M:
            wsb = mx_bf16_linear_workspace_size(M, N, K)
            ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
            mx_bf16_linear(x, w, bias, residual, M, N, K, act, z, out, out_dtype, ws, wsb, stream)
    return out, z


def bf16_linear_bwd(dout, x, w, z=None, act=MX_ACT_NONE, dx_add=None, want_dbias=True, stream=None):
    """Backward of bf16_linear: dout bf16 or fp32 [M, N], z as kept by the forward (needed with an activation).
    Returns (dx bf16 [M, K], dw bf16 [N, K], dbias fp32 [N] or None)."""
    import torch
    M, K = x.shape
    N, dev, bf = w.shape[0], x.device, torch.bfloat16
    f32 = dout.dtype == torch.float32
    _tensor("dout", dout, (M, N), torch.float32 if f32 else bf, dev)
    _tensor("x", x, (M, K), bf)
    _tensor("w", w, (N, K), bf, dev)
    _need(act == MX_ACT_NONE or z is not None, "bf16_linear_bwd: the activation's backward needs z")
    if z is not None:
        _tensor("z", z, (M, N), bf, dev)
    if dx_add is not None:
        _tensor("dx_add", dx_add, (M, K), bf, dev)
    with _on(dev, stream):
        dx = torch.empty((M, K), dtype=bf, device=dev)
        dw = torch.empty((N, K), dtype=bf, device=dev)
        db = torch.empty(N, dtype=torch.float32, device=dev) if want_dbias else None
        if M:
            wsb = mx_bf16_linear_bwd_workspace_size(M, N, K, act)
            ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
            mx_bf16_linear_bwd(dout, MX_OUT_F32 if f32 else MX_OUT_BF16, z, x, w, dx_add, M, N, K, act, dx, dw, db, ws,
                               wsb, stream)
        else:   # empty tensors have no storage to pass
            dw.zero_()
            if db is not None:
                db.zero_()
    return dx, dw, db


def _stream_kind(name, t):
    """MX_OUT_BF16 or MX_OUT_F32 of a tensor of the residual stream, and its torch type."""
    import torch
    if t is None or t.dtype in (torch.bfloat16, torch.int16):
        return MX_OUT_BF16, torch.bfloat16
    _need(t.dtype == torch.float32, f"{name} is {t.dtype}, not bf16 or fp32")
    return MX_OUT_F32, torch.float32


def rmsnorm(x, weight=None, residual=None, eps=1e-6, want_bf16=True, rowwise=False, stream=None):
    """Norm of x + residual: x bf16 [R, C], residual bf16 or fp32 [R, C], weight fp32 [C].  Returns (sum, y, row_q,
    row_s): the new residual stream (x itself without a residual), the bf16 rows and their rowwise MX, None for what is
    not asked for."""
    import torch
    R, C = x.shape
    dev, bf = x.device, torch.bfloat16
    _need(want_bf16 or rowwise, "rmsnorm: at least one of want_bf16 and rowwise")
    _tensor("x", x, (R, C), bf)
    kind, dtype = _stream_kind("residual", residual)
    if residual is not None:
        _tensor("residual", residual, (R, C), dtype, dev)
    if weight is not None:
        _tensor("weight", weight, (C,), torch.float32, dev)
    with _on(dev, stream):
        total = x if residual is None else torch.empty((R, C), dtype=dtype, device=dev)
        y = torch.empty((R, C), dtype=bf, device=dev) if want_bf16 else None
        rq, rs = _mx_pair(R, C, dev, rowwise)
        if R:
            mx_rmsnorm(x, residual, kind, weight, R, C, eps, None if residual is None else total, y, rq, rs, stream)
    return total, y, rq, rs


def rmsnorm_bwd(dy, sum, weight=None, dsum=None, eps=1e-6, want_dweight=True, stream=None):
    """Backward of rmsnorm: dy bf16 [R, C]; sum, and the gradient dsum that reaches it from elsewhere, of the residual
    stream's type.  Returns (dres in that type, dx in bf16, dweight fp32 [C] or None); dx is dres where the stream is
    bf16."""
    import torch
    R, C = sum.shape
    dev, bf = sum.device, torch.bfloat16
    kind, dtype = _stream_kind("sum", sum)
    _tensor("sum", sum, (R, C), dtype)
    _tensor("dy", dy, (R, C), bf, dev)
    if dsum is not None:
        _tensor("dsum", dsum, (R, C), dtype, dev)
    if weight is not None:
        _tensor("weight", weight, (C,), torch.float32, dev)
    with _on(dev, stream):
        dres = torch.empty((R, C), dtype=dtype, device=dev)
        dx = dres if kind == MX_OUT_BF16 else torch.empty((R, C), dtype=bf, device=dev)
        dw = torch.empty(C, dtype=torch.float32, device=dev) if want_dweight else None
        if R:
            wsb = mx_rmsnorm_bwd_workspace_size(R, C) if want_dweight else 0
            ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
            mx_rmsnorm_bwd(dy, sum, dsum, kind, weight, R, C, eps, dres, None if kind == MX_OUT_BF16 else dx, dw, ws, wsb,
                           stream)
        elif dw is not None:   # empty tensors have no storage to pass
            dw.zero_()
    return dres, dx, dw


def bf16_xent(x, w, targets, row_weight=None, want_grad=False, stream=None):
    """Cross entropy of x w^T: x bf16 [M, K], w bf16 [V, K], targets int32 [M] (outside [0, V): left out), row_weight
    fp32 [M], of the gradient.  Returns (loss fp32 [M], lse fp32 [M], dx bf16 [M, K], dw bf16 [V, K]), the last two None
    without want_grad."""
    import torch
    M, K = x.shape
    V, dev, bf = w.shape[0], x.device, torch.bfloat16
    _tensor("x", x, (M, K), bf)
    _tensor("w", w, (V, K), bf, dev)
    _tensor("targets", targets, (M,), torch.int32, dev)
    if row_weight is not None:
        _tensor("row_weight", row_weight, (M,), torch.float32, dev)
    with _on(dev, stream):
        loss, lse = (torch.empty(M, dtype=torch.float32, device=dev) for _ in range(2))
        dx = torch.empty((M, K), dtype=bf, device=dev) if want_grad else None
        dw = torch.empty((V, K), dtype=bf, device=dev) if want_grad else None
        if M:
            wsb = mx_bf16_xent_workspace_size(M, V, K, want_grad)
            ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
            mx_bf16_xent(x, w, targets, row_weight, M, V, K, loss, lse, dx, dw, ws, wsb, stream)
        elif want_grad:   # empty tensors have no storage to pass
            dw.zero_()
    return loss, lse, dx, dw


def adamw_state(param, state_bits=32):
    """(m, v, m_scale, v_scale) of a new AdamW state for a parameter: fp32 zeros, or MX codes and scales of zeros."""
    import torch
    _need(state_bits in (8, 32), "adamw_state: state_bits is 8 or 32")
    n, dev = param.numel(), param.device
    if state_bits == 32:
        z = lambda k: torch.zeros(k, dtype=torch.float32, device=dev)  # noqa: E731
        return z(n), z(n), None, None
    z = lambda k: torch.zeros(k, dtype=torch.uint8, device=dev)  # noqa: E731
    return z(n), z(n), z(-(-n // 32)), z(-(-n // 32))


def adamw_table(rows):
    """The host table mx_adamw takes, from (param, grad, m, v, m_scale, v_scale, copy) per tensor (contiguous device
    tensors of the types the header names, the same in every row; None for what is not there).  It keeps its tensors
    alive and can be used for every step; mx_adamw refuses arguments that do not fit what it holds."""
    import torch
    kinds = {torch.float32: MX_OUT_F32, torch.bfloat16: MX_OUT_BF16, torch.int16: MX_OUT_BF16}
    bytes_ = (torch.uint8, torch.float8_e4m3fn, torch.float8_e8m0fnu)
    table = (AdamwTensor * len(rows))()
    table.device = table.kinds = None
    ranges = []   # of each tensor: its addresses, and whether it is written
    for t, row in zip(table, rows):
        param, grad, m, v, m_scale, v_scale, copy = row
        n = param.numel()
        for x in row:
            if x is not None and not x.is_contiguous():
                raise ValueError("adamw_table: tensors must be contiguous")
        for x, want in ((grad, n), (m, n), (v, n), (copy, n), (m_scale, -(-n // 32)), (v_scale, -(-n // 32))):
            if x is not None and x.numel() != want:
                raise ValueError(f"adamw_table: {x.numel()} elements where {want} belong to a parameter of {n}")
        for x in row:
            _need(x is None or x.device == param.device, "adamw_table: a row's tensors are on one device")
        _need(param.dtype in kinds and grad.dtype in kinds, "adamw_table: parameters and gradients are fp32 or bf16")
        _need(copy is None or kinds.get(copy.dtype) == MX_OUT_BF16, "adamw_table: copies are bf16")
        _need(not any(x is not None and x.numel() and x.data_ptr() % 16 for x in (param, grad, m, v, copy)),
              "adamw_table: tensors (but the scales) are 16-byte aligned")
        bits = 32 if m.dtype == torch.float32 else 8
        if bits == 32:
            _need(v.dtype == torch.float32, "adamw_table: m and v are both fp32 or both codes")
        else:
            _need(m.dtype in bytes_ and v.dtype in bytes_, "adamw_table: m and v are both fp32 or both codes (one byte)")
            _need(all(x is not None and x.dtype in bytes_ for x in (m_scale, v_scale)),
                  "adamw_table: codes have scales of one byte")
        found = kinds[param.dtype], kinds[grad.dtype], bits
        _need(table.kinds in (None, found) and table.device in (None, param.device),
              "adamw_table: types and device are the same in every row")
        table.kinds, table.device = found, param.device
        t.param, t.grad, t.m, t.v = (x.data_ptr() for x in (param, grad, m, v))
        t.m_scale, t.v_scale, t.copy = (None if x is None else x.data_ptr() for x in (m_scale, v_scale, copy))
        t.n = n
        used = [(grad, False)] + [(x, True) for x in (param, m, v, *((m_scale, v_scale) if bits == 8 else ()))]
        if copy is not None and not (copy.dtype == param.dtype and copy.data_ptr() == param.data_ptr()):
            used.append((copy, True))   # (over a bf16 parameter it writes the same values)
        ranges += [(x.data_ptr(), x.data_ptr() + x.numel() * x.element_size(), w) for x, w in used
                   if x is not None and x.numel()]
    end = end_written = 0
    for a, b, w in sorted(ranges):
        _need(a >= (end if w else end_written), "adamw_table: tensors that are written overlap")
        end, end_written = max(end, b), max(end_written, b if w else 0)
    table.tensors = rows
    return table


def _adamw_fits(table, count, kinds, lr, step, grad_scale):
    """The arguments of mx_adamw are those of a table that adamw_table made."""
    import torch
    _need(count <= len(table), f"mx_adamw: {count} tensors of a table of {len(table)}")
    if table.kinds is None:
        return
    _need(kinds == table.kinds, "mx_adamw: the table's tensors are of other types (param_dtype, grad_dtype, state_bits)")
    for name, t, dtype in (("lr", lr, torch.float32), ("step", step, torch.int32), ("grad_scale", grad_scale, torch.float32)):
        _need(t is None or (t.dtype == dtype and t.numel() >= 1 and t.device == table.device),
              f"mx_adamw: {name} is a {dtype} scalar on the tensors' device")
    _need(table.device.type == "cuda", f"mx_adamw: tensors are on {table.device}, not on a GPU")
