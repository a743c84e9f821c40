"""ctypes binding of libmxq.so (include/mxq.h).  Argument marshalling only."""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(PKG, "libmxq.so")

MXQ_F32, MXQ_BF16, MXQ_E4M3, MXQ_E5M2, MXQ_E2M1 = 0, 1, 2, 3, 4
MXQ_ROWWISE, MXQ_COLWISE = 0, 1
MXQ_ACC_FP8_MFMA, MXQ_ACC_FP32 = 0, 1
MXQ_ACT_NONE, MXQ_ACT_SILU = 0, 1
MXQ_SCALE_CEIL, MXQ_SCALE_OCP, MXQ_SCALE_AMAX = 0, 1, 2

_ELEM = {"e4m3": MXQ_E4M3, "e5m2": MXQ_E5M2}
_ACC = {"fp8": MXQ_ACC_FP8_MFMA, "fp32": MXQ_ACC_FP32}
_ACT = {None: MXQ_ACT_NONE, "none": MXQ_ACT_NONE, "silu": MXQ_ACT_SILU}
_AXIS = {"row": MXQ_ROWWISE, "col": MXQ_COLWISE, 0: MXQ_ROWWISE, 1: MXQ_COLWISE}
_RULE = {"ceil": MXQ_SCALE_CEIL, "ocp": MXQ_SCALE_OCP}


class MxqError(ValueError):
    """A negative mxq_status from the library (invalid arguments or a HIP launch error)."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (%d)" % (where, mxq_status_string(status), status))


_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libmxq.so; raises if it has not been built (there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libmxq.so is not built (run __graft_entry__.build() or "
                               "python -m mxfp8_block_scaled_03_amd.build)")
        L = ctypes.CDLL(_LIB_PATH)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        L.mxq_quantize.restype = ci
        L.mxq_quantize.argtypes = [vp, ci, i64, i64, i64, ci, ci, vp, i64, vp, i64, vp]
        L.mxq_quantize_rule.restype = ci
        L.mxq_quantize_rule.argtypes = [vp, ci, i64, i64, i64, ci, ci, ci, vp, i64, vp, i64, vp]
        L.mxq_quantize_sr.restype = ci
        L.mxq_quantize_sr.argtypes = [vp, ci, i64, i64, i64, ci, ci, ctypes.c_uint64, vp, i64, vp, i64, vp]
        L.mxq_quantize_scaled.restype = ci
        L.mxq_quantize_scaled.argtypes = [vp, ci, i64, i64, i64, ci, ci, vp, i64, vp, i64, vp, i64, vp, vp, i64, vp]
        L.mxq_quantize_dual.restype = ci
        L.mxq_quantize_dual.argtypes = [vp, ci, i64, i64, i64, ci, vp, i64, vp, i64, vp, i64, vp, i64, vp]
        L.mxq_dequantize.restype = ci
        L.mxq_dequantize.argtypes = [vp, i64, vp, i64, ci, i64, i64, vp, ci, i64, vp]
        L.mxq_gemm.restype = ci
        L.mxq_gemm.argtypes = [i64, i64, i64, vp, i64, vp, i64, ci, vp, i64, vp, i64, ci,
                               ctypes.c_float, vp, vp, ci, i64, ci, vp]
        L.mxq_gemm_ex.restype = ci
        L.mxq_gemm_ex.argtypes = [i64, i64, i64, vp, i64, vp, i64, ci, vp, i64, vp, i64, ci,
                                  ctypes.c_float, vp, ci, vp, ci, i64, ci, vp, i64, vp, i64, ci, vp]
        L.mxq_gemm_ex_noalloc.restype = ci
        L.mxq_gemm_ex_noalloc.argtypes = L.mxq_gemm_ex.argtypes
        L.mxq_status_string.restype = ctypes.c_char_p
        L.mxq_status_string.argtypes = [ci]
        L.mxq_version.restype = ci
        L.mxq_version.argtypes = []
        L.mxq_gemm_exact_plan.restype = ci
        ip = ctypes.POINTER(ci)
        L.mxq_gemm_exact_plan.argtypes = [i64, i64, i64, ci, ip, ip, ip, ip, ctypes.POINTER(i64)]
        L.mxq_quantize_fp4.restype = ci
        L.mxq_quantize_fp4.argtypes = [vp, ci, i64, i64, i64, ci, ci, vp, i64, vp, i64, vp]
        L.mxq_quantize_fp4_sr.restype = ci
        L.mxq_quantize_fp4_sr.argtypes = [vp, ci, i64, i64, i64, ci, ctypes.c_uint64, vp, i64, vp, i64, vp]
        L.mxq_quantize_fp4_dual.restype = ci
        L.mxq_quantize_fp4_dual.argtypes = [vp, ci, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp]
        L.mxq_dequantize_fp4.restype = ci
        L.mxq_dequantize_fp4.argtypes = [vp, i64, vp, i64, i64, i64, vp, ci, i64, vp]
        L.mxq_gemm_fp4.restype = ci
        L.mxq_gemm_fp4.argtypes = [i64, i64, i64, vp, ci, i64, vp, i64, vp, i64, vp, i64, ctypes.c_float, vp, ci, vp,
                                   ci, i64, vp]
        L.mxq_gemm_fp4_plan.restype = ci
        L.mxq_gemm_fp4_plan.argtypes = [i64, i64, i64, ci, ci, ci, ip, ip, ip]
        L.mxq_moe_fp4_plan.restype = ci
        L.mxq_moe_fp4_plan.argtypes = [i64, i64, i64, i64, i64, ci, ci, ci, ip, ip, ip, ip]
        L.mxq_moe_fp4_workspace.restype = ci
        L.mxq_moe_fp4_workspace.argtypes = [i64, i64, i64, i64, i64, ci, ctypes.POINTER(i64)]
        L.mxq_moe_fp4.restype = ci
        L.mxq_moe_fp4.argtypes = [i64, i64, i64, i64, i64, ci, vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp, i64,
                                  i64, vp, i64, i64, vp, ci, i64, vp, i64, vp]
        f32 = ctypes.c_float
        L.mxq_quantize_b128.restype = ci
        L.mxq_quantize_b128.argtypes = [vp, ci, i64, i64, i64, ci, ci, ci, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp]
        L.mxq_gemm_b128.restype = ci
        L.mxq_gemm_b128.argtypes = [i64, i64, i64, vp, i64, vp, i64, ci, vp, i64, vp, i64, i64, ci, ci, f32, vp, ci, ci, vp,
                                    ci, i64, vp]
        L.mxq_moe_gemm_b128.restype = ci
        L.mxq_moe_gemm_b128.argtypes = [i64, i64, i64, i64, vp, vp, i64, vp, i64, ci, vp, i64, i64, vp, i64, i64, i64, ci,
                                        ci, ci, vp, ci, i64, vp]
        L.mxq_moe_wgrad_b128.restype = ci
        L.mxq_moe_wgrad_b128.argtypes = [i64, i64, i64, i64, vp, vp, i64, vp, i64, ci, vp, i64, vp, i64, ci, ci, vp, ci, i64,
                                         i64, vp]
        L.mxq_gemm_b128_plan.restype = ci
        L.mxq_gemm_b128_plan.argtypes = [ci, i64, i64, i64, i64, ci, ci, ci, ip, ip, ip]
        L.mxq_moe_route_workspace.restype = ci
        L.mxq_moe_route_workspace.argtypes = [i64, i64, i64, ctypes.POINTER(i64)]
        L.mxq_moe_route.restype = ci
        L.mxq_moe_route.argtypes = [i64, i64, i64, ci, vp, ci, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp]
        L.mxq_moe_route_grad.restype = ci
        L.mxq_moe_route_grad.argtypes = [i64, i64, i64, ci, vp, ci, i64, vp, vp, vp, vp, vp, i64, vp, vp, i64, vp]
        _lib = L
    return _lib


# ----------------------------------------------------------------- raw C entry points

def mxq_quantize(src, src_type, rows, cols, ld_src, axis, elem, codes, ld_codes, scales, ld_scales,
                 stream=None) -> int:
    return lib().mxq_quantize(src, src_type, rows, cols, ld_src, axis, elem, codes, ld_codes, scales,
                              ld_scales, stream)


def mxq_quantize_rule(src, src_type, rows, cols, ld_src, axis, elem, rule, codes, ld_codes, scales, ld_scales,
                      stream=None) -> int:
    return lib().mxq_quantize_rule(src, src_type, rows, cols, ld_src, axis, elem, rule, codes, ld_codes, scales,
                                   ld_scales, stream)


def mxq_quantize_sr(src, src_type, rows, cols, ld_src, axis, elem, seed, codes, ld_codes, scales, ld_scales,
                    stream=None) -> int:
    return lib().mxq_quantize_sr(src, src_type, rows, cols, ld_src, axis, elem, seed, codes, ld_codes, scales,
                                 ld_scales, stream)


def mxq_quantize_scaled(src, src_type, rows, cols, ld_src, axis, elem, scales, ld_scales, codes, ld_codes,
                        amax, ld_amax, clipped, flushed, ld_diag, stream=None) -> int:
    return lib().mxq_quantize_scaled(src, src_type, rows, cols, ld_src, axis, elem, scales, ld_scales, codes,
                                     ld_codes, amax, ld_amax, clipped, flushed, ld_diag, stream)


def mxq_quantize_dual(src, src_type, rows, cols, ld_src, elem, row_codes, ld_row_codes, row_scales, ld_row_scales,
                      col_codes, ld_col_codes, col_scales, ld_col_scales, stream=None) -> int:
    return lib().mxq_quantize_dual(src, src_type, rows, cols, ld_src, elem, row_codes, ld_row_codes, row_scales,
                                   ld_row_scales, col_codes, ld_col_codes, col_scales, ld_col_scales, stream)


def mxq_dequantize(codes, ld_codes, scales, ld_scales, elem, L, K, dst, dst_type, ld_dst, stream=None) -> int:
    return lib().mxq_dequantize(codes, ld_codes, scales, ld_scales, elem, L, K, dst, dst_type, ld_dst, stream)


def mxq_gemm(M, N, K, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ld_ws, w_elem,
             alpha, bias, y, y_type, ld_y, accum=MXQ_ACC_FP32, stream=None) -> int:
    return lib().mxq_gemm(M, N, K, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ld_ws,
                          w_elem, alpha, bias, y, y_type, ld_y, accum, stream)


def mxq_gemm_ex(M, N, K, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ld_ws, w_elem,
                alpha, bias, act, y, y_type, ld_y, q_elem, q_codes, ld_q_codes, q_scales, ld_q_scales,
                accum=MXQ_ACC_FP32, stream=None) -> int:
    return lib().mxq_gemm_ex(M, N, K, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ld_ws,
                             w_elem, alpha, bias, act, y, y_type, ld_y, q_elem, q_codes, ld_q_codes, q_scales,
                             ld_q_scales, accum, stream)


def mxq_gemm_ex_noalloc(M, N, K, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ld_ws, w_elem,
                        alpha, bias, act, y, y_type, ld_y, q_elem, q_codes, ld_q_codes, q_scales, ld_q_scales,
                        accum=MXQ_ACC_FP32, stream=None) -> int:
    return lib().mxq_gemm_ex_noalloc(M, N, K, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ld_ws,
                                     w_elem, alpha, bias, act, y, y_type, ld_y, q_elem, q_codes, ld_q_codes, q_scales,
                                     ld_q_scales, accum, stream)


def mxq_status_string(status: int) -> str:
    return lib().mxq_status_string(status).decode()


def mxq_version() -> int:
    return lib().mxq_version()


def mxq_gemm_exact_plan(M: int, N: int, K: int, cus: int) -> dict:
    """The exact-product GEMM's plan for an M x N x K problem on `cus` CUs (host logic, no
    device): tile width, K ranges per split tile, split and whole tiles, workspace bytes.
    Raises MxqError (a ValueError) on a negative status."""
    c = ctypes.c_int
    tn, ks, sp, wh, wb = c(), c(), c(), c(), ctypes.c_int64()
    _check(lib().mxq_gemm_exact_plan(M, N, K, cus, ctypes.byref(tn), ctypes.byref(ks), ctypes.byref(sp),
                                     ctypes.byref(wh), ctypes.byref(wb)), "mxq_gemm_exact_plan")
    return {"tile_n": tn.value, "ranges_per_tile": ks.value, "split_tiles": sp.value, "whole_tiles": wh.value,
            "workspace_bytes": wb.value}


def mxq_quantize_fp4(src, src_type, rows, cols, ld_src, axis, rule, codes, ld_codes, scales, ld_scales,
                     stream=None) -> int:
    return lib().mxq_quantize_fp4(src, src_type, rows, cols, ld_src, axis, rule, codes, ld_codes, scales, ld_scales,
                                  stream)


def mxq_quantize_fp4_sr(src, src_type, rows, cols, ld_src, axis, seed, codes, ld_codes, scales, ld_scales,
                        stream=None) -> int:
    return lib().mxq_quantize_fp4_sr(src, src_type, rows, cols, ld_src, axis, seed, codes, ld_codes, scales, ld_scales,
                                     stream)


def mxq_quantize_fp4_dual(src, src_type, rows, cols, ld_src, row_codes, ld_row_codes, row_scales, ld_row_scales,
                          col_codes, ld_col_codes, col_scales, ld_col_scales, stream=None) -> int:
    return lib().mxq_quantize_fp4_dual(src, src_type, rows, cols, ld_src, row_codes, ld_row_codes, row_scales,
                                       ld_row_scales, col_codes, ld_col_codes, col_scales, ld_col_scales, stream)


def mxq_dequantize_fp4(codes, ld_codes, scales, ld_scales, L, K, dst, dst_type, ld_dst, stream=None) -> int:
    return lib().mxq_dequantize_fp4(codes, ld_codes, scales, ld_scales, L, K, dst, dst_type, ld_dst, stream)


def mxq_gemm_fp4(M, N, K, x, x_type, ld_x, x_scales, ld_xs, w_codes, ld_w, w_scales, ld_ws, alpha, bias, act, y,
                 y_type, ld_y, stream=None) -> int:
    return lib().mxq_gemm_fp4(M, N, K, x, x_type, ld_x, x_scales, ld_xs, w_codes, ld_w, w_scales, ld_ws, alpha, bias,
                              act, y, y_type, ld_y, stream)


def mxq_gemm_fp4_plan(M: int, N: int, K: int, x_type: int, aligned: bool, cus: int) -> tuple:
    """(tile_m, tile_n, waves) of the MXFP4 product (host logic only); raises MxqError."""
    out = [ctypes.c_int() for _ in range(3)]
    st = lib().mxq_gemm_fp4_plan(M, N, K, x_type, aligned, cus, *(ctypes.byref(v) for v in out))
    _check(st, "mxq_gemm_fp4_plan")
    return tuple(v.value for v in out)


def mxq_moe_fp4_plan(T: int, H: int, I: int, E: int, k: int, y_type: int, aligned: bool, cus: int) -> tuple:
    """(launches, up_columns, down_columns, down_parts) of the expert layer (host logic only); raises MxqError."""
    out = [ctypes.c_int() for _ in range(4)]
    st = lib().mxq_moe_fp4_plan(T, H, I, E, k, y_type, aligned, cus, *(ctypes.byref(v) for v in out))
    _check(st, "mxq_moe_fp4_plan")
    return tuple(v.value for v in out)


def mxq_moe_fp4_workspace(T, H, I, E, k, y_type) -> int:
    """Bytes of workspace that mxq_moe_fp4 needs (host logic only); raises MxqError."""
    n = ctypes.c_int64()
    _check(lib().mxq_moe_fp4_workspace(T, H, I, E, k, y_type, ctypes.byref(n)), "mxq_moe_fp4_workspace")
    return n.value


def mxq_moe_fp4(T, H, I, E, k, renormalize, x, ld_x, logits, ld_logits, w13_codes, ld_w13, expert_w13, w13_scales,
                ld_s13, expert_s13, w2_codes, ld_w2, expert_w2, w2_scales, ld_s2, expert_s2, y, y_type, ld_y,
                workspace, workspace_bytes, stream=None) -> int:
    return lib().mxq_moe_fp4(T, H, I, E, k, renormalize, x, ld_x, logits, ld_logits, w13_codes, ld_w13, expert_w13,
                             w13_scales, ld_s13, expert_s13, w2_codes, ld_w2, expert_w2, w2_scales, ld_s2, expert_s2,
                             y, y_type, ld_y, workspace, workspace_bytes, stream)


def mxq_quantize_b128(src, src_type, rows, cols, ld_src, elem, rule, tile, row_codes, ld_row_codes, row_scales,
                      ld_row_scales, col_codes, ld_col_codes, col_scales, ld_col_scales, offsets, experts,
                      stream=None) -> int:
    return lib().mxq_quantize_b128(src, src_type, rows, cols, ld_src, elem, rule, tile, row_codes, ld_row_codes, row_scales,
                                   ld_row_scales, col_codes, ld_col_codes, col_scales, ld_col_scales, offsets, experts,
                                   stream)


def mxq_gemm_b128(M, N, K, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ws_line, ws_block, w_block,
                  w_elem, alpha, bias, act, accum, y, y_type, ld_y, stream=None) -> int:
    return lib().mxq_gemm_b128(M, N, K, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ws_line, ws_block,
                               w_block, w_elem, alpha, bias, act, accum, y, y_type, ld_y, stream)


def mxq_moe_gemm_b128(rows, N, K, E, offsets, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, expert_w, w_scales,
                      ws_line, ws_block, expert_ws, w_block, w_elem, accum, y, y_type, ld_y, stream=None) -> int:
    return lib().mxq_moe_gemm_b128(rows, N, K, E, offsets, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, expert_w,
                                   w_scales, ws_line, ws_block, expert_ws, w_block, w_elem, accum, y, y_type, ld_y, stream)


def mxq_moe_wgrad_b128(M, N, rows, E, offsets, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales, ld_ws,
                       w_elem, accum, y, y_type, ld_y, expert_y, stream=None) -> int:
    return lib().mxq_moe_wgrad_b128(M, N, rows, E, offsets, x_codes, ld_x, x_scales, ld_xs, x_elem, w_codes, ld_w, w_scales,
                                    ld_ws, w_elem, accum, y, y_type, ld_y, expert_y, stream)


def mxq_gemm_b128_plan(mode: int, M: int, N: int, K: int, E: int, w_block: int, accum: int, cus: int) -> tuple:
    """(tile_m, tile_n, waves) of a product in blocks of 128 on `cus` CUs (host logic only); raises MxqError."""
    out = [ctypes.c_int() for _ in range(3)]
    _check(lib().mxq_gemm_b128_plan(mode, M, N, K, E, w_block, accum, cus, *[ctypes.byref(v) for v in out]),
           "mxq_gemm_b128_plan")
    return tuple(v.value for v in out)


def mxq_moe_route_workspace(T: int, E: int, k: int) -> int:
    """Bytes of workspace that mxq_moe_route needs (host logic only); raises MxqError."""
    n = ctypes.c_int64()
    _check(lib().mxq_moe_route_workspace(T, E, k, ctypes.byref(n)), "mxq_moe_route_workspace")
    return n.value


def mxq_moe_route(T, E, k, renormalize, logits, logits_type, ld_logits, mask, experts, shares, counts, offsets, order, loss,
                  slope, workspace, workspace_bytes, stream=None) -> int:
    return lib().mxq_moe_route(T, E, k, renormalize, logits, logits_type, ld_logits, mask, experts, shares, counts, offsets,
                               order, loss, slope, workspace, workspace_bytes, stream)


def mxq_moe_route_grad(T, E, k, renormalize, logits, logits_type, ld_logits, mask, experts, shares, slope, d_shares,
                       ld_d_shares, d_loss, d_logits, ld_d_logits, stream=None) -> int:
    return lib().mxq_moe_route_grad(T, E, k, renormalize, logits, logits_type, ld_logits, mask, experts, shares, slope,
                                    d_shares, ld_d_shares, d_loss, d_logits, ld_d_logits, stream)


# ----------------------------------------------------------------- torch conveniences

def _torch():
    import torch
    return torch


def _stream_handle():
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise MxqError(status, where)


def _wide_type(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return MXQ_F32
    if t.dtype == torch.bfloat16:
        return MXQ_BF16
    raise TypeError("expected a float32 or bfloat16 tensor, got %s" % t.dtype)


def _round_up(v: int, m: int) -> int:
    return (v + m - 1) // m * m


# Argument checks of the torch conveniences.  The C ABI sees only pointers, so an
# undersized or host-resident tensor would reach a kernel as an out-of-bounds or host
# address; these checks run first and raise ValueError.  Dtype and shape are checked
# before the device, so every rejection can be exercised without a GPU.

def _req_2d(t, name: str, dtype=None, min_rows=None, min_cols=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape[0] > 1 and t.shape[1] > 0 and t.stride(1) != 1:
        raise ValueError("%s must have unit stride along its last dimension" % name)
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError("%s rows overlap (row stride %d < %d columns)" % (name, t.stride(0), t.shape[1]))
    if min_rows is not None and t.shape[0] < min_rows:
        raise ValueError("%s has %d rows, needs at least %d" % (name, t.shape[0], min_rows))
    if min_cols is not None and t.shape[1] < min_cols:
        raise ValueError("%s has %d columns, needs at least %d" % (name, t.shape[1], min_cols))


def _req_cuda(*named):
    for name, t in named:
        if t is not None and not t.is_cuda:
            raise ValueError("%s must be a CUDA (HIP device) tensor, got device %s" % (name, t.device))


def _req_wide(t, name: str):
    torch = _torch()
    _req_2d(t, name)
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))


def _ld(t) -> int:
    """Leading dimension passed to the ABI: the row stride, or the width where the stride
    says nothing about the layout (no rows, or a single row of a broadcast view)."""
    return t.stride(0) if t.shape[0] > 0 and t.stride(0) >= t.shape[1] else max(t.shape[1], 1)


def quantize(x, elem: str = "e4m3", axis="row", codes=None, scales=None, rule: str = "ceil"):
    """MX-quantize a 2-D bf16/fp32 CUDA tensor.

    axis="row": 1x32 groups along each row -> codes [rows][Kp], scales [rows][Kp/32].
    axis="col": 32x1 groups down each column, stored transposed -> codes [cols][Kp],
                scales [cols][Kp/32] (K = rows).
    Codes are uint8 OCP bytes; scales are uint8 E8M0 bytes.  Optional preallocated
    outputs may be wider than Kp (their row stride is passed as the leading dimension).
    Scales allocated here are a [L][Kp/32] view of rows padded to a multiple of 16 bytes,
    the layout the fastest GEMM kernel reads.
    rule="ceil": the pages' scale rule (mxq_quantize); rule="ocp": the OCP MX
    specification's (floor(log2 amax) - emax, satfinite codes), via mxq_quantize_rule.
    """
    torch = _torch()
    _req_wide(x, "x")
    if axis not in _AXIS or elem not in _ELEM:
        raise ValueError("axis must be 'row' or 'col' and elem 'e4m3' or 'e5m2'")
    if rule not in _RULE:
        raise ValueError("rule must be 'ceil' or 'ocp'")
    rows, cols = x.shape
    ax = _AXIS[axis]
    L, K = (rows, cols) if ax == MXQ_ROWWISE else (cols, rows)
    Kp = _round_up(K, 32)
    nb = Kp // 32
    if codes is not None:
        _req_2d(codes, "codes", torch.uint8, L, Kp)
    if scales is not None:
        _req_2d(scales, "scales", torch.uint8, L, nb)
    _req_cuda(("x", x), ("codes", codes), ("scales", scales))
    if codes is None:
        codes = torch.empty((L, Kp), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((L, _round_up(nb, 16)), dtype=torch.uint8, device=x.device)[:, :nb]
    if rule == "ceil":
        st = mxq_quantize(x.data_ptr(), _wide_type(x), rows, cols, _ld(x), ax,
                          _ELEM[elem], codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales),
                          _stream_handle())
        _check(st, "mxq_quantize")
    else:
        st = mxq_quantize_rule(x.data_ptr(), _wide_type(x), rows, cols, _ld(x), ax, _ELEM[elem],
                               _RULE[rule], codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales),
                               _stream_handle())
        _check(st, "mxq_quantize_rule")
    return codes, scales


def quantize_sr(x, seed: int, elem: str = "e5m2", axis: str = "row", codes=None, scales=None):
    """quantize() with stochastically rounded codes (Philox4x32-10 keyed by `seed`, see
    mxq_quantize_sr); E5M2 by default, the gradient format."""
    torch = _torch()
    _req_wide(x, "x")
    if axis not in ("row", "col") or elem not in _ELEM:
        raise ValueError("axis must be 'row' or 'col' and elem 'e4m3' or 'e5m2'")
    rows, cols = x.shape
    L, K = (rows, cols) if axis == "row" else (cols, rows)
    Kp = _round_up(K, 32)
    if codes is not None:
        _req_2d(codes, "codes", torch.uint8, L, Kp)
    if scales is not None:
        _req_2d(scales, "scales", torch.uint8, L, Kp // 32)
    _req_cuda(("x", x), ("codes", codes), ("scales", scales))
    if codes is None:
        codes = torch.empty((L, Kp), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((L, _round_up(Kp // 32, 16)), dtype=torch.uint8, device=x.device)[:, :Kp // 32]
    st = mxq_quantize_sr(x.data_ptr(), _wide_type(x), rows, cols, _ld(x),
                         MXQ_ROWWISE if axis == "row" else MXQ_COLWISE, _ELEM[elem], int(seed) & (2 ** 64 - 1),
                         codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales), _stream_handle())
    _check(st, "mxq_quantize_sr")
    return codes, scales


def quantize_scaled(x, scales, elem: str = "e4m3", axis: str = "row", diagnostics: bool = True):
    """Quantize with caller-owned E8M0 scale bytes `scales` [L][nb] (uint8 CUDA tensor).

    Returns codes [L][Kp], or (codes, amax [L][nb] float32, clipped [L][nb] uint8,
    flushed [L][nb] uint8) with diagnostics=True (see mxq_quantize_scaled)."""
    torch = _torch()
    _req_wide(x, "x")
    if axis not in ("row", "col") or elem not in _ELEM:
        raise ValueError("axis must be 'row' or 'col' and elem 'e4m3' or 'e5m2'")
    rows, cols = x.shape
    L, K = (rows, cols) if axis == "row" else (cols, rows)
    Kp = _round_up(K, 32)
    nb = Kp // 32
    _req_2d(scales, "scales", torch.uint8)
    if tuple(scales.shape) != (L, nb):
        raise ValueError("scales must be a uint8 [L][nb] = [%d][%d] tensor, got %s" % (L, nb, tuple(scales.shape)))
    _req_cuda(("x", x), ("scales", scales))
    codes = torch.empty((L, Kp), dtype=torch.uint8, device=x.device)
    amax = clipped = flushed = None
    if diagnostics:
        amax = torch.empty((L, nb), dtype=torch.float32, device=x.device)
        clipped = torch.empty((L, nb), dtype=torch.uint8, device=x.device)
        flushed = torch.empty((L, nb), dtype=torch.uint8, device=x.device)
    st = mxq_quantize_scaled(x.data_ptr(), _wide_type(x), rows, cols, _ld(x),
                             MXQ_ROWWISE if axis == "row" else MXQ_COLWISE, _ELEM[elem], scales.data_ptr(),
                             scales.stride(0) if L > 0 else nb, codes.data_ptr(), codes.stride(0),
                             None if amax is None else amax.data_ptr(), nb,
                             None if clipped is None else clipped.data_ptr(),
                             None if flushed is None else flushed.data_ptr(), nb, _stream_handle())
    _check(st, "mxq_quantize_scaled")
    return (codes, amax, clipped, flushed) if diagnostics else codes


def quantize_dual(x, elem: str = "e4m3"):
    """Both MX orientations of a 2-D bf16/fp32 CUDA tensor from one read of it.

    Returns (row_codes [rows][Kp_r], row_scales [rows][Kp_r/32], col_codes [cols][Kp_c],
    col_scales [cols][Kp_c/32]) with K_r = cols and K_c = rows; identical to
    quantize(x, elem, "row") and quantize(x, elem, "col").
    """
    torch = _torch()
    _req_wide(x, "x")
    if elem not in _ELEM:
        raise ValueError("elem must be 'e4m3' or 'e5m2'")
    _req_cuda(("x", x))
    rows, cols = x.shape
    kp_r, kp_c = _round_up(cols, 32), _round_up(rows, 32)
    rc = torch.empty((rows, kp_r), dtype=torch.uint8, device=x.device)
    rs = torch.empty((rows, _round_up(kp_r // 32, 16)), dtype=torch.uint8, device=x.device)[:, :kp_r // 32]
    cc = torch.empty((cols, kp_c), dtype=torch.uint8, device=x.device)
    cs = torch.empty((cols, _round_up(kp_c // 32, 16)), dtype=torch.uint8, device=x.device)[:, :kp_c // 32]
    st = mxq_quantize_dual(x.data_ptr(), _wide_type(x), rows, cols, _ld(x), _ELEM[elem],
                           rc.data_ptr(), rc.stride(0), rs.data_ptr(), rs.stride(0), cc.data_ptr(), cc.stride(0),
                           cs.data_ptr(), cs.stride(0), _stream_handle())
    _check(st, "mxq_quantize_dual")
    return rc, rs, cc, cs


def dequantize(codes, scales, K: int, elem: str = "e4m3", out_dtype=None):
    """Reconstruct dec(code) * 2^(s-127) as fp32 (default) or bf16, shape [L][K]."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    if out_dtype not in (torch.float32, torch.bfloat16) or elem not in _ELEM:
        raise ValueError("out_dtype must be float32 or bfloat16 and elem 'e4m3' or 'e5m2'")
    if K < 0:
        raise ValueError("K must be >= 0")
    _req_2d(codes, "codes", torch.uint8, None, K)
    L = codes.shape[0]
    _req_2d(scales, "scales", torch.uint8, L, (K + 31) // 32)
    _req_cuda(("codes", codes), ("scales", scales))
    dst = torch.empty((L, K), dtype=out_dtype, device=codes.device)
    st = mxq_dequantize(codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales), _ELEM[elem], L, K,
                        dst.data_ptr(), _wide_type(dst), max(K, 1), _stream_handle())
    _check(st, "mxq_dequantize")
    return dst


def gemm(x_codes, x_scales, w_codes, w_scales, K: int, x_elem: str = "e4m3", w_elem: str = "e4m3",
         alpha: float = 1.0, bias=None, out_dtype=None, out=None, accum: str = "fp32", act=None,
         quant_out=None, wide_out: bool = True):
    """Y[M][N] = act(alpha * (X W) + bias) with X = (x_codes [M][Kp], x_scales) and W column-major
    (w_codes [N][Kp], w_scales).  accum="fp32" (default): exact products summed in FP32, the
    mode that meets |Y - Y_ref| <= 1e-5 * sum_k |s x w|; accum="fp8": the FP8 matrix cores,
    faster, but each group of 8 products is truncated ~13 bits below its largest, outside
    that bound (see mxq_accum in include/mxq.h).  act: None or "silu".

    quant_out="e4m3"/"e5m2" also returns the MX codes [M][Np] and scales of bf16(Y) along
    N, produced in the GEMM's epilogue (byte for byte quantize(Y_bf16, elem, "row"));
    wide_out=False then skips writing Y.  Returns Y, or (Y or None, codes, scales)."""
    torch = _torch()
    if K < 0:
        raise ValueError("K must be >= 0")
    Kp = _round_up(K, 32)
    nb = Kp // 32
    _req_2d(x_codes, "x_codes", torch.uint8, None, Kp)
    _req_2d(w_codes, "w_codes", torch.uint8, None, Kp)
    M, N = x_codes.shape[0], w_codes.shape[0]
    _req_2d(x_scales, "x_scales", torch.uint8, M, nb)
    _req_2d(w_scales, "w_scales", torch.uint8, N, nb)
    if x_elem not in _ELEM or w_elem not in _ELEM or (quant_out is not None and quant_out not in _ELEM):
        raise ValueError("element formats must be 'e4m3' or 'e5m2'")
    if accum not in _ACC:
        raise ValueError("accum must be 'fp32' or 'fp8'")
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype != torch.float32 or bias.numel() != N \
                or (N > 1 and bias.stride(-1) != 1) or bias.dim() != 1:
            raise ValueError("bias must be a contiguous 1-D float32 tensor of N = %d elements" % N)
    if act not in _ACT:
        raise ValueError("act must be None or 'silu'")
    if quant_out is None and not wide_out:
        raise ValueError("nothing to write: wide_out=False needs quant_out")
    if wide_out and out is not None:
        _req_wide(out, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out must have shape (M, N) = (%d, %d), got %s" % (M, N, tuple(out.shape)))
    _req_cuda(("x_codes", x_codes), ("x_scales", x_scales), ("w_codes", w_codes), ("w_scales", w_scales),
              ("bias", bias), ("out", out if wide_out else None))
    if wide_out and out is None:
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=x_codes.device)
    y = out if wide_out else None
    qc = qs = None
    if quant_out is not None:
        np_ = _round_up(N, 32)
        qc = torch.empty((M, np_), dtype=torch.uint8, device=x_codes.device)
        qs = torch.empty((M, _round_up(np_ // 32, 16)), dtype=torch.uint8, device=x_codes.device)[:, :np_ // 32]
    st = mxq_gemm_ex(M, N, K, x_codes.data_ptr(), _ld(x_codes), x_scales.data_ptr(), _ld(x_scales),
                     _ELEM[x_elem], w_codes.data_ptr(), _ld(w_codes), w_scales.data_ptr(), _ld(w_scales),
                     _ELEM[w_elem], float(alpha), None if bias is None else bias.data_ptr(), _ACT[act],
                     None if y is None else y.data_ptr(), MXQ_BF16 if y is None else _wide_type(y),
                     0 if y is None else _ld(y), _ELEM[quant_out or "e4m3"],
                     None if qc is None else qc.data_ptr(), 0 if qc is None else _ld(qc),
                     None if qs is None else qs.data_ptr(), 0 if qs is None else _ld(qs),
                     _ACC[accum], _stream_handle())
    _check(st, "mxq_gemm_ex")
    if quant_out is None:
        return y
    return y, qc, qs
