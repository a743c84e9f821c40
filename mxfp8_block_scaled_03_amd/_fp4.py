"""The MXFP4 operators on torch tensors: quantize, dequantize, product and the
mixture-of-experts layer (the ``mxq_*_fp4`` entry points of include/mxq.h).  Argument checks
and marshalling only, like ``_binding``; every call raises if the library is missing."""
from __future__ import annotations

import ctypes

import torch

from ._binding import (_ACT, _AXIS, _RULE, MXQ_BF16, MXQ_COLWISE, MXQ_E2M1, MXQ_F32, MXQ_ROWWISE, MxqError, _ld,
                       _req_2d, _req_cuda, _req_wide, lib)

_WIDE = {torch.float32: MXQ_F32, torch.bfloat16: MXQ_BF16}


def _call(name: str, device, *args):
    """The library's entry point `name` on torch's current stream of `device`."""
    fn = getattr(lib(), name)
    if device.index == torch.cuda.current_device():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if status != 0:
        raise MxqError(status, name)


def _same_device(first, *named):
    for name, t in named:
        if t is not None and t.device != first.device:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, first.device))


def _blocks(k: int) -> int:
    return (k + 31) // 32


def _code_array(lines: int, k: int, device):
    """Empty codes [lines][16 * blocks] and scales [lines][blocks], the scale rows padded to 16
    bytes (the layout that the product reads fastest)."""
    nb = _blocks(k)
    return (torch.empty((lines, 16 * nb), dtype=torch.uint8, device=device),
            torch.empty((lines, (nb + 15) // 16 * 16), dtype=torch.uint8, device=device)[:, :nb])


def _outputs(x, lines: int, k: int, codes, scales):
    nb = _blocks(k)
    if codes is not None:
        _req_2d(codes, "codes", torch.uint8, lines, 16 * nb)
    if scales is not None:
        _req_2d(scales, "scales", torch.uint8, lines, nb)
    _req_cuda(("x", x), ("codes", codes), ("scales", scales))
    _same_device(x, ("codes", codes), ("scales", scales))
    if codes is None or scales is None:
        c, s = _code_array(lines, k, x.device)
        codes, scales = c if codes is None else codes, s if scales is None else scales
    return codes, scales


def quantize_fp4(x, axis="row", codes=None, scales=None, rule: str = "ceil"):
    """MXFP4-quantize a 2-D bf16/fp32 CUDA tensor.

    axis="row": 1x32 blocks along each row -> codes [rows][16 nb], scales [rows][nb];
    axis="col": 32x1 blocks down each column, stored transposed -> codes [cols][16 nb],
    scales [cols][nb].  A code byte holds two E2M1 codes, the even element in the low half;
    scales are E8M0 bytes.  rule "ceil" (no code saturates) or "ocp" (the MX specification's
    floor(log2 amax) - 2), see mxq_quantize_fp4.  Preallocated outputs may be wider.
    """
    _req_wide(x, "x")
    if axis not in _AXIS:
        raise ValueError("axis must be 'row' or 'col'")
    if rule not in _RULE:
        raise ValueError("rule must be 'ceil' or 'ocp'")
    rows, cols = x.shape
    ax = _AXIS[axis]
    L, K = (rows, cols) if ax == MXQ_ROWWISE else (cols, rows)
    codes, scales = _outputs(x, L, K, codes, scales)
    _call("mxq_quantize_fp4", x.device, x.data_ptr(), _WIDE[x.dtype], rows, cols, _ld(x), ax, _RULE[rule],
          codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales))
    return codes, scales


def quantize_fp4_sr(x, seed: int, axis="row", codes=None, scales=None):
    """quantize_fp4() with stochastically rounded codes (Philox4x32-10 keyed by `seed`, see
    mxq_quantize_fp4_sr): for gradients."""
    _req_wide(x, "x")
    if axis not in _AXIS:
        raise ValueError("axis must be 'row' or 'col'")
    rows, cols = x.shape
    ax = _AXIS[axis]
    L, K = (rows, cols) if ax == MXQ_ROWWISE else (cols, rows)
    codes, scales = _outputs(x, L, K, codes, scales)
    _call("mxq_quantize_fp4_sr", x.device, x.data_ptr(), _WIDE[x.dtype], rows, cols, _ld(x), ax,
          int(seed) & (2 ** 64 - 1), codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales))
    return codes, scales


def quantize_fp4_dual(x):
    """Both orientations of a 2-D bf16/fp32 CUDA tensor from one read of it: (row_codes,
    row_scales, col_codes, col_scales), as quantize_fp4(x, "row") and quantize_fp4(x, "col")."""
    _req_wide(x, "x")
    _req_cuda(("x", x))
    rows, cols = x.shape
    rc, rs = _code_array(rows, cols, x.device)
    cc, cs = _code_array(cols, rows, x.device)
    _call("mxq_quantize_fp4_dual", x.device, x.data_ptr(), _WIDE[x.dtype], rows, cols, _ld(x), rc.data_ptr(), _ld(rc),
          rs.data_ptr(), _ld(rs), cc.data_ptr(), _ld(cc), cs.data_ptr(), _ld(cs))
    return rc, rs, cc, cs


def dequantize_fp4(codes, scales, K: int, out_dtype=None):
    """Reconstruct code * 2^(s-127) as fp32 (default) or bf16, shape [L][K]."""
    out_dtype = out_dtype or torch.float32
    if out_dtype not in _WIDE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    if K < 0:
        raise ValueError("K must be >= 0")
    _req_2d(codes, "codes", torch.uint8, None, 16 * _blocks(K))
    L = codes.shape[0]
    _req_2d(scales, "scales", torch.uint8, L, _blocks(K))
    _req_cuda(("codes", codes), ("scales", scales))
    _same_device(codes, ("scales", scales))
    dst = torch.empty((L, K), dtype=out_dtype, device=codes.device)
    _call("mxq_dequantize_fp4", codes.device, codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales), L, K,
          dst.data_ptr(), _WIDE[out_dtype], max(K, 1))
    return dst


def gemm_fp4(x, x_scales, w_codes, w_scales, K: int, alpha: float = 1.0, bias=None, out_dtype=None, out=None,
             act=None):
    """Y[M][N] = act(alpha * (X W) + bias), W in MXFP4 (w_codes [N][16 nb], w_scales [N][nb], K
    contiguous).  X is MXFP4 (x [M][16 nb] uint8 and x_scales [M][nb]) or, with x_scales=None,
    bf16 [M][K].  FP32 sums of exact products (see mxq_gemm_fp4).  act: None or "silu";
    out_dtype bf16 (default) or fp32, or a preallocated `out`.
    """
    if K < 0:
        raise ValueError("K must be >= 0")
    nb = _blocks(K)
    _req_2d(w_codes, "w_codes", torch.uint8, None, 16 * nb)
    N = w_codes.shape[0]
    _req_2d(w_scales, "w_scales", torch.uint8, N, nb)
    if x_scales is None:
        _req_2d(x, "x", torch.bfloat16)
        if x.shape[1] != K:
            raise ValueError("x has %d columns, expected K = %d" % (x.shape[1], K))
        M = x.shape[0]
    else:
        _req_2d(x, "x", torch.uint8, None, 16 * nb)
        M = x.shape[0]
        _req_2d(x_scales, "x_scales", torch.uint8, M, nb)
    if bias is not None and (not isinstance(bias, torch.Tensor) or bias.dtype != torch.float32 or bias.dim() != 1
                             or bias.shape[0] != N or (N > 1 and bias.stride(0) != 1)):
        raise ValueError("bias must be a contiguous 1-D float32 tensor of N = %d elements" % N)
    if act not in _ACT:
        raise ValueError("act must be None or 'silu'")
    if out is not None:
        _req_wide(out, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out must have shape (M, N) = (%d, %d), got %s" % (M, N, tuple(out.shape)))
    elif out_dtype is not None and out_dtype not in _WIDE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    _req_cuda(("x", x), ("x_scales", x_scales), ("w_codes", w_codes), ("w_scales", w_scales), ("bias", bias),
              ("out", out))
    _same_device(x, ("x_scales", x_scales), ("w_codes", w_codes), ("w_scales", w_scales), ("bias", bias), ("out", out))
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=x.device)
    _call("mxq_gemm_fp4", x.device, M, N, K, x.data_ptr(), MXQ_BF16 if x_scales is None else MXQ_E2M1, _ld(x),
          None if x_scales is None else x_scales.data_ptr(), 0 if x_scales is None else _ld(x_scales),
          w_codes.data_ptr(), _ld(w_codes), w_scales.data_ptr(), _ld(w_scales), float(alpha),
          None if bias is None else bias.data_ptr(), _ACT[act], out.data_ptr(), _WIDE[out.dtype], _ld(out))
    return out


def _req_expert(t, name: str, experts: int, rows: int, cols: int):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.dim() != 3:
        raise ValueError("%s must be a 3-D uint8 tensor" % name)
    if t.shape[0] != experts or t.shape[1] != rows or t.shape[2] < cols:
        raise ValueError("%s must have shape (%d, %d, >= %d), got %s" % (name, experts, rows, cols, tuple(t.shape)))
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError("%s must have unit stride along its last dimension" % name)


def moe_fp4(x, logits, w13_codes, w13_scales, w2_codes, w2_scales, k: int, renormalize: bool = True, out_dtype=None,
            out=None):
    """A mixture-of-experts layer for a few tokens (up to 1024; made for tens), from the router's
    logits on: softmax, the k greatest, gate and up products, SiLU, down product, weighted sum.

    x [T][H] bf16, logits [T][E] fp32, w13 [E][2I][16 ceil(H/32)] (gate rows, then up rows, along
    H) and w2 [E][H][16 ceil(I/32)] (along I) MXFP4 codes with their scales [E][..][blocks].
    renormalize: the k shares sum to 1.  Returns [T][H] in out_dtype (bf16 by default, or fp32).
    See mxq_moe_fp4 for ties, masked experts and precision.
    """
    _req_2d(x, "x", torch.bfloat16)
    _req_2d(logits, "logits", torch.float32)
    (T, H), E = x.shape, logits.shape[1]
    if logits.shape[0] != T:
        raise ValueError("logits has %d rows, expected T = %d" % (logits.shape[0], T))
    if not isinstance(w13_codes, torch.Tensor) or w13_codes.dim() != 3 or w13_codes.shape[1] % 2:
        raise ValueError("w13_codes must be a 3-D tensor with an even number of rows")
    I = w13_codes.shape[1] // 2
    if not 1 <= k <= E:
        raise ValueError("k must be between 1 and E = %d" % E)
    _req_expert(w13_codes, "w13_codes", E, 2 * I, 16 * _blocks(H))
    _req_expert(w13_scales, "w13_scales", E, 2 * I, _blocks(H))
    _req_expert(w2_codes, "w2_codes", E, H, 16 * _blocks(I))
    _req_expert(w2_scales, "w2_scales", E, H, _blocks(I))
    if out is not None:
        _req_wide(out, "out")
        if tuple(out.shape) != (T, H):
            raise ValueError("out must have shape (T, H) = (%d, %d), got %s" % (T, H, tuple(out.shape)))
    elif out_dtype is not None and out_dtype not in _WIDE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    named = (("logits", logits), ("w13_codes", w13_codes), ("w13_scales", w13_scales), ("w2_codes", w2_codes),
             ("w2_scales", w2_scales), ("out", out))
    _req_cuda(("x", x), *named)
    _same_device(x, *named)
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype or torch.bfloat16, device=x.device)
    y_type = _WIDE[out.dtype]
    need = ctypes.c_int64()
    status = lib().mxq_moe_fp4_workspace(T, H, I, E, k, y_type, ctypes.byref(need))
    if status != 0:
        raise MxqError(status, "mxq_moe_fp4_workspace")
    workspace = torch.empty((max(need.value, 1),), dtype=torch.uint8, device=x.device)
    _call("mxq_moe_fp4", x.device, T, H, I, E, k, 1 if renormalize else 0, x.data_ptr(), _ld(x), logits.data_ptr(),
          _ld(logits), w13_codes.data_ptr(), w13_codes.stride(1), w13_codes.stride(0), w13_scales.data_ptr(),
          w13_scales.stride(1), w13_scales.stride(0), w2_codes.data_ptr(), w2_codes.stride(1), w2_codes.stride(0),
          w2_scales.data_ptr(), w2_scales.stride(1), w2_scales.stride(0), out.data_ptr(), y_type, _ld(out),
          workspace.data_ptr(), need.value)
    return out
