"""The MXFP4 operators on torch tensors: quantize, dequantize, product and the
mixture-of-experts layer (the ``mxq_*_fp4`` entry points of include/mxq.h).  Argument checks
and marshalling only, like ``_binding``; every call raises if the library is missing."""
from __future__ import annotations

import functools

import torch

from ._binding import (_ACT, _AXIS, _RULE, MXQ_BF16, MXQ_COLWISE, MXQ_E2M1, MXQ_F32, MxqError, _req_2d,
                       _req_wide, lib, mxq_moe_fp4_workspace)

_WIDE = {torch.float32: MXQ_F32, torch.bfloat16: MXQ_BF16}
_U8 = torch.uint8
_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice
_entry = {}


def _call(name: str, device: int, args: tuple) -> None:
    """The library's entry point `name` on torch's current stream of the device."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(lib(), name)
    if device == _current():
        status = fn(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream(device))
    if status != 0:
        raise MxqError(status, name)


# These calls are short, so the checks read few attributes, once each: what is wrong is found here, and
# _req_2d says what it is.  (torch.empty_strided is the quickest of torch's allocating calls.)
_empty = torch.empty_strided


def _lines(t, name: str, dtype, rows: int, cols: int) -> int:
    """Checks rows of at least `cols` elements, `rows` of them at least; the row pitch."""
    try:
        r, c = t.shape
        pitch, step = t.stride()
        if step == 1 and pitch >= c >= cols and r >= rows and t.dtype is dtype and c > 0 and r > 0:
            return pitch
    except (AttributeError, TypeError, ValueError):
        pass
    # no rows, one row or one column, or something wrong
    _req_2d(t, name, dtype, rows, cols)
    if step != 1 and c > 1 and r > 0:
        raise ValueError("%s must have unit stride along its last dimension" % name)
    return pitch if r > 0 and pitch >= c else max(c, 1)


def _same_device(named: tuple) -> int:
    """The index of the device that holds every given tensor: the slow way, which finds what is wrong."""
    first = named[0][1]
    for name, t in named:
        if t is not None and t.get_device() < 0:
            raise ValueError("%s must be a CUDA (HIP device) tensor, got device %s" % (name, t.device))
        if t is not None and t.get_device() != first.get_device():
            raise ValueError("%s is on %s, expected %s" % (name, t.device, first.device))
    return first.get_device()


def _wide(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in _WIDE:
        _req_wide(t, name)
    return _lines(t, name, t.dtype, 0, 0)


def _code_array(lines: int, k: int, device):
    """Empty codes [lines][16 * blocks] and scales [lines][blocks] and their pitches, the scale rows
    padded to 16 bytes (the layout that the product reads fastest)."""
    nb = (k + 31) // 32
    wide, pitch = max(16 * nb, 1), max((nb + 15) // 16 * 16, 1)
    return (_empty((lines, 16 * nb), (wide, 1), dtype=_U8, device=device), wide,
            _empty((lines, nb), (pitch, 1), dtype=_U8, device=device), pitch)


def _orient(x, axis, codes, scales):
    """What the one-orientation quantizers share: sizes and pitch of x, axis tag, device, outputs."""
    ld = _wide(x, "x")
    ax = _AXIS.get(axis)
    if ax is None:
        raise ValueError("axis must be 'row' or 'col'")
    rows, cols = x.shape
    L, K = (cols, rows) if ax == MXQ_COLWISE else (rows, cols)
    nb = (K + 31) // 32
    ld_c = None if codes is None else _lines(codes, "codes", _U8, L, 16 * nb)
    ld_s = None if scales is None else _lines(scales, "scales", _U8, L, nb)
    device = x.get_device()
    if device < 0 or (codes is not None and codes.get_device() != device) or \
            (scales is not None and scales.get_device() != device):
        _same_device((("x", x), ("codes", codes), ("scales", scales)))
    if codes is None or scales is None:
        c, pitch_c, s, pitch_s = _code_array(L, K, x.device)
        if codes is None:
            codes, ld_c = c, pitch_c
        if scales is None:
            scales, ld_s = s, pitch_s
    return rows, cols, ld, ax, device, codes, ld_c, scales, ld_s


def quantize_fp4(x, axis="row", codes=None, scales=None, rule: str = "ceil"):
    """MXFP4-quantize a 2-D bf16/fp32 CUDA tensor.

    axis="row": 1x32 blocks along each row -> codes [rows][16 nb], scales [rows][nb];
    axis="col": 32x1 blocks down each column, stored transposed -> codes [cols][16 nb],
    scales [cols][nb].  A code byte holds two E2M1 codes, the even element in the low half;
    scales are E8M0 bytes.  rule "ceil" (no code saturates) or "ocp" (the MX specification's
    floor(log2 amax) - 2), see mxq_quantize_fp4.  Preallocated outputs may be wider.
    """
    if rule not in _RULE:
        raise ValueError("rule must be 'ceil' or 'ocp'")
    rows, cols, ld, ax, device, codes, ld_c, scales, ld_s = _orient(x, axis, codes, scales)
    _call("mxq_quantize_fp4", device, (x.data_ptr(), _WIDE[x.dtype], rows, cols, ld, ax, _RULE[rule],
                                       codes.data_ptr(), ld_c, scales.data_ptr(), ld_s))
    return codes, scales


def quantize_fp4_sr(x, seed: int, axis="row", codes=None, scales=None):
    """quantize_fp4() with stochastically rounded codes (Philox4x32-10 keyed by `seed`, see
    mxq_quantize_fp4_sr): for gradients."""
    rows, cols, ld, ax, device, codes, ld_c, scales, ld_s = _orient(x, axis, codes, scales)
    _call("mxq_quantize_fp4_sr", device, (x.data_ptr(), _WIDE[x.dtype], rows, cols, ld, ax, int(seed) & (2 ** 64 - 1),
                                          codes.data_ptr(), ld_c, scales.data_ptr(), ld_s))
    return codes, scales


def quantize_fp4_dual(x):
    """Both orientations of a 2-D bf16/fp32 CUDA tensor from one read of it: (row_codes,
    row_scales, col_codes, col_scales), as quantize_fp4(x, "row") and quantize_fp4(x, "col")."""
    ld = _wide(x, "x")
    device = x.get_device()
    if device < 0:
        _same_device((("x", x),))
    rows, cols = x.shape
    rc, ld_rc, rs, ld_rs = _code_array(rows, cols, x.device)
    cc, ld_cc, cs, ld_cs = _code_array(cols, rows, x.device)
    _call("mxq_quantize_fp4_dual", device, (x.data_ptr(), _WIDE[x.dtype], rows, cols, ld, rc.data_ptr(), ld_rc,
                                            rs.data_ptr(), ld_rs, cc.data_ptr(), ld_cc, cs.data_ptr(), ld_cs))
    return rc, rs, cc, cs


def dequantize_fp4(codes, scales, K: int, out_dtype=None):
    """Reconstruct code * 2^(s-127) as fp32 (default) or bf16, shape [L][K]."""
    out_dtype = out_dtype or torch.float32
    if out_dtype not in _WIDE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    if K < 0:
        raise ValueError("K must be >= 0")
    nb = (K + 31) // 32
    ld_c = _lines(codes, "codes", _U8, 0, 16 * nb)
    L = codes.shape[0]
    ld_s = _lines(scales, "scales", _U8, L, nb)
    device = codes.get_device()
    if device < 0 or scales.get_device() != device:
        _same_device((("codes", codes), ("scales", scales)))
    ld = max(K, 1)
    dst = _empty((L, K), (ld, 1), dtype=out_dtype, device=codes.device)
    _call("mxq_dequantize_fp4", device, (codes.data_ptr(), ld_c, scales.data_ptr(), ld_s, L, K, dst.data_ptr(),
                                         _WIDE[out_dtype], ld))
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
    nb = (K + 31) // 32
    ld_w = _lines(w_codes, "w_codes", _U8, 0, 16 * nb)
    N = w_codes.shape[0]
    ld_ws = _lines(w_scales, "w_scales", _U8, N, nb)
    if x_scales is None:
        ld_x = _lines(x, "x", torch.bfloat16, 0, K)
        M = x.shape[0]
        if x.shape[1] != K:
            raise ValueError("x has %d columns, expected K = %d" % (x.shape[1], K))
        x_type, xs_ptr, ld_xs = MXQ_BF16, None, 0
    else:
        ld_x = _lines(x, "x", _U8, 0, 16 * nb)
        M = x.shape[0]
        ld_xs = _lines(x_scales, "x_scales", _U8, M, nb)
        x_type, xs_ptr = MXQ_E2M1, x_scales.data_ptr()
    if bias is not None and (not isinstance(bias, torch.Tensor) or bias.dtype != torch.float32 or bias.dim() != 1
                             or bias.shape[0] != N or (N > 1 and bias.stride(0) != 1)):
        raise ValueError("bias must be a contiguous 1-D float32 tensor of N = %d elements" % N)
    if act not in _ACT:
        raise ValueError("act must be None or 'silu'")
    if out is not None:
        ld_y = _wide(out, "out")
        if tuple(out.shape) != (M, N):
            raise ValueError("out must have shape (M, N) = (%d, %d), got %s" % (M, N, tuple(out.shape)))
    elif out_dtype is not None and out_dtype not in _WIDE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    device = x.get_device()
    if device < 0 or w_codes.get_device() != device or w_scales.get_device() != device or \
            (x_scales is not None and x_scales.get_device() != device) or \
            (bias is not None and bias.get_device() != device) or (out is not None and out.get_device() != device):
        _same_device((("x", x), ("x_scales", x_scales), ("w_codes", w_codes), ("w_scales", w_scales), ("bias", bias),
                      ("out", out)))
    if out is None:
        out_dtype, ld_y = out_dtype or torch.bfloat16, max(N, 1)
        out = _empty((M, N), (ld_y, 1), dtype=out_dtype, device=x.device)
        y_type = _WIDE[out_dtype]
    else:
        y_type = _WIDE[out.dtype]
    _call("mxq_gemm_fp4", device, (M, N, K, x.data_ptr(), x_type, ld_x, xs_ptr, ld_xs, w_codes.data_ptr(), ld_w,
                                   w_scales.data_ptr(), ld_ws, alpha, None if bias is None else bias.data_ptr(), _ACT[act],
                                   out.data_ptr(), y_type, ld_y))
    return out


def _expert(t, name: str, experts: int, rows: int, cols: int):
    """Checks a stack of code or scale rows; the expert and row pitches."""
    try:
        e, r, c = t.shape
        far, pitch, step = t.stride()
        good = t.dtype is _U8
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        raise ValueError("%s must be a 3-D uint8 tensor" % name)
    if e != experts or r != rows or c < cols:
        raise ValueError("%s must have shape (%d, %d, >= %d), got %s" % (name, experts, rows, cols, tuple(t.shape)))
    if c > 1 and step != 1:
        raise ValueError("%s must have unit stride along its last dimension" % name)
    return far, pitch


@functools.lru_cache(maxsize=1024)
def _moe_workspace(device: int, T: int, H: int, I: int, E: int, k: int, y_type: int) -> int:
    """The plan, and with it the workspace, follows from the sizes and the device's CUs."""
    with torch.cuda.device(device):
        return mxq_moe_fp4_workspace(T, H, I, E, k, y_type)


def moe_fp4(x, logits, w13_codes, w13_scales, w2_codes, w2_scales, k: int, renormalize: bool = True, out_dtype=None,
            out=None):
    """A mixture-of-experts layer for a few tokens (up to 1024; made for tens), from the router's
    logits on: softmax, the k greatest, gate and up products, SiLU, down product, weighted sum.

    x [T][H] bf16, logits [T][E] fp32, w13 [E][2I][16 ceil(H/32)] (gate rows, then up rows, along
    H) and w2 [E][H][16 ceil(I/32)] (along I) MXFP4 codes with their scales [E][..][blocks].
    renormalize: the k shares sum to 1.  Returns [T][H] in out_dtype (bf16 by default, or fp32).
    See mxq_moe_fp4 for ties, masked experts and precision.
    """
    ld_x = _lines(x, "x", torch.bfloat16, 0, 0)
    ld_l = _lines(logits, "logits", torch.float32, 0, 0)
    (T, H), (rows, E) = x.shape, logits.shape
    if rows != T:
        raise ValueError("logits has %d rows, expected T = %d" % (rows, T))
    if not isinstance(w13_codes, torch.Tensor) or w13_codes.dim() != 3 or w13_codes.shape[1] % 2:
        raise ValueError("w13_codes must be a 3-D tensor with an even number of rows")
    I = w13_codes.shape[1] // 2
    if not 1 <= k <= E:
        raise ValueError("k must be between 1 and E = %d" % E)
    nb_h, nb_i = (H + 31) // 32, (I + 31) // 32
    e13, l13 = _expert(w13_codes, "w13_codes", E, 2 * I, 16 * nb_h)
    es13, ls13 = _expert(w13_scales, "w13_scales", E, 2 * I, nb_h)
    e2, l2 = _expert(w2_codes, "w2_codes", E, H, 16 * nb_i)
    es2, ls2 = _expert(w2_scales, "w2_scales", E, H, nb_i)
    if out is not None:
        ld_y = _wide(out, "out")
        if tuple(out.shape) != (T, H):
            raise ValueError("out must have shape (T, H) = (%d, %d), got %s" % (T, H, tuple(out.shape)))
    elif out_dtype is not None and out_dtype not in _WIDE:
        raise ValueError("out_dtype must be float32 or bfloat16")
    device = x.get_device()
    if device < 0 or logits.get_device() != device or w13_codes.get_device() != device or \
            w13_scales.get_device() != device or w2_codes.get_device() != device or \
            w2_scales.get_device() != device or (out is not None and out.get_device() != device):
        _same_device((("x", x), ("logits", logits), ("w13_codes", w13_codes), ("w13_scales", w13_scales),
                      ("w2_codes", w2_codes), ("w2_scales", w2_scales), ("out", out)))
    if out is None:
        out_dtype, ld_y = out_dtype or torch.bfloat16, max(H, 1)
        out = _empty((T, H), (ld_y, 1), dtype=out_dtype, device=x.device)
        y_type = _WIDE[out_dtype]
    else:
        y_type = _WIDE[out.dtype]
    need = _moe_workspace(device, T, H, I, E, k, y_type)
    workspace = _empty((need,), (1,), dtype=_U8, device=x.device)
    _call("mxq_moe_fp4", device, (T, H, I, E, k, 1 if renormalize else 0, x.data_ptr(), ld_x, logits.data_ptr(), ld_l,
                                  w13_codes.data_ptr(), l13, e13, w13_scales.data_ptr(), ls13, es13, w2_codes.data_ptr(),
                                  l2, e2, w2_scales.data_ptr(), ls2, es2, out.data_ptr(), y_type, ld_y,
                                  workspace.data_ptr(), need))
    return out
