"""FP8 in blocks of 128 with FP32 scales, and expert routing, on torch tensors (the ``*_b128`` and
``mxq_moe_route*`` entry points of include/mxq.h).  Argument checks and marshalling only, like
``_binding``; every call raises if the library is missing.

Codes are uint8 [lines][128 * blocks]; scales float32 [lines][blocks] (a tile's: [tiles][blocks]),
those of lines stored block by block (stride 1 along the lines), as the quantizer gives them.

A product forms the product of two scales in FP32, which should lie inside its normal range: past it a
block whose sum is 0 gives NaN, below it bits are lost.  It multiplies whole blocks: codes past K that
the quantizer did not write have to be zero for one operand and finite for the other."""
from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from ._binding import _ACC, _ACT, _ELEM, MXQ_SCALE_AMAX, MXQ_SCALE_CEIL, mxq_moe_route_workspace
from ._fp4 import _WIDE, _call, _empty, _lines, _same_device, _U8, _wide

B = 128
_RULES = {"amax": MXQ_SCALE_AMAX, "ceil": MXQ_SCALE_CEIL}
_F32, _I32, _BF16 = torch.float32, torch.int32, torch.bfloat16


def _blocks(k: int) -> int:
    return (k + B - 1) // B


def _elem(name: str, *elems) -> None:
    for e in elems:
        if e not in _ELEM:
            raise ValueError("%s must be 'e4m3' or 'e5m2'" % name)


def _offsets(t) -> int:
    """Checks expert offsets; the number of experts."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _I32 or t.dim() != 1 or t.shape[0] < 2 or t.stride(0) != 1:
        raise ValueError("offsets must be a contiguous 1-D int32 tensor of E + 1 elements")
    return t.shape[0] - 1


# These calls are short, as those of _fp4 are: what is needed is read once, and the slow ways only find what is wrong.

def _devices(x, *named) -> int:
    """The device of x, which all given tensors have to be on."""
    device = x.get_device()
    for _, t in named:
        if t is not None and t.get_device() != device:
            device = -1
    if device < 0:
        _same_device((("the first tensor", x),) + named)
    return device


def _line_scales(t, name: str, lines: int, nb: int) -> int:
    """Checks scales of lines; the pitch from block to block."""
    try:
        n, b = t.shape
        step, pitch = t.stride()
        if n == lines and b >= nb > 1 and step == 1 and pitch >= n > 1 and t.dtype is _F32:
            return pitch
    except (AttributeError, TypeError, ValueError):
        pass
    # one line, one block or none, or something wrong
    if not isinstance(t, torch.Tensor) or t.dtype is not _F32 or t.dim() != 2:
        raise ValueError("%s must be a 2-D float32 tensor" % name)
    if t.shape[0] != lines or t.shape[1] < nb:
        raise ValueError("%s must have shape (%d, >= %d), got %s" % (name, lines, nb, tuple(t.shape)))
    step, pitch = t.stride()
    if lines > 1 and nb > 0 and step != 1:
        raise ValueError("%s must be stored block by block (stride 1 along the lines)" % name)
    if nb > 1 and pitch < lines:
        raise ValueError("%s has overlapping blocks" % name)
    return pitch if nb > 1 else max(lines, 1)


def _weight_scales(t, name: str, lines: int, nb: int, line_dim: int = 0):
    """Checks scales of lines or of tiles, by their number; (block, line or tile stride, block stride)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _F32 or t.dim() != 2 + line_dim:
        raise ValueError("%s must be a %d-D float32 tensor" % (name, 2 + line_dim))
    n, b = t.shape[-2:]
    if (n != lines and n != _blocks(lines)) or b < nb:
        raise ValueError("%s must have %d (lines) or %d (tiles) rows and at least %d columns, got %s"
                         % (name, lines, _blocks(lines), nb, tuple(t.shape)))
    step, pitch = t.stride()[-2:]
    if n != lines:
        return B, step, pitch
    if lines > 1 and nb > 0 and step != 1:
        raise ValueError("%s must be stored block by block (stride 1 along the lines)" % name)
    return 1, 1, pitch if nb > 1 else max(lines, 1)


def _code_lines(lines: int, nb: int, device):
    return _empty((lines, B * nb), (max(B * nb, 1), 1), dtype=_U8, device=device)


def _scale_lines(lines: int, nb: int, device):
    return _empty((lines, nb), (1, max(lines, 1)), dtype=_F32, device=device)


def _rule(rule: str) -> int:
    if rule not in _RULES:
        raise ValueError("rule must be 'amax' or 'ceil'")
    return _RULES[rule]




def quantize_b128(x, elem: str = "e4m3", axis: str = "row", rule: str = "amax", offsets=None):
    """FP8-quantize a 2-D bf16/fp32 CUDA tensor in blocks of 128: (codes, scales).

    axis="row": blocks along each row -> codes [rows][128 nb], scales [rows][nb];
    axis="col": blocks down each column, transposed -> codes [cols][128 nb], scales [cols][nb];
    axis="tile": tiles of 128 x 128 -> codes [rows][128 nb], scales [ceil(rows/128)][nb].
    rule "amax": scale amax / fmax; "ceil": that rounded up to a power of two.  offsets (int32
    [E + 1], axis="col"): blocks begin anew with every expert's rows; rows past the last
    expert's are skipped.  See mxq_quantize_b128.
    """
    ld = _wide(x, "x")
    _elem("elem", elem)
    r = _rule(rule)
    if axis not in ("row", "col", "tile"):
        raise ValueError("axis must be 'row', 'col' or 'tile'")
    experts, off = 1, None
    if offsets is not None:
        if axis != "col":
            raise ValueError("offsets need axis='col'")
        experts, off = _offsets(offsets), offsets.data_ptr()
    device = x.get_device()
    if device < 0 or (offsets is not None and offsets.get_device() != device):
        _devices(x, ("offsets", offsets))
    rows, cols = x.shape
    where, head = x.device, (x.data_ptr(), _WIDE[x.dtype], rows, cols, ld, _ELEM[elem], r)
    if axis == "row":
        nb = (cols + (B - 1)) // B
        c, s = _code_lines(rows, nb, where), _scale_lines(rows, nb, where)
        args = head + (0, c.data_ptr(), B * nb, s.data_ptr(), rows, None, 0, None, 0, None, 1)
    elif axis == "col":
        nb = (rows + (B - 1) * experts) // B
        c, s = _code_lines(cols, nb, where), _scale_lines(cols, nb, where)
        args = head + (0, None, 0, None, 0, c.data_ptr(), B * nb, s.data_ptr(), cols, off, experts)
    else:
        nb = (cols + (B - 1)) // B
        c, s = _code_lines(rows, nb, where), _empty((_blocks(rows), nb), (max(nb, 1), 1), dtype=_F32, device=where)
        args = head + (1, c.data_ptr(), B * nb, s.data_ptr(), nb, None, 0, None, 0, None, 1)
    if rows and cols:
        _call("mxq_quantize_b128", device, args)
    return c, s


def quantize_b128_dual(x, elem: str = "e4m3", tile: bool = False, rule: str = "amax", offsets=None):
    """Both orientations from one read: (row_codes, row_scales, col_codes, col_scales), as
    quantize_b128 along rows and columns; with tile=True the codes of 128 x 128 tiles and the same
    codes transposed, whose scales are the transposed view of row_scales.  With offsets only the
    experts' rows are quantized, in both orientations.
    """
    ld = _wide(x, "x")
    _elem("elem", elem)
    r = _rule(rule)
    experts, off = 1, None
    if offsets is not None:
        if tile:
            raise ValueError("tiles cannot follow offsets")
        experts, off = _offsets(offsets), offsets.data_ptr()
    device = x.get_device()
    if device < 0 or (offsets is not None and offsets.get_device() != device):
        _devices(x, ("offsets", offsets))
    rows, cols = x.shape
    where, nbc, nbr = x.device, (cols + (B - 1)) // B, (rows + (B - 1) * experts) // B
    rc, cc = _code_lines(rows, nbc, where), _code_lines(cols, nbr, where)
    if tile:
        rs = _empty((nbr, nbc), (max(nbc, 1), 1), dtype=_F32, device=where)
        cs, tail = rs.t(), (rs.data_ptr(), nbc, cc.data_ptr(), B * nbr, None, 0, None, 1)
    else:
        rs, cs = _scale_lines(rows, nbc, where), _scale_lines(cols, nbr, where)
        tail = (rs.data_ptr(), rows, cc.data_ptr(), B * nbr, cs.data_ptr(), cols, off, experts)
    if rows and cols:
        _call("mxq_quantize_b128", device, (x.data_ptr(), _WIDE[x.dtype], rows, cols, ld, _ELEM[elem], r,
                                            1 if tile else 0, rc.data_ptr(), B * nbc) + tail)
    return rc, rs, cc, cs


def _out(out, rows: int, cols: int, out_dtype, like):
    """The output [rows][cols] on the device of `like`, its type tag and row pitch."""
    if out is None:
        dtype = out_dtype or _BF16
        if dtype not in _WIDE:
            raise ValueError("out_dtype must be float32 or bfloat16")
        pitch = cols if cols > 0 else 1
        return _empty((rows, cols), (pitch, 1), dtype=dtype, device=like.device), _WIDE[dtype], pitch
    pitch = _wide(out, "out")
    if tuple(out.shape) != (rows, cols):
        raise ValueError("out must have shape (%d, %d), got %s" % (rows, cols, tuple(out.shape)))
    if out.get_device() != like.get_device():
        _devices(like, ("out", out))
    return out, _WIDE[out.dtype], pitch


def _accum(accum: str) -> int:
    if accum not in _ACC:
        raise ValueError("accum must be 'fp32' or 'fp8'")
    return _ACC[accum]


def gemm_b128(x_codes, x_scales, w_codes, w_scales, K: int, x_elem: str = "e4m3", w_elem: str = "e4m3",
              alpha: float = 1.0, bias=None, out_dtype=None, out=None, accum: str = "fp32", act=None):
    """Y[M][N] = act(alpha * (X W) + bias), both operands in blocks of 128: x_codes [M][128 nb] and
    x_scales [M][nb] of lines; w_codes [N][128 nb] and w_scales [N][nb] of lines or [ceil(N/128)][nb] of
    tiles.  accum="fp32": exact products, FP32 sums; "fp8": the FP8 matrix cores, faster (see
    mxq_gemm_b128).  act: None or "silu"; out_dtype bf16 (default) or fp32, or a preallocated `out`.
    """
    if K < 0:
        raise ValueError("K must be >= 0")
    nb = _blocks(K)
    ld_x, ld_w = _lines(x_codes, "x_codes", _U8, 0, B * nb), _lines(w_codes, "w_codes", _U8, 0, B * nb)
    M, N = x_codes.shape[0], w_codes.shape[0]
    ld_xs = _line_scales(x_scales, "x_scales", M, nb)
    w_block, ws_n, ws_k = _weight_scales(w_scales, "w_scales", N, nb)
    _elem("element formats", x_elem, w_elem)
    acc = _accum(accum)
    if bias is not None and (not isinstance(bias, torch.Tensor) or bias.dtype != _F32 or bias.dim() != 1
                             or bias.shape[0] != N or (N > 1 and bias.stride(0) != 1)):
        raise ValueError("bias must be a contiguous 1-D float32 tensor of N = %d elements" % N)
    if act not in _ACT:
        raise ValueError("act must be None or 'silu'")
    device = x_codes.get_device()
    if device < 0 or x_scales.get_device() != device or w_codes.get_device() != device or \
            w_scales.get_device() != device or (bias is not None and bias.get_device() != device):
        _devices(x_codes, ("x_scales", x_scales), ("w_codes", w_codes), ("w_scales", w_scales), ("bias", bias))
    out, y_type, ld_y = _out(out, M, N, out_dtype, x_codes)
    _call("mxq_gemm_b128", device, (
        M, N, K, x_codes.data_ptr(), ld_x, x_scales.data_ptr(), ld_xs, _ELEM[x_elem], w_codes.data_ptr(), ld_w,
        w_scales.data_ptr(), ws_n, ws_k, w_block, _ELEM[w_elem], alpha, None if bias is None else bias.data_ptr(),
        _ACT[act], acc, out.data_ptr(), y_type, ld_y))
    return out


def moe_gemm_b128(x_codes, x_scales, w_codes, w_scales, offsets, K: int, x_elem: str = "e4m3", w_elem: str = "e4m3",
                  out_dtype=None, out=None, accum: str = "fp32"):
    """Every expert's rows times its own matrix: Y[r] = X[r] W_e for r in offsets[e] .. offsets[e+1] - 1.
    x_codes [R][128 nb] and x_scales [R][nb], rows sorted by expert; w_codes [E][N][128 nb], w_scales
    [E][N or ceil(N/128)][nb]; offsets int32 [E + 1] on the device.  Rows of no expert are left as they
    were (without `out`: unset).  Otherwise as gemm_b128; see mxq_moe_gemm_b128.
    """
    if K < 0:
        raise ValueError("K must be >= 0")
    nb, E = _blocks(K), _offsets(offsets)
    ld_x = _lines(x_codes, "x_codes", _U8, 0, B * nb)
    if not isinstance(w_codes, torch.Tensor) or w_codes.dim() != 3 or w_codes.shape[0] != E:
        raise ValueError("w_codes must be a 3-D tensor of E = %d matrices" % E)
    if not isinstance(w_scales, torch.Tensor) or w_scales.dim() != 3 or w_scales.shape[0] != E:
        raise ValueError("w_scales must be a 3-D tensor of E = %d matrices" % E)
    R, N = x_codes.shape[0], w_codes.shape[1]
    ld_w = _lines(w_codes[0], "w_codes", _U8, 0, B * nb)
    ld_xs = _line_scales(x_scales, "x_scales", R, nb)
    w_block, ws_n, ws_k = _weight_scales(w_scales, "w_scales", N, nb, 1)
    _elem("element formats", x_elem, w_elem)
    acc = _accum(accum)
    device = _devices(x_codes, ("x_scales", x_scales), ("w_codes", w_codes), ("w_scales", w_scales),
                      ("offsets", offsets))
    out, y_type, ld_y = _out(out, R, N, out_dtype, x_codes)
    _call("mxq_moe_gemm_b128", device, (
        R, N, K, E, offsets.data_ptr(), x_codes.data_ptr(), ld_x, x_scales.data_ptr(), ld_xs, _ELEM[x_elem],
        w_codes.data_ptr(), ld_w, w_codes.stride(0), w_scales.data_ptr(), ws_n, ws_k, w_scales.stride(0), w_block,
        _ELEM[w_elem], acc, out.data_ptr(), y_type, ld_y))
    return out


def moe_wgrad_b128(dy_codes, dy_scales, x_codes, x_scales, offsets, x_elem: str = "e5m2", w_elem: str = "e4m3",
                   out_dtype=None, out=None, accum: str = "fp32"):
    """Every expert's weight gradient: dW[e] = sum over its rows r of dY[r]^T X[r] -> [E][N][K], fp32 by default.
    dy_codes [N][128 nb] in format x_elem and x_codes [K][128 nb] in w_elem, with their scales, from
    quantize_b128(..., "col" or dual, offsets=offsets).  An expert without rows gets zeros.  See
    mxq_moe_wgrad_b128.
    """
    E = _offsets(offsets)
    if not isinstance(dy_codes, torch.Tensor) or dy_codes.dim() != 2:
        raise ValueError("dy_codes must be a 2-D uint8 tensor")
    nb = dy_codes.shape[1] // B
    rows = max(B * nb + B - 1 - (B - 1) * E, 0)         # the most rows that give lines of nb blocks
    ld_dy, ld_x = _lines(dy_codes, "dy_codes", _U8, 0, B * nb), _lines(x_codes, "x_codes", _U8, 0, B * nb)
    N, K = dy_codes.shape[0], x_codes.shape[0]
    ld_ds, ld_xs = _line_scales(dy_scales, "dy_scales", N, nb), _line_scales(x_scales, "x_scales", K, nb)
    _elem("element formats", x_elem, w_elem)
    acc = _accum(accum)
    device = _devices(dy_codes, ("dy_scales", dy_scales), ("x_codes", x_codes), ("x_scales", x_scales),
                      ("offsets", offsets))
    if out is None:
        if out_dtype is not None and out_dtype not in _WIDE:
            raise ValueError("out_dtype must be float32 or bfloat16")
        out = _empty((E, N, K), (max(N * K, 1), max(K, 1), 1), dtype=out_dtype or _F32, device=dy_codes.device)
    else:
        if not isinstance(out, torch.Tensor) or out.dim() != 3 or out.dtype not in _WIDE or \
                (out.shape[2] > 1 and out.stride(2) != 1):
            raise ValueError("out must be a 3-D float32 or bfloat16 tensor with unit stride along its last dimension")
        if tuple(out.shape) != (E, N, K):
            raise ValueError("out must have shape (%d, %d, %d), got %s" % (E, N, K, tuple(out.shape)))
        _devices(dy_codes, ("out", out))
    _call("mxq_moe_wgrad_b128", device, (
        N, K, rows, E, offsets.data_ptr(), dy_codes.data_ptr(), ld_dy, dy_scales.data_ptr(), ld_ds, _ELEM[x_elem],
        x_codes.data_ptr(), ld_x, x_scales.data_ptr(), ld_xs, _ELEM[w_elem], acc, out.data_ptr(), _WIDE[out.dtype],
        out.stride(1) if N > 1 else max(K, 1), out.stride(0)))
    return out


class MoeRoute(NamedTuple):
    """What moe_route gives, see there."""
    experts: torch.Tensor
    shares: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    order: torch.Tensor
    loss: torch.Tensor
    slope: torch.Tensor


@functools.lru_cache(maxsize=1024)
def _route_workspace(T: int, E: int, k: int) -> int:
    return mxq_moe_route_workspace(T, E, k)


def _route_inputs(logits, mask):
    ld = _wide(logits, "logits")
    T, E = logits.shape
    if mask is not None and (not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.bool, _U8)
                             or mask.dim() != 1 or mask.shape[0] != T or (T > 1 and mask.stride(0) != 1)):
        raise ValueError("mask must be a contiguous 1-D bool or uint8 tensor of T = %d elements" % T)
    return T, E, ld


def moe_route(logits, k: int, renormalize: bool = True, mask=None) -> MoeRoute:
    """Routes tokens to experts: softmax of logits [T][E] (fp32 or bf16), the k greatest, shares, per-expert
    counts and order, and the balance loss E sum_e f_e P_e.  mask [T] (bool): tokens that count.

    experts [T][k] int32 (-1 where there is none), shares [T][k] fp32, counts [E] and offsets [E + 1]
    int32, order [T k] int32 (the slots t k + rank by expert: order // k are the rows to gather for
    moe_gemm_b128; -1 from offsets[E] on), loss [1] and slope [E] fp32.  See mxq_moe_route.
    """
    T, E, ld = _route_inputs(logits, mask)
    if not 1 <= k <= min(E, 64):
        raise ValueError("k must be between 1 and min(E, 64) = %d" % min(E, 64))
    device = _devices(logits, ("mask", mask))
    dev = logits.device
    experts = _empty((T, k), (k, 1), dtype=_I32, device=dev)
    shares = _empty((T, k), (k, 1), dtype=_F32, device=dev)
    counts = _empty((E,), (1,), dtype=_I32, device=dev)
    offsets = _empty((E + 1,), (1,), dtype=_I32, device=dev)
    order = _empty((T * k,), (1,), dtype=_I32, device=dev)
    loss = _empty((1,), (1,), dtype=_F32, device=dev)
    slope = _empty((E,), (1,), dtype=_F32, device=dev)
    need = _route_workspace(T, E, k)
    workspace = _empty((need,), (1,), dtype=_U8, device=dev) if need else None
    _call("mxq_moe_route", device, (
        T, E, k, 1 if renormalize else 0, logits.data_ptr(), _WIDE[logits.dtype], ld,
        None if mask is None else mask.data_ptr(), experts.data_ptr(), shares.data_ptr(), counts.data_ptr(),
        offsets.data_ptr(), order.data_ptr(), loss.data_ptr(), slope.data_ptr(),
        None if workspace is None else workspace.data_ptr(), need))
    return MoeRoute(experts, shares, counts, offsets, order, loss, slope)


def moe_route_grad(logits, route: MoeRoute, d_shares=None, d_loss=None, renormalize: bool = True, mask=None):
    """The gradient of the logits (in their type) from those of moe_route's shares (fp32 [T][k]) and loss (one fp32
    element on the device); either may be None.  route, renormalize and mask: of the forward call.  See
    mxq_moe_route_grad.
    """
    T, E, ld = _route_inputs(logits, mask)
    experts, shares, slope = route.experts, route.shares, route.slope
    k = experts.shape[1]
    if tuple(experts.shape) != (T, k) or tuple(shares.shape) != (T, k) or tuple(slope.shape) != (E,):
        raise ValueError("route is of other sizes than logits (%d, %d)" % (T, E))
    for name, t, dtype in (("experts", experts, _I32), ("shares", shares, _F32), ("slope", slope, _F32)):
        if t.dtype is not dtype or not t.is_contiguous():
            raise ValueError("route.%s must be a contiguous %s tensor" % (name, dtype))
    ld_ds = 0
    if d_shares is not None:
        ld_ds = _lines(d_shares, "d_shares", _F32, T, k)
        if tuple(d_shares.shape) != (T, k):
            raise ValueError("d_shares must have shape (%d, %d), got %s" % (T, k, tuple(d_shares.shape)))
    if d_loss is not None and (not isinstance(d_loss, torch.Tensor) or d_loss.dtype is not _F32 or d_loss.numel() != 1):
        raise ValueError("d_loss must be a float32 tensor of one element")
    device = _devices(logits, ("mask", mask), ("experts", experts), ("shares", shares), ("slope", slope),
                      ("d_shares", d_shares), ("d_loss", d_loss))
    d = _empty((T, E), (max(E, 1), 1), dtype=logits.dtype, device=logits.device)
    _call("mxq_moe_route_grad", device, (
        T, E, k, 1 if renormalize else 0, logits.data_ptr(), _WIDE[logits.dtype], ld,
        None if mask is None else mask.data_ptr(), experts.data_ptr(), shares.data_ptr(), slope.data_ptr(),
        None if d_shares is None else d_shares.data_ptr(), ld_ds, None if d_loss is None else d_loss.data_ptr(),
        d.data_ptr(), max(E, 1)))
    return d
