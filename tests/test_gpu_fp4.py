"""GPU parity of the MXFP4 operators with the 64-bit reference (fp4_reference): codes and
scales byte for byte, products and the expert layer within the reference's derived bounds."""
import numpy as np
import pytest
import torch

import fp4_reference as ref
import mxfp8_block_scaled_03_amd as mxq
from gpu_helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def f64(t):
    return t.detach().cpu().double().numpy()


def data(rng, rows, cols, dtype, spread=20):
    """Rows of very different sizes, signed zeros, exact ties."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-spread, spread + 1, (rows, 1)))
    x.flat[::7] = np.copysign(0.0, rng.standard_normal(x.flat[::7].size))
    x.flat[3::11] = rng.integers(-24, 25, x.flat[3::11].size) * 0.25
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def check_bytes(got, want, what):
    got, want = got.cpu().numpy(), np.asarray(want)
    assert got.shape == want.shape, what
    if not np.array_equal(got, want):
        at = np.argwhere(got != want)[0].tolist()
        raise AssertionError("%s: at %s 0x%02x, expected 0x%02x" % (what, at, got[tuple(at)], want[tuple(at)]))


SHAPES = [(1, 1), (3, 5), (7, 31), (5, 32), (4, 33), (16, 64), (9, 100), (130, 72), (33, 513), (129, 257), (260, 40)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("axis", ["row", "col"])
@pytest.mark.parametrize("how", ["ceil", "ocp", "sr"])
def test_quantize(dtype, axis, how):
    rng = np.random.default_rng(10)
    for rows, cols in SHAPES:
        say("quantize_fp4 %s %s %s %dx%d" % (dtype, axis, how, rows, cols))
        x = data(rng, rows, cols, dtype)
        lines = f64(x) if axis == "row" else f64(x).T
        seed = 0xFEDCBA9876543210 + rows
        want = ref.quantize(lines, "ocp" if how == "ocp" else "ceil", seed if how == "sr" else None)
        L, nb = want[1].shape
        # outputs wider than needed, rows of the source padded: nothing else is touched
        codes = torch.full((L, 16 * nb + 16), 0xCD, dtype=torch.uint8, device=DEV)
        scales = torch.full((L, nb + 3), 0xCD, dtype=torch.uint8, device=DEV)
        wide = torch.full((rows, cols + 3), 99.0, dtype=dtype, device=DEV)
        wide[:, :cols] = x.to(DEV)
        call = (lambda y, **k: mxq.quantize_fp4_sr(y, seed, axis, **k)) if how == "sr" else \
            (lambda y, **k: mxq.quantize_fp4(y, axis, rule=how, **k))
        call(wide[:, :cols], codes=codes, scales=scales)
        assert (codes[:, 16 * nb:] == 0xCD).all() and (scales[:, nb:] == 0xCD).all()
        check_bytes(scales[:, :nb], want[1], "scales")
        check_bytes(codes[:, :16 * nb], want[0], "codes")
        c, s = call(x.to(DEV))
        check_bytes(s, want[1], "scales, dense")
        check_bytes(c, want[0], "codes, dense")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_extremes(dtype):
    """Blocks of zeros, subnormals, the largest values, infinities and NaN; scale byte 0."""
    rng = np.random.default_rng(11)
    x = np.zeros((12, 64), np.float32)
    x[1] = rng.standard_normal(64) * 1e-39
    x[2] = rng.standard_normal(64) * 2.0 ** -127
    x[3] = 3.3e38 * rng.uniform(-1, 1, 64)
    x[4, 5], x[5, 6], x[6, 40] = np.inf, -np.inf, np.nan
    x[7] = np.copysign(0, rng.standard_normal(64))
    x[8, 0], x[8, 1:] = 6e30, 1e-30
    x[9] = 2.0 ** -149
    x[10] = 6.0 * 2.0 ** rng.integers(-140, 120, 64)
    x[11] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 8)
    t = torch.from_numpy(x).to(dtype)
    for axis in ("row", "col"):
        lines = f64(t) if axis == "row" else f64(t).T
        for how in ("ceil", "ocp"):
            got = mxq.quantize_fp4(t.to(DEV), axis, rule=how)
            want = ref.quantize(lines, how)
            check_bytes(got[1], want[1], "%s %s scales" % (axis, how))
            check_bytes(got[0], want[0], "%s %s codes" % (axis, how))
        got, want = mxq.quantize_fp4_sr(t.to(DEV), 5, axis), ref.quantize(lines, "ceil", 5)
        check_bytes(got[1], want[1], axis + " sr scales")
        check_bytes(got[0], want[0], axis + " sr codes")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_dual(dtype):
    rng = np.random.default_rng(12)
    for rows, cols in SHAPES + [(300, 1000), (1030, 264)]:
        say("quantize_fp4_dual %s %dx%d" % (dtype, rows, cols))
        x = data(rng, rows, cols, dtype).to(DEV)
        rc, rs, cc, cs = mxq.quantize_fp4_dual(x)
        for got, want in zip((rc, rs, cc, cs), mxq.quantize_fp4(x, "row") + mxq.quantize_fp4(x, "col")):
            assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dequantize(dtype):
    rng = np.random.default_rng(13)
    for L, K in [(1, 1), (3, 7), (5, 32), (4, 33), (9, 100), (2, 2048), (65, 515), (256, 32)]:
        codes = rng.integers(0, 256, (L, 16 * ref.blocks(K)), dtype=np.uint8)
        scales = rng.integers(0, 256, (L, ref.blocks(K)), dtype=np.uint8)
        got = mxq.dequantize_fp4(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), K, out_dtype=dtype)
        with np.errstate(over="ignore"):
            want = torch.from_numpy(ref.values(codes, scales, K).astype(np.float32)).to(dtype)
        got = got.cpu()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan], want[~nan]) and torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))


# ------------------------------------------------------------------------------- products

def operand(rng, rows, K, pad=0, std=1.0):
    """Codes and scales on the GPU (rows wider by `pad` blocks of garbage) and their values."""
    x = rng.standard_normal((rows, K)) * std
    x.flat[::97] *= 50
    codes, scales = ref.quantize(x.astype(np.float32).astype(np.float64)) if rows * K < 40000 else fast_codes(rng, rows, K)
    nb = scales.shape[1]
    v = ref.values(codes, scales, K)
    c = np.full((rows, 16 * (nb + pad)), 0x5D, np.uint8)
    s = np.full((rows, nb + pad), 255, np.uint8)
    c[:, :16 * nb], s[:, :nb] = codes, scales
    return torch.from_numpy(c).to(DEV)[:, :16 * nb], torch.from_numpy(s).to(DEV)[:, :nb], v


def fast_codes(rng, rows, K):
    return (rng.integers(0, 256, (rows, 16 * ref.blocks(K)), dtype=np.uint8),
            rng.integers(118, 128, (rows, ref.blocks(K)), dtype=np.uint8))


def bf16_operand(rng, rows, K, pad=0):
    x = torch.from_numpy(rng.standard_normal((rows, K)).astype(np.float32)).to(BF16)
    wide = torch.full((rows, K + pad), float("nan"), dtype=BF16, device=DEV)
    wide[:, :K] = x.to(DEV)
    return wide[:, :K], None, f64(x)


def check_product(y, want, bound, what):
    got = f64(y)
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    assert (err <= bound).all(), "%s: off by %.3g, bound %.3g, at %s" % (
        what, err.flat[np.argmax(err - bound)], bound.flat[np.argmax(err - bound)], np.argwhere(err > bound)[0].tolist())


PRODUCTS = [(1, 1, 1), (1, 16, 32), (2, 5, 33), (3, 17, 127), (1, 64, 128), (16, 40, 129), (17, 33, 300), (15, 130, 1000),
            (40, 70, 257), (64, 64, 1024), (65, 65, 1025), (130, 200, 511), (1, 300, 4096), (257, 129, 640), (300, 520, 384)]


@pytest.mark.parametrize("xt", ["bf16", "fp4"])
@pytest.mark.parametrize("out", [F32, BF16])
def test_gemm(xt, out):
    rng = np.random.default_rng(20)
    for n, (M, N, K) in enumerate(PRODUCTS):
        pad = n % 3
        x, xs, xv = operand(rng, M, K, pad) if xt == "fp4" else bf16_operand(rng, M, K, pad)
        w, ws, wv = operand(rng, N, K, pad, 0.1)
        bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(DEV) if n % 2 else None
        alpha, act = (0.75 if n % 5 == 1 else 1.0), ("silu" if n % 3 == 2 else None)
        say("gemm_fp4 %s %s %dx%dx%d" % (xt, out, M, N, K))
        wide = torch.full((M, N + pad), 7.0, dtype=out, device=DEV)
        y = mxq.gemm_fp4(x, xs, w, ws, K, alpha=alpha, bias=bias, act=act, out=wide[:, :N])
        want, bound = ref.product(xv, wv, alpha, None if bias is None else f64(bias), act, out == BF16)
        check_product(y, want, bound, "%dx%dx%d" % (M, N, K))
        assert (wide[:, N:] == 7.0).all()


@pytest.mark.parametrize("xt", ["bf16", "fp4"])
@pytest.mark.parametrize("M,N,K", [(512, 768, 512), (700, 1030, 289), (1030, 1100, 1000), (2100, 64, 160), (64, 2100, 4001)])
def test_gemm_large(xt, M, N, K):
    rng = np.random.default_rng(21)
    x, xs, xv = operand(rng, M, K) if xt == "fp4" else bf16_operand(rng, M, K)
    w, ws, wv = operand(rng, N, K)
    y = mxq.gemm_fp4(x, xs, w, ws, K, out_dtype=F32)
    check_product(y, *ref.product(xv, wv), "%dx%dx%d" % (M, N, K))
    assert torch.equal(y, mxq.gemm_fp4(x, xs, w, ws, K, out_dtype=F32))


@pytest.mark.parametrize("xt", ["bf16", "fp4"])
def test_gemm_empty_and_special(xt):
    rng = np.random.default_rng(22)
    x, xs, xv = operand(rng, 5, 96) if xt == "fp4" else bf16_operand(rng, 5, 96)
    w, ws, wv = operand(rng, 33, 96)
    bias = torch.arange(33, dtype=F32, device=DEV)
    none = None if xs is None else xs[:, :0]
    y = mxq.gemm_fp4(x[:, :0], none, w[:, :0], ws[:, :0], 0, bias=bias, out_dtype=F32)
    assert torch.equal(y, bias.expand(5, 33))
    assert mxq.gemm_fp4(x[:0], None if xs is None else xs[:0], w, ws, 96).shape == (0, 33)
    assert mxq.gemm_fp4(x, xs, w[:0], ws[:0], 96).shape == (5, 0)
    # a NaN scale byte reaches its row and column only
    ws2 = ws.clone()
    ws2[7, 1] = 255
    y = f64(mxq.gemm_fp4(x, xs, w, ws2, 96, out_dtype=F32))
    assert np.isnan(y[:, 7]).all() and np.isfinite(np.delete(y, 7, 1)).all()
    if xs is not None:
        xs2 = xs.clone()
        xs2[2, 2] = 255
        y = f64(mxq.gemm_fp4(x, xs2, w, ws, 96, out_dtype=F32))
        assert np.isnan(y[2]).all() and np.isfinite(np.delete(y, 2, 0)).all()
    # the smallest scales: 2^-127 against large ones, products in FP32's normal range
    wz = torch.zeros_like(ws)
    big = torch.full((5, 96), 2.0 ** 100, dtype=BF16, device=DEV)
    if xs is None:
        y, want = mxq.gemm_fp4(big, None, w, wz, 96, out_dtype=F32), ref.product(
            np.full((5, 96), 2.0 ** 100), ref.values(w.cpu().numpy(), np.zeros((33, 3), np.uint8), 96))
    else:
        xb = torch.full_like(xs, 227)
        y, want = mxq.gemm_fp4(x, xb, w, wz, 96, out_dtype=F32), ref.product(
            ref.values(x.cpu().numpy(), np.full((5, 3), 227, np.uint8), 96),
            ref.values(w.cpu().numpy(), np.zeros((33, 3), np.uint8), 96))
    check_product(y, *want, "smallest scales")


def test_gemm_infinite_input():
    rng = np.random.default_rng(23)
    x, _, _ = bf16_operand(rng, 4, 64)
    w = torch.full((16, 32), 0x22, dtype=torch.uint8, device=DEV)          # all ones
    ws = torch.full((16, 2), 127, dtype=torch.uint8, device=DEV)
    x[1, 3], x[2, 60] = float("inf"), float("nan")
    y = mxq.gemm_fp4(x, None, w, ws, 64, out_dtype=F32)
    assert torch.isinf(y[1]).all() and torch.isnan(y[2]).all() and torch.isfinite(y[[0, 3]]).all()


def test_linear_gradients():
    """dX and dW of a linear layer against float64 products of the same quantized values, and
    the mean of many stochastic roundings against the unquantized gradient."""
    rng = np.random.default_rng(24)
    M, N, K = 96, 160, 64
    dy = torch.from_numpy((rng.standard_normal((M, N)) * 1e-3).astype(np.float32)).to(BF16)
    w, ws, wv = operand(rng, K, N)
    xt, xts, xv = operand(rng, K, M)
    r, rs = mxq.quantize_fp4_sr(dy.to(DEV), 3, "row")
    c, cs = mxq.quantize_fp4_sr(dy.to(DEV), 4, "col")
    rv = ref.values(r.cpu().numpy(), rs.cpu().numpy(), N)
    cv = ref.values(c.cpu().numpy(), cs.cpu().numpy(), M)
    check_product(mxq.gemm_fp4(r, rs, w, ws, N, out_dtype=BF16), *ref.product(rv, wv, bf16=True), "dx")
    check_product(mxq.gemm_fp4(c, cs, xt, xts, M, out_dtype=F32), *ref.product(cv, xv), "dw")
    total, n = torch.zeros((M, K), dtype=torch.float64, device=DEV), 400
    for seed in range(n):
        r, rs = mxq.quantize_fp4_sr(dy.to(DEV), seed, "row")
        total += mxq.gemm_fp4(r, rs, w, ws, N, out_dtype=F32)
    # a rounding's variance is at most (step / 2)^2 with a step of at most 2 S, S <= amax / 3
    step = 2 * np.abs(f64(dy)).reshape(M, -1, 32).max(-1) / 3
    var = (np.repeat(step, 32, 1) / 2) ** 2 @ (wv ** 2).T / n
    off = np.abs(total.cpu().numpy() / n - f64(dy) @ wv.T)
    assert (off <= 6 * np.sqrt(var) + 1e-9).all()


# -------------------------------------------------------------------------------- experts

def experts(rng, E, H, I):
    w = [operand(rng, E * r, c, 0, c ** -0.5) for r, c in ((2 * I, H), (H, I))]
    out = []
    for (codes, scales, v), rows in zip(w, (2 * I, H)):
        pitch = (scales.shape[1] + 15) // 16 * 16
        s = torch.full((E, rows, pitch), 255, dtype=torch.uint8, device=DEV)
        s[..., :scales.shape[1]] = scales.view(E, rows, -1)
        out += [codes.reshape(E, rows, -1).contiguous(), s[..., :scales.shape[1]], v.reshape(E, rows, -1)]
    return out


def run_experts(rng, T, H, I, E, k, renorm, out, logits=None):
    w13, s13, v13, w2, s2, v2 = experts(rng, E, H, I)
    x, _, xv = bf16_operand(rng, T, H, 3)
    lg = rng.standard_normal((T, E)) * 1.5 if logits is None else np.asarray(logits, np.float64)
    lg = lg.astype(np.float32)
    y = mxq.moe_fp4(x, torch.from_numpy(lg).to(DEV), w13, s13, w2, s2, k, renormalize=renorm, out_dtype=out)
    want, bound = ref.moe(xv, lg.astype(np.float64), v13, v2, k, renorm, out == BF16)
    check_product(y, want, bound, "T%d H%d I%d E%d k%d" % (T, H, I, E, k))
    return y


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,H,I,E,k", [
    (1, 32, 16, 1, 1), (1, 64, 40, 8, 2), (1, 256, 136, 70, 5), (2, 100, 30, 4, 4), (5, 130, 65, 16, 3), (7, 200, 104, 60, 6),
    (16, 64, 32, 8, 2), (17, 96, 48, 3, 2), (40, 64, 24, 4, 3), (64, 128, 64, 16, 4), (70, 33, 129, 2, 1), (3, 64, 24, 130, 2)])
def test_experts(out, renorm, T, H, I, E, k):
    say("moe_fp4 T%d H%d I%d E%d k%d %s" % (T, H, I, E, k, out))
    run_experts(np.random.default_rng(30), T, H, I, E, k, renorm, out)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("T,H,I,E,k", [(200, 72, 120, 512, 8), (40, 1032, 1100, 64, 8), (150, 520, 520, 64, 8)])
def test_experts_many(out, T, H, I, E, k):
    """Sizes whose weights occupy every CU for long: the persistent kernels, several tiles of
    tokens, ragged columns, K of several chunks."""
    say("moe_fp4 T%d H%d I%d E%d k%d %s" % (T, H, I, E, k, out))
    run_experts(np.random.default_rng(35), T, H, I, E, k, True, out)


def test_experts_many_with_unused_experts():
    """Most experts unused, one overloaded, tokens without any."""
    rng = np.random.default_rng(36)
    lg = rng.standard_normal((130, 256)).astype(np.float32)
    lg[:, 200] = 9.0
    lg[5] = -np.inf
    lg[::3, 100:190] = -np.inf
    run_experts(rng, 130, 64, 300, 256, 4, False, BF16, lg)


def test_experts_ties_and_masks():
    """Equal logits (ties to the lower index), -inf and the lowest float, rows with fewer than k
    experts or none, one expert for everybody."""
    rng = np.random.default_rng(31)
    low = np.finfo(np.float32).min
    lg = np.zeros((8, 6))
    lg[1] = [1, 2, 2, 2, 0, 2]
    lg[2] = [-np.inf, 0, -np.inf, -np.inf, 1, -np.inf]
    lg[3] = -np.inf
    lg[4] = low
    lg[5] = [low, low, 3, low, low, low]
    lg[6] = [-0.0, 0.0, -0.0, -1, -1, -1]
    lg[7] = [-np.inf, -np.inf, 5, -np.inf, -np.inf, -np.inf]
    for renorm in (True, False):
        for out in (F32, BF16):
            y = run_experts(rng, 8, 96, 40, 6, 3, renorm, out, lg)
            assert (y[3] == 0).all()
    run_experts(rng, 40, 64, 32, 6, 2, True, F32, np.tile([0, 9, 0, 0, 8, 0], (40, 1)))
    run_experts(rng, 1, 64, 32, 9, 2, True, F32, [[-np.inf] * 8 + [0.0]])


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,H,I,k", [(1, 100, 40, 3), (3, 33, 129, 2), (17, 64, 24, 4), (33, 130, 65, 2), (70, 96, 200, 1),
                                     (64, 520, 136, 4), (5, 1030, 33, 8)])
def test_experts_of_many(out, renorm, T, H, I, k):
    """More experts than one wave of logits takes: the kernels with a launch for routing, at small
    odd sizes."""
    say("moe_fp4 T%d H%d I%d k%d of 264 %s" % (T, H, I, k, out))
    run_experts(np.random.default_rng(37), T, H, I, 264, k, renorm, out)


@pytest.mark.parametrize("masked", [0, 260])
@pytest.mark.parametrize("out", [F32, BF16])
def test_experts_special_logits(masked, out):
    """Ties, -inf, the lowest float, rows with nothing left, +inf and NaN, also among many masked experts
    (the other kernels); masked ones stand in front, so that ties are decided far from index 0."""
    rng = np.random.default_rng(38)
    low = np.finfo(np.float32).min
    lg = np.zeros((7, 6), np.float32)
    lg[1] = [1, 2, 2, 2, 0, 2]
    lg[2] = [-np.inf, 0, -np.inf, -np.inf, 1, -np.inf]
    lg[3] = -np.inf
    lg[4] = low
    lg[5] = [-0.0, 0.0, -0.0, -1, -1, -1]
    lg = np.concatenate([np.full((7, masked), -np.inf, np.float32), lg], 1)
    for renorm in (True, False):
        y = run_experts(rng, 7, 72, 40, 6 + masked, 3, renorm, out, lg)
        assert (y[3] == 0).all()
    w13, s13, _, w2, s2, _ = experts(rng, 6 + masked, 72, 40)
    x, _, _ = bf16_operand(rng, 7, 72)
    bad = torch.from_numpy(lg).to(DEV)
    bad[0, masked + 2], bad[6, masked + 4] = float("nan"), float("inf")
    y = mxq.moe_fp4(x, bad, w13, s13, w2, s2, 3, out_dtype=out)
    assert torch.isnan(y[[0, 6]]).all() and torch.isfinite(y[1:6]).all()


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 4096, 264, 8, 2), (2, 2080, 2100, 5, 3), (1, 9000, 40, 4, 1), (3, 70, 4200, 6, 2),
                                       (1, 40, 72, 256, 9), (6, 2000, 1064, 10, 1)])
def test_experts_of_few_tokens(out, T, H, I, E, k):
    """Rows of several 2048-element segments, in both products, and waves with several row groups."""
    say("moe_fp4 T%d H%d I%d E%d k%d %s" % (T, H, I, E, k, out))
    run_experts(np.random.default_rng(39), T, H, I, E, k, True, out)


def test_experts_nan_logits():
    """A NaN logit makes its own token NaN and no other."""
    rng = np.random.default_rng(32)
    w13, s13, _, w2, s2, _ = experts(rng, 4, 64, 32)
    x, _, _ = bf16_operand(rng, 3, 64)
    lg = torch.zeros((3, 4), device=DEV)
    lg[1, 2] = float("nan")
    y = mxq.moe_fp4(x, lg, w13, s13, w2, s2, 2, out_dtype=F32)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()


def test_experts_strided_weights_and_output():
    """Experts that are slices of wider arrays, logits with a pitch, a preallocated output."""
    rng = np.random.default_rng(33)
    E, T, H, I, k = 5, 6, 96, 72, 2
    w13, s13, v13, w2, s2, v2 = experts(rng, E, H, I)

    def embed(t, rows, cols):
        big = torch.full((E, t.shape[1] + rows, t.shape[2] + cols), 0x7F, dtype=torch.uint8, device=DEV)
        big[:, :t.shape[1], :t.shape[2]] = t
        return big[:, :t.shape[1], :t.shape[2]]
    x, _, xv = bf16_operand(rng, T, H)
    lg = torch.from_numpy(rng.standard_normal((T, E + 4)).astype(np.float32)).to(DEV)[:, 2:2 + E]
    out = torch.full((T, H + 5), 3.0, dtype=BF16, device=DEV)
    y = mxq.moe_fp4(x, lg, embed(w13, 3, 16), embed(s13, 1, 3), embed(w2, 2, 32), embed(s2, 4, 1), k, out=out[:, :H])
    want, bound = ref.moe(xv, f64(lg), v13, v2, k, True, True)
    check_product(y, want, bound, "strided")
    assert (out[:, H:] == 3.0).all()


def test_other_stream_and_graph():
    """The operators on a side stream, and captured into a graph that is replayed on new inputs
    with eager work between the replays."""
    rng = np.random.default_rng(34)
    w13, s13, _, w2, s2, _ = experts(rng, 8, 128, 64)
    x = torch.from_numpy(rng.standard_normal((4, 128)).astype(np.float32)).to(BF16).to(DEV)
    lg = torch.from_numpy(rng.standard_normal((4, 8)).astype(np.float32)).to(DEV)

    def step(x, lg):
        c, s = mxq.quantize_fp4(x)
        return (mxq.moe_fp4(x, lg, w13, s13, w2, s2, 2), mxq.gemm_fp4(x, None, w13[0], s13[0], 128),
                mxq.gemm_fp4(c, s, w13[1], s13[1], 128), mxq.dequantize_fp4(c, s, 128), *mxq.quantize_fp4_dual(x))

    want = step(x, lg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x, lg)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gx, gl = x.clone(), lg.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(gx, gl)
    for r in range(4):
        gx.copy_(torch.roll(x, r, 0) * (r + 1))
        gl.copy_(torch.roll(lg, r, 1))
        want = step(gx, gl)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), r


def test_experts_strided_of_many():
    """Slices of wider arrays, scale rows at odd addresses and a column of logits' array, where routing has
    a launch of its own."""
    rng = np.random.default_rng(40)
    E, T, H, I, k = 264, 20, 96, 72, 3
    w13, s13, v13, w2, s2, v2 = experts(rng, E, H, I)

    def embed(t, rows, cols):
        big = torch.full((E, t.shape[1] + rows, t.shape[2] + cols), 0x7F, dtype=torch.uint8, device=DEV)
        big[:, :t.shape[1], :t.shape[2]] = t
        return big[:, :t.shape[1], :t.shape[2]]
    x, _, xv = bf16_operand(rng, T, H, 5)
    lg = torch.from_numpy(rng.standard_normal((T, E + 4)).astype(np.float32)).to(DEV)[:, 2:2 + E]
    for dtype in (BF16, F32):
        out = torch.full((T, H + 5), 3.0, dtype=dtype, device=DEV)
        y = mxq.moe_fp4(x, lg, embed(w13, 3, 16), embed(s13, 1, 3), embed(w2, 2, 32), embed(s2, 4, 1), k, out=out[:, :H])
        want, bound = ref.moe(xv, f64(lg), v13, v2, k, True, dtype == BF16)
        check_product(y, want, bound, "strided")
        assert (out[:, H:] == 3.0).all()


@pytest.mark.parametrize("T,E", [(2, 6), (48, 264)])
def test_experts_graph(T, E):
    """The expert layer captured and replayed on new inputs, with eager calls between the replays, in two
    launches and in four."""
    rng = np.random.default_rng(41)
    w13, s13, _, w2, s2, _ = experts(rng, E, 72, 40)
    x = torch.from_numpy(rng.standard_normal((T, 72)).astype(np.float32)).to(BF16).to(DEV)
    lg = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)

    def step(x, lg):
        return [mxq.moe_fp4(x, lg, w13, s13, w2, s2, 3, renormalize=n, out_dtype=d) for n in (True, False) for d in (F32, BF16)]
    step(x, lg)
    gx, gl = x.clone(), lg.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(gx, gl)
    for r in range(4):
        gx.copy_(torch.roll(x, r, 0) * (r + 1))
        gl.copy_(torch.roll(lg, r, 1))
        want = step(gx, gl)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), r


def far(t, pitch):
    """The rows of t, `pitch` elements apart in a buffer that is written nowhere else."""
    big = torch.empty((t.shape[0] * pitch,), dtype=t.dtype, device=DEV).view(t.shape[0], pitch)[:, :t.shape[1]]
    big.copy_(t)
    return big


def test_offsets_past_32_bits():
    """Rows and experts further apart than 2^32 bytes reach."""
    rng = np.random.default_rng(42)
    K = 96
    w, ws, wv = operand(rng, 600, K)
    x, xs, xv = operand(rng, 520, K)
    b, _, bv = bf16_operand(rng, 40, K)
    say("gemm_fp4, rows of W 8 MiB apart")
    wf, wsf = far(w, 1 << 23), far(ws, 1 << 23)
    check_product(mxq.gemm_fp4(b, None, wf, wsf, K, out_dtype=F32), *ref.product(bv, wv), "bf16")
    check_product(mxq.gemm_fp4(x, xs, wf, wsf, K, out_dtype=F32), *ref.product(xv, wv), "fp4")
    check_product(mxq.gemm_fp4(far(x, 1 << 23), far(xs, 1 << 23), w, ws, K, out_dtype=F32), *ref.product(xv, wv), "far x")
    say("gemm_fp4, rows of X and Y 128 MiB apart")
    y = torch.empty((40 * (1 << 25),), dtype=F32, device=DEV).view(40, 1 << 25)[:, :600]
    check_product(mxq.gemm_fp4(far(b, 1 << 26), None, w, ws, K, out=y), *ref.product(bv, wv), "far y")
    del wf, wsf, y
    say("quantize_fp4 and dequantize_fp4, rows 1 GiB apart")
    v = data(rng, 6, 130, F32).to(DEV)
    for got, want in zip(mxq.quantize_fp4_dual(far(v, 1 << 28)), mxq.quantize_fp4_dual(v)):
        assert torch.equal(got, want)
    c, s = mxq.quantize_fp4(v)
    assert torch.equal(mxq.dequantize_fp4(far(c, 1 << 30), far(s, 1 << 30), 130), mxq.dequantize_fp4(c, s, 130))
    say("moe_fp4, experts 3 GiB apart")
    E, T, H, I = 3, 4, 64, 40
    w13, s13, v13, w2, s2, v2 = experts(rng, E, H, I)

    def apart(t):
        big = torch.empty((E * 3 << 30,), dtype=torch.uint8, device=DEV)
        out = big.as_strided(t.shape, (3 << 30, t.shape[2] + (-t.shape[2]) % 16, 1))
        out.copy_(t)
        return out
    h, _, hv = bf16_operand(rng, T, H)
    lg = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    y = mxq.moe_fp4(h, lg, apart(w13), apart(s13), apart(w2), apart(s2), 2, out_dtype=F32)
    check_product(y, *ref.moe(hv, f64(lg), v13, v2, 2, True, False), "far experts")


def test_tile_product_with_far_rows():
    """The 256 x 256 tiles with rows 1 MiB apart: 3 GB from the first row to the last."""
    rng = np.random.default_rng(43)
    M, N, K = 2900, 2900, 160
    x, xs, xv = operand(rng, M, K)
    w, ws, wv = operand(rng, N, K)
    y = mxq.gemm_fp4(far(x, 1 << 20), far(xs, 1 << 20), far(w, 1 << 20), far(ws, 1 << 20), K, out_dtype=F32)
    check_product(y, *ref.product(xv, wv), "far tiles")


@pytest.mark.parametrize("xt", ["bf16", "fp4"])
@pytest.mark.parametrize("M,N,K", [(1100, 1100, 300), (1100, 1100, 1300), (2100, 2100, 1100), (1500, 2900, 129), (40, 2100, 200),
                                   (3000, 1500, 65)])
def test_gemm_tiles_and_splits(xt, M, N, K):
    """Sizes for every tile and split of K that the product chooses from, with a ragged end on each axis,
    bias and SiLU; y in bf16 with an odd pitch and in fp32, nothing written beside it."""
    rng = np.random.default_rng(44)
    x, xs, xv = operand(rng, M, K) if xt == "fp4" else bf16_operand(rng, M, K)
    w, ws, wv = operand(rng, N, K, 0, K ** -0.5)
    bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(DEV)
    say("gemm_fp4 %s %dx%dx%d" % (xt, M, N, K))
    for out, pad, act in ((BF16, 3, "silu"), (F32, 1, None), (BF16, (-N) % 8 + 8, None)):
        wide = torch.full((M + 2, N + pad), 7.0, dtype=out, device=DEV)
        y = mxq.gemm_fp4(x, xs, w, ws, K, bias=bias, act=act, out=wide[1:M + 1, :N])
        check_product(y, *ref.product(xv, wv, 1.0, f64(bias), act, out == BF16), "%s %s" % (out, act))
        assert (wide[1:M + 1, N:] == 7.0).all() and (wide[0] == 7.0).all() and (wide[M + 1] == 7.0).all()


@pytest.mark.parametrize("xt", ["bf16", "fp4"])
@pytest.mark.parametrize("M,N,K", [(1, 9000, 1100), (16, 8200, 200), (3, 500, 1030), (20, 17000, 1040), (32, 4100, 1100), (48, 8300, 1100),
                                   (9, 300, 700)])
def test_gemm_few_rows_many_columns(xt, M, N, K):
    rng = np.random.default_rng(45)
    x, xs, xv = operand(rng, M, K) if xt == "fp4" else bf16_operand(rng, M, K, 1)
    w, ws, wv = operand(rng, N, K, 1)
    say("gemm_fp4 %s %dx%dx%d" % (xt, M, N, K))
    check_product(mxq.gemm_fp4(x, xs, w, ws, K, out_dtype=F32), *ref.product(xv, wv), "%dx%dx%d" % (M, N, K))


# ------------------------------------------------------------ the most columns that there may be

TOP = 2 ** 31 - 1
PIECE = 1 << 24


def top_weights(K):
    """W with 2^31 - 1 rows: zeros but for the first and the last byte of a row, which repeat every PIECE
    rows; and the float64 values of the elements that they hold."""
    rng = np.random.default_rng(50)
    w = torch.zeros((TOP, 16), dtype=torch.uint8, device=DEV)
    s = torch.full((TOP, 1), 127, dtype=torch.uint8, device=DEV)
    first, last = (rng.integers(0, 256, PIECE, dtype=np.uint8) for _ in range(2))
    for at, b in ((0, first), ((K - 1) // 2, last)):
        b = torch.from_numpy(b).to(DEV)
        for c in range(0, TOP, PIECE):
            w[c:c + PIECE, at] = b[:min(PIECE, TOP - c)]
    table = np.concatenate([ref.MAG, -ref.MAG])
    lo, hi = (table[v] for v in (first & 15, first >> 4))
    return w, s, torch.from_numpy(np.stack([lo, hi, table[last & 15], table[last >> 4]])).to(DEV)


def check_top(call, want, rows):
    """call(y) fills y [rows][TOP]; every column against `want` [rows][PIECE], which repeats; nothing is
    written beside y."""
    flat = torch.full((rows * TOP + 64,), 7.0, dtype=BF16, device=DEV)
    y = flat[32:32 + rows * TOP].view(rows, TOP)
    call(y)
    want = want.to(BF16)
    for c in range(0, TOP, PIECE):
        assert torch.equal(y[:, c:c + PIECE], want[:, :min(PIECE, TOP - c)]), c
    assert (flat[:32] == 7.0).all() and (flat[-32:] == 7.0).all()


def test_gemm_short_rows_of_most_columns():
    """K < 8 at N = 2^31 - 1, whose last group of columns has three.  All sums are exact in bf16: multiples
    of 1/2 of at most 54."""
    w, s, v = top_weights(2)
    x = torch.tensor([[1.0, 8.0], [-8.0, 1.0]], dtype=BF16, device=DEV)
    say("gemm_fp4 bf16 2x%dx2" % TOP)
    check_top(lambda y: mxq.gemm_fp4(x, None, w, s, 2, out=y), x.double() @ v[2:], 2)


@pytest.mark.parametrize("xt", ["bf16", "fp4"])
def test_gemm_one_row_of_most_columns(xt):
    """One row and one block of K at N = 2^31 - 1: more workgroups than a row of the grid takes.  All sums are
    exact in bf16: multiples of 1/2 of at most 72."""
    K = 32
    w, s, v = top_weights(K)
    say("gemm_fp4 %s 1x%dx%d" % (xt, TOP, K))
    xv = torch.zeros((1, K), dtype=F32, device=DEV)
    xv[0, [0, 1, 30, 31]] = torch.tensor([1.0, 4.0, -4.0, 3.0], device=DEV)
    x, xs = mxq.quantize_fp4(xv) if xt == "fp4" else (xv.to(BF16), None)
    check_top(lambda y: mxq.gemm_fp4(x, xs, w, s, K, out=y), xv[:, [0, 1, 30, 31]].double() @ v, 1)


def test_gemm_short_rows_of_many_rows_and_columns():
    """K < 8 where four columns a thread are more than 2^32 threads."""
    M, N, K = 1 << 17, (1 << 17) + 3, 1
    w = torch.full((N, 16), 0x22, dtype=torch.uint8, device=DEV)           # all ones
    s = (torch.arange(N, device=DEV) % 7 + 124).to(torch.uint8)[:, None].contiguous()
    x = (torch.arange(M, device=DEV) % 251).to(BF16)[:, None]
    say("gemm_fp4 bf16 %dx%dx%d" % (M, N, K))
    y = mxq.gemm_fp4(x, None, w, s, K)
    scale = torch.exp2(s[:, 0].float() - 127)
    for c in range(0, M, 4096):
        assert torch.equal(y[c:c + 4096], (x[c:c + 4096].float() * scale).to(BF16)), c


def test_quantize_column_of_most_rows():
    """2^24 tiles of a single column: more workgroups than a row of the grid takes."""
    x = torch.zeros((TOP, 1), dtype=BF16, device=DEV)
    n = 1 << 20
    part = torch.randn((n, 1), device=DEV).to(BF16)
    x[:n], x[TOP - n:] = part, part
    x[1 << 30:(1 << 30) + n] = part
    say("quantize_fp4 %dx1, columns" % TOP)
    c, s = mxq.quantize_fp4(x, "col")
    # the last rows begin inside a block, so their blocks are those of the rows from that block on
    for r in (0, 1 << 30, (TOP - n) // 32 * 32):
        want = mxq.quantize_fp4(x[r:r + n], "col")
        assert torch.equal(c[:, r // 2:(r + n) // 2], want[0][:, :n // 2]) and torch.equal(s[:, r // 32:(r + n) // 32], want[1])
    tail = mxq.quantize_fp4(x[TOP // 32 * 32:], "col")
    assert torch.equal(c[:, TOP // 32 * 16:], tail[0]) and torch.equal(s[:, TOP // 32:], tail[1])
    assert (c[:, n // 2:1 << 29] == 0).all() and (s[:, n // 32:1 << 25] == 127).all()


def gpu_product(x, w):
    """ref.product without an epilogue, in float64 on the GPU."""
    y = x @ w.T
    return y, (x.shape[1] / 32 + 40) * ref.U * (x.abs() @ w.abs().T) + ref.U * y.abs() + 2.0 ** -149


def test_experts_over_many_workgroups():
    """An up product over more workgroups than a row of the grid takes: 1024 experts, one token each, of 2^18
    + 64 columns, 64 a workgroup.  H = 30 keeps the persistent kernel out and leaves codes past H to be
    ignored.  Three of the 16 tokens against float64 on the GPU, with the bounds of ref.moe."""
    T, H, I, E, k = 16, 30, (1 << 18) + 64, 1024, 64
    g = torch.Generator(device=DEV)
    g.manual_seed(51)

    def random(*shape, low=0, high=256):
        return torch.randint(low, high, shape, generator=g, device=DEV, dtype=torch.uint8)
    w13, s13 = random(E, 2 * I, 16), random(E, 2 * I, 4, low=122, high=125)[..., :1]
    w2, s2 = random(E, H, I // 2), random(E, H, I // 32, low=115, high=118)
    x = torch.randn((T, H), generator=g, device=DEV).to(BF16)
    own = torch.arange(E, device=DEV) % T == torch.arange(T, device=DEV)[:, None]
    lg = torch.where(own, torch.randn((T, E), generator=g, device=DEV), torch.tensor(-20.0, device=DEV))
    say("moe_fp4 T%d H%d I%d E%d k%d" % (T, H, I, E, k))
    y = mxq.moe_fp4(x, lg, w13, s13, w2, s2, k, out_dtype=BF16).double()
    for t in (0, 7, 15):
        ids = torch.nonzero(own[t])[:, 0].tolist()
        share = torch.softmax(lg[t, ids].double(), 0).tolist()
        want, bound, total = (torch.zeros(H, dtype=torch.float64, device=DEV) for _ in range(3))
        for e, p in zip(ids, share):
            gu, d = gpu_product(x[t:t + 1].double(), mxq.dequantize_fp4(w13[e], s13[e], H).double())
            gate, up, dg, du = gu[:, :I], gu[:, I:], d[:, :I], d[:, I:]
            act = gate * torch.sigmoid(gate)
            h = p * act * up
            dh = p * (1.1 * dg * (up.abs() + du) + act.abs() * du) + (2.0 ** -19 + 2.0 ** -16) * h.abs()
            v = mxq.dequantize_fp4(w2[e], s2[e], I).double()
            size = ((h.abs() + dh) @ v.abs().T)[0]
            want += (h @ v.T)[0]
            total += size
            bound += (dh @ v.abs().T)[0] + (I / 32 + 40) * ref.U * size
        bound += k * ref.U * total
        bound += 2.0 ** -8 * (want.abs() + bound) + 2.0 ** -149
        assert ((y[t] - want).abs() <= bound).all(), t


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("T,H,I,E", [(3, 32, 16, 4), (3, 32, 16, 264), (200, 72, 120, 512)])
def test_experts_largest_hidden_values(out, T, H, I, E):
    """Hidden values next to FP32's largest, which no single bf16 holds: finite ones stay finite and as exact as
    others, in two and in four launches and in the persistent up product; infinite ones stay infinite.  h = gate * up
    with gate = 2^60 and up = +-1.998046875 * 2^67, the sum of two bf16, in column 0, share 1 (k = 1)."""
    rng = np.random.default_rng(52)
    w13 = np.zeros((E, 2 * I, 16 * ref.blocks(H)), np.uint8)
    w13[:, 0, 0] = 0x02                                                    # column 0's gate, element 0: 1
    w13[:, I, 0], w13[:, I, 1] = 0x20, 0x02                                # and up, elements 1 and 2: 1
    s13 = np.full((E, 2 * I, ref.blocks(H)), 127, np.uint8)
    w2 = np.zeros((E, H, 16 * ref.blocks(I)), np.uint8)
    w2[:, :, 0] = 0x01                                                     # element 0: 1/2
    s2 = np.full((E, H, ref.blocks(I)), 107, np.uint8)                     # 2^-20
    x = np.zeros((T, H))
    x[:, 0], x[:, 1], x[:, 2] = 2.0 ** 60, 1.9921875 * 2.0 ** 67, 0.75 * 2.0 ** 60
    x[1::3, 1:] *= -1
    lg = rng.standard_normal((T, E)).astype(np.float32)

    def stack(t):
        wide = torch.zeros(t.shape[:2] + ((t.shape[2] + 15) // 16 * 16,), dtype=torch.uint8, device=DEV)
        wide[..., :t.shape[2]] = torch.from_numpy(t).to(DEV)
        return wide[..., :t.shape[2]]
    weights = [stack(t) for t in (w13, s13, w2, s2)]
    xd = torch.from_numpy(x.astype(np.float32)).to(BF16).to(DEV)
    assert torch.equal(xd.double().cpu(), torch.from_numpy(x))
    lgd = torch.from_numpy(lg).to(DEV)
    y = mxq.moe_fp4(xd, lgd, *weights, 1, out_dtype=out)
    v13 = ref.values(w13.reshape(-1, w13.shape[2]), s13.reshape(-1, s13.shape[2]), H).reshape(E, 2 * I, H)
    v2 = ref.values(w2.reshape(-1, w2.shape[2]), s2.reshape(-1, s2.shape[2]), I).reshape(E, H, I)
    want, bound = ref.moe(x[:3], lg[:3].astype(np.float64), v13, v2, 1, True, out == BF16)
    n = (T + 2) // 3
    check_product(y, np.tile(want, (n, 1))[:T], np.tile(bound, (n, 1))[:T], "largest hidden values")
    xd[0, 0] = 2.0 ** 62
    y = mxq.moe_fp4(xd, lgd, *weights, 1, out_dtype=out)
    assert torch.isinf(y[0]).all() and torch.isfinite(y[1:]).all()
