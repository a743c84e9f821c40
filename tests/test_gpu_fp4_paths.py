"""Every tile, split and kernel that the MXFP4 product and the expert layer choose from, at sizes that the
host's plans (mxq_gemm_fp4_plan, mxq_moe_fp4_plan) send there; results against float64 on the GPU, with the
bounds of fp4_reference."""
import pytest
import torch

import fp4_reference as ref
import mxfp8_block_scaled_03_amd as mxq
from gpu_helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
CUS = 256


@pytest.fixture(autouse=True)
def device():
    assert torch.cuda.get_device_properties(0).multi_processor_count == CUS


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def operand(g, *shape, low=118, high=128, aligned=True):
    """Random codes [..][16 nb], those past K among them, and scales [..][nb], in rows wider by one block of
    other codes and by bytes 255; scale rows whole 16-byte pieces apart, or an odd number of bytes."""
    nb = ref.blocks(shape[-1])
    codes = torch.randint(0, 256, shape[:-1] + (16 * nb + 16,), generator=g, device=DEV, dtype=torch.uint8)
    wide = torch.full(shape[:-1] + ((nb + 15) // 16 * 16 + (0 if aligned else 1),), 255, device=DEV, dtype=torch.uint8)
    wide[..., :nb] = torch.randint(low, high, shape[:-1] + (nb,), generator=g, device=DEV, dtype=torch.uint8)
    return codes[..., :16 * nb], wide[..., :nb]


def values(codes, scales, K):
    table = torch.tensor(list(ref.MAG) + [-m for m in ref.MAG], dtype=F64, device=DEV)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1))[..., :K]


def rounded(y, bound, bf16):
    return (bound + 2.0 ** -8 * (y.abs() + bound) if bf16 else bound) + 2.0 ** -149


def product(x, w, alpha=1.0, bias=None, act=None, bf16=False):
    """ref.product on the GPU."""
    y = alpha * (x @ w.T)
    bound = abs(alpha) * (x.shape[1] / 32 + 40) * ref.U * (x.abs() @ w.abs().T)
    if bias is not None:
        y = y + bias
    bound = bound + ref.U * y.abs()
    if act == "silu":
        y = y * torch.sigmoid(y)
        bound = 1.1 * bound + 2.0 ** -20 * y.abs() + 2.0 ** -126
    return y, rounded(y, bound, bf16)


def moe(x, logits, w13, s13, w2, s2, k, renorm, bf16):
    """ref.moe on the GPU, for logits without ties or masks, expert by expert."""
    (T, H), (E, I2, _) = x.shape, w13.shape
    I = I2 // 2
    y, bound, total = (torch.zeros((T, H), dtype=F64, device=DEV) for _ in range(3))
    split = 2.0 ** -16 if bf16 else 2.0 ** -24
    ids = torch.topk(logits, k)[1]
    p = torch.softmax(logits, 1)
    for e in torch.unique(ids).tolist():
        t = torch.nonzero((ids == e).any(1))[:, 0]
        share = p[t, e] / (torch.gather(p[t], 1, ids[t]).sum(1) if renorm else 1.0)
        gu, d = product(x[t], values(w13[e], s13[e], H))
        g, u, dg, du = gu[:, :I], gu[:, I:], d[:, :I], d[:, I:]
        act = g * torch.sigmoid(g)
        h = share[:, None] * act * u
        dh = share[:, None] * (1.1 * dg * (u.abs() + du) + act.abs() * du) + (2.0 ** -19 + split) * h.abs()
        v = values(w2[e], s2[e], I)
        size = (h.abs() + dh) @ v.abs().T
        y[t] += h @ v.T
        total[t] += size
        bound[t] += dh @ v.abs().T + (I / 32 + 40) * ref.U * size
    bound = bound + k * ref.U * total
    return y, rounded(y, bound, bf16)


def check(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), "%s: past the bound by %.3g at %s" % (what, off.max().item(), divmod(off.argmax().item(), off.shape[1]))


def test_references_agree():
    """The functions above are those of fp4_reference, the CPU's tests of which hold for them."""
    g = generator(1)
    x, w = torch.randn((5, 70), generator=g, device=DEV, dtype=F64), operand(g, 9, 70)
    v = values(*w, 70)
    assert (v.cpu().numpy() == ref.values(*(t.cpu().numpy() for t in w), 70)).all()
    b = torch.randn(9, generator=g, device=DEV, dtype=F64)
    for got, want in zip(product(x, v, 0.75, b, "silu", True), ref.product(x.cpu().numpy(), v.cpu().numpy(), 0.75, b.cpu().numpy(), "silu", True)):
        assert torch.allclose(got.cpu(), torch.from_numpy(want), rtol=1e-10, atol=0)
    logits = torch.randn((5, 6), generator=g, device=DEV, dtype=F64)
    a, c = operand(g, 6, 40, 70), operand(g, 6, 70, 20)
    host = [torch.stack([values(q[0][e], q[1][e], K) for e in range(6)]).cpu().numpy() for q, K in ((a, 70), (c, 20))]
    for renorm in (True, False):
        for got, want in zip(moe(x, logits, *a, *c, 3, renorm, True), ref.moe(x.cpu().numpy(), logits.cpu().numpy(), *host, 3, renorm, True)):
            assert torch.allclose(got.cpu(), torch.from_numpy(want), rtol=1e-10, atol=1e-300)


# -------------------------------------------------------------------------------- product

FP4, B16 = "fp4", "bf16"
# X, M, N, K, scale rows aligned, (tile_m, tile_n, waves)
PRODUCTS = [
    # the 256 x 256 tiles: K of whole steps of 128 and not, one step, fewer than stages, many; whole and ragged tiles
    (FP4, 2560, 2816, 128, True, (256, 256, 8)), (FP4, 2700, 2817, 256, True, (256, 256, 8)),
    (FP4, 2561, 2820, 640, True, (256, 256, 8)), (FP4, 2816, 2560, 1152, True, (256, 256, 8)),
    (FP4, 3000, 2501, 96, True, (256, 256, 8)), (FP4, 2690, 2690, 33, True, (256, 256, 8)),
    (FP4, 2570, 2999, 2001, True, (256, 256, 8)), (FP4, 3001, 2700, 1, True, (256, 256, 8)),
    (FP4, 26400, 17, 300, True, (256, 256, 8)), (FP4, 3, 27000, 520, True, (256, 256, 8)), (FP4, 30, 27000, 1024, True, (256, 256, 8)),
    # the same sizes with scale rows that are not 16-byte aligned
    (FP4, 2700, 2817, 256, False, (64, 32, 2)), (FP4, 2570, 2999, 2001, False, (64, 64, 1)), (FP4, 3, 27000, 520, False, (16, 32, 4)),
]
for xt in (FP4, B16):
    PRODUCTS += [
        (xt, 1000, 1000, 1300, True, (64, 64, 8)), (xt, 64, 16321, 1100, False, (64, 64, 8)),
        (xt, 64, 19200, 1100, True, (64, 64, 4)), (xt, 130, 6500, 1500, False, (64, 64, 4)),
        (xt, 600, 4096, 1100, True, (64, 64, 2)), (xt, 2100, 2100, 1030, True, (64, 64, 1)),
        (xt, 64, 8192, 1100, True, (32, 64, 8)), (xt, 17, 16383, 2000, False, (32, 64, 8)),
        (xt, 20, 17000, 1040, True, (32, 64, 4)), (xt, 32, 8200, 1100, True, (32, 32, 8)),
        (xt, 64, 4096, 500, True, (32, 32, 4)), (xt, 50, 5001, 1024, False, (32, 32, 4)),
        (xt, 32, 500, 1100, True, (32, 16, 8)), (xt, 30, 500, 100, True, (32, 16, 8)),
        (xt, 16, 8193, 1030, True, (16, 32, 8)), (xt, 5, 8193, 1024, False, (16, 32, 4)),
        (xt, 16, 900, 3001, True, (16, 16, 8)), (xt, 9, 900, 40, True, (16, 16, 4))]
PRODUCTS += [(FP4, 64, 17000, 500, True, (64, 32, 2)), (FP4, 1100, 1100, 1024, True, (64, 32, 2)), (B16, 64, 19200, 500, True, (64, 64, 4)),
             (B16, 600, 4096, 300, True, (64, 64, 2)), (B16, 2100, 2100, 129, True, (64, 64, 1))]
# X in bf16, K shorter than a 16-byte piece, and shorter than a block, by rows, columns and tiles
PRODUCTS += [(B16, M, N, K, True, (1, 4, 0)) for K in range(1, 8) for M, N in ((1, 1), (2, 5), (17, 40), (70, 131))]
PRODUCTS += [(B16, M, N, K, True, tile) for K in (8, 9, 15, 16, 23, 31, 63, 65)
             for M, N, tile in ((1, 3, (16, 16, 4)), (17, 40, (32, 16, 8)), (40, 8300, (32, 32, 4)), (1100, 1100, (64, 64, 4)))]


def plan(xt, M, N, K, aligned):
    return mxq.mxq_gemm_fp4_plan(M, N, K, mxq.MXQ_E2M1 if xt == FP4 else mxq.MXQ_BF16, aligned, CUS)


@pytest.mark.parametrize("xt,M,N,K,aligned,tile", PRODUCTS)
def test_product(xt, M, N, K, aligned, tile):
    """Bias, alpha and SiLU into bf16 rows of an odd pitch, plain sums into fp32 of an odd pitch and into aligned
    bf16; nothing is written beside y."""
    assert plan(xt, M, N, K, aligned) == tile
    say("gemm_fp4 %s %dx%dx%d %s" % (xt, M, N, K, tile))
    g = generator(2)
    w, ws = operand(g, N, K, aligned=aligned)
    wv = values(w, ws, K) / 64
    ws = ws.sub_(6)
    if xt == FP4:
        x, xs = operand(g, M, K, aligned=aligned)
        xv = values(x, xs, K)
    else:
        x, xs = torch.full((M, K + 3), float("nan"), dtype=BF16, device=DEV)[:, 1:K + 1], None
        x.copy_(torch.randn((M, K), generator=g, device=DEV))
        xv = x.double()
    bias = torch.randn(N, generator=g, device=DEV)
    for out, pad, alpha, b, act in ((BF16, N % 2 + 1, 0.75, bias, "silu"), (F32, 1, 1.0, None, None), (BF16, (-N) % 8, 1.0, None, None)):
        wide = torch.full((M + 2, N + pad), 7.0, dtype=out, device=DEV)
        y = wide[1:M + 1, :N]
        mxq.gemm_fp4(x, xs, w, ws, K, alpha=alpha, bias=b, act=act, out=y)
        check(y, *product(xv, wv, alpha, None if b is None else b.double(), act, out == BF16), "%s %s" % (out, act))
        assert (wide[0] == 7.0).all() and (wide[M + 1] == 7.0).all() and (wide[:, N:] == 7.0).all()
        again = torch.empty_like(y)
        mxq.gemm_fp4(x, xs, w, ws, K, alpha=alpha, bias=b, act=act, out=again)
        assert torch.equal(again, y)


def test_products_cover_every_tile():
    """The plans of many sizes are among those above."""
    for xt in (FP4, B16):
        have = {c[5] for c in PRODUCTS if c[0] == xt}
        sizes = [1, 5, 16, 17, 32, 33, 64, 100, 300, 512, 1000, 2048, 4096, 8192, 16384, 32768, 100000]
        found = {plan(xt, M, N, K, a) for M in sizes for N in sizes for K in (1, 5, 8, 300, 1024, 1025, 5000) for a in (True, False)}
        assert found == have


# -------------------------------------------------------------------------------- experts

# T, H, I, E, k, the plans (columns up and down, ranges of I) with y in bf16 and in fp32, and whether x and the
# scale rows are whole 16-byte pieces
EXPERTS = [
    # the persistent down product over 2, 4 and 8 ranges of I
    (15, 2163, 920, 34, 5, (64, 256, 2), (64, 256, 2), True), (14, 4141, 1558, 41, 8, (64, 256, 4), (64, 256, 4), True),
    (25, 1277, 3894, 31, 8, (64, 256, 8), (64, 256, 8), True),
    # the persistent up product, with one group of scale bytes and with more, and experts of more than 16 tokens
    (36, 5056, 2542, 25, 5, (128, 128, 1), (128, 256, 1), True), (64, 2056, 1032, 128, 8, (128, 256, 1), (128, 256, 1), True),
    (200, 72, 120, 512, 8, (128, 128, 1), (128, 32, 1), True),
    # X through the ring a chunk at a time, with more than 16 tokens an expert and a short last chunk
    (10, 1744, 260, 10, 8, (16, 64, 1), (16, 32, 1), True), (50, 1030, 200, 12, 8, (16, 32, 1), (16, 32, 1), True),
    (36, 1600, 1542, 25, 5, (64, 128, 1), (64, 32, 1), False), (36, 1600, 1542, 25, 5, (64, 128, 1), (64, 256, 4), True),
    (30, 1000, 500, 32, 4, (32, 64, 1), (32, 32, 1), True),
    # rows shorter than a 16-byte piece
    (3, 5, 3, 264, 2, (16, 32, 1), (16, 32, 1), True), (20, 7, 33, 264, 3, (16, 32, 1), (16, 32, 1), False),
    (20, 40, 1, 300, 2, (16, 32, 1), (16, 32, 1), True), (70, 3, 700, 300, 4, (64, 32, 1), (64, 32, 1), False),
]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,H,I,E,k,bf16_plan,f32_plan,aligned", EXPERTS)
def test_experts(T, H, I, E, k, bf16_plan, f32_plan, aligned, out):
    got = mxq.mxq_moe_fp4_plan(T, H, I, E, k, mxq.MXQ_BF16 if out == BF16 else mxq.MXQ_F32, aligned, CUS)
    assert got == (4,) + (bf16_plan if out == BF16 else f32_plan)
    say("moe_fp4 T%d H%d I%d E%d k%d %s" % (T, H, I, E, k, got))
    g = generator(3)
    mean = 122 - round(0.5 * torch.tensor(float(max(H, 1))).log2().item())  # products of about 1
    w13 = operand(g, E, 2 * I, H, low=mean, high=mean + 3, aligned=aligned)
    w2 = operand(g, E, H, I, low=mean, high=mean + 3, aligned=aligned)
    x = torch.zeros((T, (H + 7) // 8 * 8 + (0 if aligned else 1)), dtype=BF16, device=DEV)[:, :H]
    x.copy_(torch.randn((T, H), generator=g, device=DEV))
    logits = torch.randn((T, E), generator=g, device=DEV) * 1.5
    for renorm in (True, False):
        wide = torch.full((T + 2, H + 3), 7.0, dtype=out, device=DEV)
        y = wide[1:T + 1, :H]
        mxq.moe_fp4(x, logits, *w13, *w2, k, renormalize=renorm, out=y)
        check(y, *moe(x.double(), logits.double(), *w13, *w2, k, renorm, out == BF16), "renorm %s" % renorm)
        assert (wide[0] == 7.0).all() and (wide[T + 1] == 7.0).all() and (wide[:, H:] == 7.0).all()
        again = torch.empty_like(y)
        mxq.moe_fp4(x, logits, *w13, *w2, k, renormalize=renorm, out=again)
        assert torch.equal(again, y)


def test_experts_cover_every_plan():
    """The plans of many sizes are among those above."""
    for t, at in ((mxq.MXQ_BF16, 5), (mxq.MXQ_F32, 6)):
        have = {c[at] for c in EXPERTS} | {(0, 0, 0)}
        sizes = [(T, H, I, E, k) for T in (1, 7, 16, 40, 200) for H in (5, 64, 1000, 2048, 5120) for I in (5, 64, 520, 2048, 8192)
                 for E in (8, 32, 64, 264) for k in (1, 2, 8)]
        found = {mxq.mxq_moe_fp4_plan(*c, t, a, CUS)[1:] for c in sizes for a in (True, False)}
        assert {p[0] for p in found} <= {p[0] for p in have} and {p[1:] for p in found} <= {p[1:] for p in have}
