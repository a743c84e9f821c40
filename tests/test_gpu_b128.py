"""FP8 in blocks of 128 on the GPU against 64 bits (b128_reference.py): the quantizer bit for bit, the products
within derived bounds."""
import pytest
import torch

import b128_reference as ref
import mxfp8_block_scaled_03_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def wide(rows, cols, dtype, seed, spikes=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g)
    if spikes:
        x = torch.where(torch.rand((rows, cols), generator=g) < 1e-2, x * 1000, x)
        x = x * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    return x.to(dtype)


def coded(lines, K, elem, seed, tile=False):
    """Codes and scales as the reference quantizes them, on the CPU."""
    return ref.quantize(wide(lines, K, F32, seed), elem, tile=tile)


def by_block(scales):
    """Scales of lines as the library takes them: stored block by block."""
    return scales.float().to(DEV).t().contiguous().t()


def same(codes, scales, want, what):
    c, s = want
    assert torch.equal(codes.cpu(), c), "%s: %d codes differ" % (what, int((codes.cpu() != c).sum()))
    assert torch.equal(torch.nan_to_num(scales.cpu().double(), -1.0), torch.nan_to_num(s.double(), -1.0)), what


# ---------------------------------------------------------------------------------- quantize

SIZES = [(1, 1), (1, 128), (3, 129), (128, 128), (127, 255), (130, 300), (17, 1000), (300, 64), (257, 513), (512, 640)]


@pytest.mark.parametrize("rule", ["amax", "ceil"])
@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize(rows, cols, dtype, elem, rule):
    x = wide(rows, cols, dtype, rows * 1000 + cols)
    d = x.to(DEV)
    row, col = ref.quantize(x, elem, rule), ref.quantize(x.T, elem, rule)
    same(*mxq.quantize_b128(d, elem, "row", rule), row, "row")
    same(*mxq.quantize_b128(d, elem, "col", rule), col, "col")
    rc, rs, cc, cs = mxq.quantize_b128_dual(d, elem, rule=rule)
    same(rc, rs, row, "dual rows")
    same(cc, cs, col, "dual columns")
    tile = ref.quantize(x, elem, rule, tile=True)
    same(*mxq.quantize_b128(d, elem, "tile", rule), tile, "tile")
    tc, ts, ttc, tts = mxq.quantize_b128_dual(d, elem, tile=True, rule=rule)
    same(tc, ts, tile, "tiles")
    same(ttc, tts, ref.quantize(x.T, elem, rule, tile=True), "tiles transposed")


def test_quantize_large_rows_take_the_wide_kernel():
    x = wide(2048, 4200, BF16, 5)
    same(*mxq.quantize_b128(x.to(DEV)), ref.quantize(x, "e4m3"), "row")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
def test_quantize_special_values(dtype, elem):
    """Zero blocks, signed zeros, subnormals, tiny and huge blocks, NaN and infinities (each in a block of its own)."""
    x = wide(130, 400, F32, 9)
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= 2.0 ** -140
    x[3] = 2.0 ** -101
    x[4] = 3.0e38 * torch.sign(x[4])
    x[5, 3] = float("nan")
    x[6, 130] = float("inf")
    x[7, 399] = float("-inf")
    x[129, 0] = 1e-45
    x = x.to(dtype)
    d = x.to(DEV)
    for rule in ("amax", "ceil"):
        same(*mxq.quantize_b128(d, elem, "row", rule), ref.quantize(x, elem, rule), "row " + rule)
        rc, rs, cc, cs = mxq.quantize_b128_dual(d, elem, rule=rule)
        same(cc, cs, ref.quantize(x.T, elem, rule), "col " + rule)
        tc, ts, ttc, tts = mxq.quantize_b128_dual(d, elem, tile=True, rule=rule)
        same(tc, ts, ref.quantize(x, elem, rule, tile=True), "tile " + rule)
        same(ttc, tts, ref.quantize(x.T, elem, rule, tile=True), "tile transposed " + rule)


@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
def test_quantize_every_bf16_value(elem):
    """Every finite bf16 value beside a block maximum that it does not pass."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    v = v[torch.isfinite(v)]
    a = torch.where(v.float().abs() == 0, torch.ones(len(v)), v.float().abs() * 1.37).clamp(max=3.3e38)
    x = torch.zeros((len(v), 2))
    x[:, 0], x[:, 1] = v.float(), a
    same(*mxq.quantize_b128(x.to(DEV), elem), ref.quantize(x, elem), "row")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_strides_and_alignment(dtype):
    """Row pitches and bases that no 16-byte load can take, and ones that it can."""
    big = wide(140, 517, dtype, 3).to(DEV)
    for x in (big[3:133, 1:300], big[:, 8:264], big[::2, :511], big[:1].expand(1, 517)):
        want = ref.quantize(x.cpu(), "e4m3")
        same(*mxq.quantize_b128(x), want, "row %s" % (x.stride(),))
        same(*mxq.quantize_b128(x, axis="col"), ref.quantize(x.cpu().T, "e4m3"), "col")


SPLITS = [[5], [128, 128], [0, 7, 0, 300, 128, 1], [0, 0, 0], [129, 0, 127, 1, 1, 255] + [0] * 60 + [3] * 10]


@pytest.mark.parametrize("sizes", SPLITS)
def test_quantize_by_expert(sizes):
    """Blocks of columns begin anew with every expert; rows of no expert are skipped."""
    E, used = len(sizes), sum(sizes)
    x = wide(used + 9, 200, BF16, 11 + E)
    offsets = torch.tensor([0] + sizes).cumsum(0).int().to(DEV)
    rc, rs, cc, cs = mxq.quantize_b128_dual(x.to(DEV), offsets=offsets)
    c1, s1 = mxq.quantize_b128(x.to(DEV), axis="col", offsets=offsets)
    row = ref.quantize(x, "e4m3")
    same(rc[:used], rs[:used], (row[0][:used], row[1][:used]), "rows")
    first = block = 0
    assert cc.shape[1] == (used + 9 + 127 * E) // 128 * 128
    for n in sizes:
        want = ref.quantize(x[first:first + n].T, "e4m3")
        nb = ref.blocks(n)
        for c, s in ((cc, cs), (c1, s1)):
            same(c[:, 128 * block:128 * (block + nb)], s[:, block:block + nb], want, "expert of %d rows" % n)
        first, block = first + n, block + nb


def test_quantize_empty():
    for shape in ((0, 5), (5, 0), (0, 0)):
        x = torch.empty(shape, device=DEV)
        c, s = mxq.quantize_b128(x)
        assert c.shape == (shape[0], 128 * ref.blocks(shape[1])) and s.shape == (shape[0], ref.blocks(shape[1]))
        mxq.quantize_b128_dual(x, tile=True)


# ---------------------------------------------------------------------------------- products

def run_product(M, N, K, fx="e4m3", fw="e4m3", lines=False, accum="fp32", out=F32, alpha=1.0, bias=False, act=None, seed=0):
    xc, xs = coded(M, K, fx, seed + 1)
    wc, ws = coded(N, K, fw, seed + 2, tile=not lines)
    g = torch.Generator().manual_seed(seed)
    b = torch.randn(N, generator=g) if bias else None
    want, tol = ref.product(xc, xs.float(), fx, wc, ws.float(), fw, accum, alpha, b, act, out)
    got = mxq.gemm_b128(xc.to(DEV), by_block(xs), wc.to(DEV), by_block(ws) if lines else ws.float().to(DEV), K, fx, fw,
                        alpha=alpha, bias=None if b is None else b.to(DEV), out_dtype=out, accum=accum, act=act)
    ref.check(got, want, tol, "%dx%dx%d %s %s %s" % (M, N, K, accum, out, "lines" if lines else "tiles"))


# every kernel: rows of 16 to 64, 64 x 64 tiles and 256 x 256 ones, whole and ragged
SHAPES = [(1, 1, 1), (1, 130, 128), (16, 64, 256), (15, 17, 1100), (20, 200, 300), (33, 95, 2100), (64, 256, 640),
          (70, 130, 129), (200, 70, 1000), (257, 300, 400)]


@pytest.mark.parametrize("lines", [False, True])
@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, out, accum, lines):
    run_product(M, N, K, lines=lines, accum=accum, out=out, seed=M + N)


@pytest.mark.parametrize("fx,fw", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("M,N,K", [(10, 40, 200), (130, 70, 300)])
def test_product_formats(M, N, K, accum, fx, fw):
    for lines in (False, True):
        run_product(M, N, K, fx, fw, lines, accum, seed=7)


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("M,N,K", [(5, 37, 300), (100, 201, 300)])
def test_product_epilogue(M, N, K, act):
    for out in (F32, BF16):
        run_product(M, N, K, accum="fp32", out=out, alpha=-0.375, bias=True, act=act, seed=3)


# sizes that take each kernel of tiles, whole and ragged, two tiles a CU and one, and the tile of the 256 x 256 kernel that
# is the last of its row and column
TILED = [((64, 64, 0), (1280, 640, 1280)), ((64, 64, 0), (1300, 1090, 300)), ((64, 64, 0), (2570, 700, 129)),
         ((128, 128, 0), (2048, 2048, 1280)), ((128, 128, 0), (1900, 2100, 900)), ((128, 128, 0), (3000, 3000, 640)),
         ((256, 256, 0), (4000, 4090, 1300)), ((256, 256, 0), (4090, 4001, 1700))]


def tiled(M, N, K, accum, lines, out, fx="e4m3", fw="e4m3"):
    """A large problem: every 17th row and 13th column, and the last ones, against the reference."""
    x, w = wide(M, K, BF16, 21).to(DEV), wide(N, K, BF16, 22).to(DEV)
    xc, xs = mxq.quantize_b128(x, fx)
    wc, ws = mxq.quantize_b128(w, fw, "row" if lines else "tile")
    got = mxq.gemm_b128(xc, xs, wc, ws, K, fx, fw, accum=accum, out_dtype=out)
    rows = torch.tensor(sorted(set(range(0, M, 17)) | set(range(max(0, M - 20), M))))
    cols = torch.tensor(sorted(set(range(0, N, 13)) | set(range(max(0, N - 20), N))))
    wsl = ws.cpu() if lines else ws.cpu().repeat_interleave(128, 0)[:N]
    want, tol = ref.product(xc.cpu()[rows], xs.cpu()[rows], fx, wc.cpu()[cols], wsl[cols], fw, accum, out=out)
    ref.check(got.cpu()[rows][:, cols], want, tol, "%dx%dx%d %s" % (M, N, K, accum))


@pytest.mark.parametrize("lines", [False, True])
@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("M,N,K", [(1000, 1000, 4001), (900, 1000, 640), (961, 1024, 300), (1000, 1000, 1)])
def test_product_small_tiles_alone_on_their_cu(M, N, K, accum, lines):
    """Tiles of 64, fewer than CUs: their waves share the blocks, an odd number of them too."""
    assert -(-M // 64) * -(-N // 64) <= 256
    tiled(M, N, K, accum, lines, F32)
    tiled(M, N, K, accum, lines, BF16, "e5m2", "e4m3")


@pytest.mark.parametrize("lines", [False, True])
@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("tile,size", TILED)
def test_product_tiled(tile, size, accum, lines):
    M, N, K = size
    assert mxq.mxq_gemm_b128_plan(0, M, N, K, 1, 1 if lines else 128, 0 if accum == "fp8" else 1, 256) == tile
    tiled(M, N, K, accum, lines, F32)
    tiled(M, N, K, accum, lines, BF16)


@pytest.mark.parametrize("M,N,K", [(700, 900, 200), (1900, 2100, 200), (4001, 4003, 1300)])
def test_product_tiled_formats(M, N, K):
    for fx, fw in (("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")):
        for accum in ("fp32", "fp8"):
            for lines in (False, True):
                tiled(M, N, K, accum, lines, F32, fx, fw)


def test_product_tiled_epilogue():
    """Bias, alpha and SiLU in every kernel, columns that end inside a group of four."""
    for M, N, K in ((20, 203, 200), (120, 803, 1000), (640, 1201, 200), (4001, 4003, 200), (4001, 4003, 1300)):
        for act in (None, "silu"):
            xc, xs = mxq.quantize_b128(wide(M, K, BF16, 1, False).to(DEV))
            wc, ws = mxq.quantize_b128(wide(N, K, BF16, 2, False).to(DEV))
            b = torch.randn(N, generator=torch.Generator().manual_seed(3))
            got = mxq.gemm_b128(xc, xs, wc, ws, K, alpha=0.625, bias=b.to(DEV), act=act, out_dtype=F32)
            rows = torch.arange(0, M, 1 + M // 60)
            want, tol = ref.product(xc.cpu()[rows], xs.cpu()[rows], "e4m3", wc.cpu(), ws.cpu(), "e4m3", "fp32", 0.625, b, act)
            ref.check(got.cpu()[rows], want, tol, "%dx%d %s" % (M, N, act))


def test_product_into_strided_output_leaves_the_rest():
    for M, N, K in ((5, 33, 256), (100, 100, 256), (640, 1203, 256), (4001, 4003, 256), (4001, 4003, 1300)):
        for dtype in (F32, BF16):
            for pad in (3, 8):
                whole = torch.full((M + 2, N + pad), 7.0, dtype=dtype, device=DEV)
                xc, xs = mxq.quantize_b128(wide(M, K, BF16, 1).to(DEV))
                wc, ws = mxq.quantize_b128(wide(N, K, BF16, 2).to(DEV), axis="tile")
                want = mxq.gemm_b128(xc, xs, wc, ws, K, out_dtype=dtype)
                mxq.gemm_b128(xc, xs, wc, ws, K, out=whole[1:1 + M, :N])
                assert torch.equal(whole[1:1 + M, :N], want)
                rest = whole.clone()
                rest[1:1 + M, :N] = 7.0
                assert bool((rest == 7.0).all())


def test_product_no_blocks():
    b = torch.randn(40, device=DEV)
    z = torch.empty((3, 0), dtype=torch.uint8, device=DEV)
    w = torch.empty((40, 0), dtype=torch.uint8, device=DEV)
    xs, ws = torch.empty((3, 0), device=DEV), torch.empty((1, 0), device=DEV)
    assert torch.equal(mxq.gemm_b128(z, xs, w, ws, 0, bias=b, out_dtype=F32), b.expand(3, 40))
    assert bool((mxq.gemm_b128(z, xs, w, ws, 0, out_dtype=F32) == 0).all())


def test_experts_without_rows_or_blocks():
    """No rows: nothing is written, and weight gradients are zero; no blocks along K: zeros."""
    off = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device=DEV)
    y = torch.full((7, 40), 5.0, device=DEV)
    for accum in ("fp32", "fp8"):
        y.fill_(5.0)
        mxq.moe_gemm_b128(torch.empty((7, 0), dtype=torch.uint8, device=DEV), torch.empty((7, 0), device=DEV),
                          torch.empty((3, 40, 0), dtype=torch.uint8, device=DEV), torch.empty((3, 1, 0), device=DEV),
                          off, 0, out=y, accum=accum)
        assert bool((y[:5] == 0).all()) and bool((y[5:] == 5.0).all())
        z, none = torch.empty((0, 130), device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
        c, s = mxq.quantize_b128(z)
        wc = torch.zeros((3, 40, 256), dtype=torch.uint8, device=DEV)
        assert mxq.moe_gemm_b128(c, s, wc, torch.ones((3, 1, 2), device=DEV), none, 130, accum=accum).shape == (0, 40)
        gc, gs = mxq.quantize_b128(torch.empty((0, 40), device=DEV), "e5m2", "col", offsets=none)
        c, s = mxq.quantize_b128(z, "e4m3", "col", offsets=none)
        dw = mxq.moe_wgrad_b128(gc, gs, c, s, none, out=torch.full((3, 40, 130), 5.0, device=DEV), accum=accum)
        assert bool((dw == 0).all())


def test_product_nan_scale():
    """A block whose scale is NaN makes its row (of X) or its columns (of W) NaN and nothing else."""
    for M, N in ((4, 300), (300, 300)):
        x, w = wide(M, 300, F32, 1, False), wide(N, 300, F32, 2, False)
        x[2, 150] = float("nan")
        w[5, 0] = float("inf")
        for lines in (True, False):
            for accum in ("fp32", "fp8"):
                xc, xs = mxq.quantize_b128(x.to(DEV))
                wc, ws = mxq.quantize_b128(w.to(DEV), axis="row" if lines else "tile")
                y = mxq.gemm_b128(xc, xs, wc, ws, 300, accum=accum, out_dtype=F32).cpu()
                nan = torch.zeros((M, N), dtype=torch.bool)
                nan[2] = True
                nan[:, 5:6] = True
                if not lines:
                    nan[:, :128] = True
                assert torch.equal(torch.isnan(y), nan)


def test_transposed_tiles_are_the_weights_transposed():
    """dX = dY W from the transposed codes of the same tiles."""
    N, K, M = 300, 200, 50
    w = wide(N, K, BF16, 4).to(DEV)
    wc, ws, wt, wts = mxq.quantize_b128_dual(w, tile=True)
    dc, ds = mxq.quantize_b128(wide(M, N, BF16, 5).to(DEV), "e5m2")
    got = mxq.gemm_b128(dc, ds, wt, wts, N, "e5m2", out_dtype=F32)
    wv = ref.values(wc.cpu(), ws.cpu(), "e4m3")[:, :K]
    dv = ref.values(dc.cpu(), ds.cpu(), "e5m2")[:, :N]
    tol = (ref.blocks(N) + 50) * ref.U * (dv.abs() @ wv.abs())
    ref.check(got, dv @ wv, tol, "dx")


# ---------------------------------------------------------------------------------- experts

def experts_case(sizes, N, K, extra, accum, out, lines, seed=0):
    E, used = len(sizes), sum(sizes)
    R = used + extra
    xc, xs = coded(R, K, "e4m3", seed + 1)
    w = [coded(N, K, "e4m3", seed + 10 + e, tile=not lines) for e in range(E)]
    wc, ws = torch.stack([c for c, _ in w]), torch.stack([s for _, s in w]).float()
    offsets = torch.tensor([0] + sizes).cumsum(0).int().to(DEV)
    y = torch.full((R, N), 5.0, dtype=out, device=DEV)
    wsd = ws.to(DEV)
    if lines:
        wsd = wsd.transpose(1, 2).contiguous().transpose(1, 2)
    mxq.moe_gemm_b128(xc.to(DEV), by_block(xs), wc.to(DEV), wsd, offsets, K, out=y, accum=accum)
    first = 0
    for e, n in enumerate(sizes):
        if n:
            want, tol = ref.product(xc[first:first + n], xs[first:first + n].float(), "e4m3", wc[e], ws[e], "e4m3", accum, out=out)
            ref.check(y[first:first + n], want, tol, "expert %d of %d rows" % (e, n))
        first += n
    assert bool((y[used:] == 5.0).all()), "rows of no expert were written"


@pytest.mark.parametrize("lines", [False, True])
@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("sizes", [[1], [0, 3, 0, 17, 1], [40, 0, 33, 70], [100, 200, 0, 90], [0, 0], [1] * 70])
def test_experts(sizes, accum, lines):
    for out in (F32, BF16):
        experts_case(sizes, 100, 300, 3, accum, out, lines)


# the kernels that rows of experts may take: their numbers of rows, columns and plan
EXPERT_TILES = [((16, 64, 1), [2, 0, 17, 1] + [1] * 6 + [0] * 10, 4200, 384), ((64, 64, 0), [300, 0, 1, 70, 64, 65], 900, 384),
                ((128, 128, 0), [700, 0, 1, 1300], 4100, 640), ((256, 256, 0), [1300, 0, 2500], 3000, 1280)]


@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("lines", [False, True])
@pytest.mark.parametrize("tile,sizes,N,K", EXPERT_TILES)
def test_experts_tiled(tile, sizes, N, K, lines, accum):
    E, R = len(sizes), sum(sizes) + 11
    assert mxq.mxq_gemm_b128_plan(1, R, N, K, E, 1 if lines else 128, 0 if accum == "fp8" else 1, 256) == tile
    xc, xs = mxq.quantize_b128(wide(R, K, BF16, 3).to(DEV))
    wc, ws = mxq.quantize_b128(wide(E * N, K, BF16, 4).to(DEV), axis="row")
    wc, ws = wc.view(E, N, -1), ws.t().contiguous().view(-1, E, N).permute(1, 2, 0)
    wl = ws
    if not lines:       # (any scales may be a tile's)
        ws = torch.exp2(torch.randint(-12, -4, (E, ref.blocks(N), ref.blocks(K)), device=DEV).float()) * 1.25
        wl = ws.repeat_interleave(128, 1)[:, :N]
    offsets = torch.tensor([0] + sizes).cumsum(0).int().to(DEV)
    y = torch.full((R, N), 5.0, device=DEV)
    mxq.moe_gemm_b128(xc, xs, wc, ws, offsets, K, out=y, accum=accum)
    first = 0
    for e, n in enumerate(sizes):
        rows = torch.tensor(sorted(set(range(first, first + n, 7)) | set(range(first + max(0, n - 3), first + n))), dtype=torch.int64)
        cols = torch.tensor(sorted(set(range(e, N, 23)) | {N - 1}))
        if n:
            want, tol = ref.product(xc.cpu()[rows], xs.cpu()[rows], "e4m3", wc[e].cpu()[cols], wl[e].cpu()[cols], "e4m3", accum)
            ref.check(y.cpu()[rows][:, cols], want, tol, "expert %d" % e)
        first += n
    assert bool((y[first:] == 5.0).all())


@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("N,K", [(20, 30), (300, 70), (600, 900), (2600, 2500)])
@pytest.mark.parametrize("sizes", [[40], [0, 130, 1, 0, 257], [128, 0, 128], [1000, 0, 3]])
def test_expert_weight_gradients(sizes, N, K, accum):
    E, R = len(sizes), sum(sizes) + 5
    dy, x = wide(R, N, BF16, 6, False), wide(R, K, BF16, 7, False)
    offsets = torch.tensor([0] + sizes).cumsum(0).int().to(DEV)
    dc, ds = mxq.quantize_b128(dy.to(DEV), "e5m2", "col", offsets=offsets)
    xc, xs = mxq.quantize_b128(x.to(DEV), "e4m3", "col", offsets=offsets)
    for out in (F32, BF16):
        got = mxq.moe_wgrad_b128(dc, ds, xc, xs, offsets, out_dtype=out, accum=accum)
        block = 0
        pick_n, pick_k = torch.arange(0, N, 1 + N // 150), torch.arange(0, K, 1 + K // 150)
        for e, n in enumerate(sizes):
            nb = ref.blocks(n)
            part = [t.cpu() for t in (dc[:, 128 * block:128 * (block + nb)], ds[:, block:block + nb],
                                      xc[:, 128 * block:128 * (block + nb)], xs[:, block:block + nb])]
            want, tol = ref.product(part[0][pick_n], part[1][pick_n], "e5m2", part[2][pick_k], part[3][pick_k], "e4m3", accum,
                                    out=out)
            ref.check(got[e].cpu()[pick_n][:, pick_k], want, tol, "expert %d of %d rows" % (e, n))
            block += nb


# the kernels that the experts' weight gradients may take; the later ones' outputs in fp32 are past 128 MiB
GRAD_TILES = [((64, 64, 0), [100, 0, 70, 300], 512, 500), ((128, 128, 0), [30, 0, 129] + [1] * 7, 1999, 2003),
              ((256, 256, 0), [4000, 5000, 0, 6000], 8001, 2041)]


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("tile,sizes,N,K", GRAD_TILES)
def test_expert_weight_gradients_tiled(tile, sizes, N, K, accum, out):
    """Every kernel, into an output of odd pitch: every expert's values, and nothing beside them."""
    E, R = len(sizes), sum(sizes) + 5
    assert mxq.mxq_gemm_b128_plan(2, N, K, R, E, 1, 0 if accum == "fp8" else 1, 256) == tile
    dy, x = torch.randn((R, N), device=DEV, dtype=BF16), torch.randn((R, K), device=DEV, dtype=BF16)
    offsets = torch.tensor([0] + sizes).cumsum(0).int().to(DEV)
    dc, ds = mxq.quantize_b128(dy, "e5m2", "col", offsets=offsets)
    xc, xs = mxq.quantize_b128(x, "e4m3", "col", offsets=offsets)
    whole = torch.full((E, N + 1, K + 3), 5.0, dtype=out, device=DEV)
    got = mxq.moe_wgrad_b128(dc, ds, xc, xs, offsets, out=whole[:, :N, :K], accum=accum)
    pick_n = torch.tensor(sorted(set(range(0, N, 1 + N // 60)) | {N - 1}))
    pick_k = torch.tensor(sorted(set(range(0, K, 1 + K // 60)) | {K - 1}))
    block = 0
    for e, n in enumerate(sizes):
        nb = ref.blocks(n)
        part = [t.cpu() for t in (dc[:, 128 * block:128 * (block + nb)], ds[:, block:block + nb],
                                  xc[:, 128 * block:128 * (block + nb)], xs[:, block:block + nb])]
        want, tol = ref.product(part[0][pick_n], part[1][pick_n], "e5m2", part[2][pick_k], part[3][pick_k], "e4m3", accum, out=out)
        ref.check(got[e].cpu()[pick_n][:, pick_k], want, tol, "expert %d of %d rows" % (e, n))
        block += nb
    assert bool((whole[:, N:] == 5.0).all()) and bool((whole[:, :, K:] == 5.0).all())
    dense = torch.empty((E, N, K), dtype=out, device=DEV)
    assert torch.equal(mxq.moe_wgrad_b128(dc, ds, xc, xs, offsets, out=dense, accum=accum), got)


@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("E", [64, 65, 130])
def test_many_experts(E, accum):
    """More experts than lanes: products of a few rows each and weight gradients, every expert's."""
    sizes = [(7 * e) % 11 for e in range(E)]
    N, K, R = 200, 140, sum(sizes) + 3
    assert R > 3 * E
    offsets = torch.tensor([0] + sizes).cumsum(0).int().to(DEV)
    xc, xs = mxq.quantize_b128(wide(R, K, BF16, 31).to(DEV))
    wc, ws = mxq.quantize_b128(wide(E * N, K, BF16, 32).to(DEV), axis="row")
    wc, ws = wc.view(E, N, -1), ws.t().contiguous().view(-1, E, N).permute(1, 2, 0)
    y = torch.full((R, N), 5.0, device=DEV)
    mxq.moe_gemm_b128(xc, xs, wc, ws, offsets, K, out=y, accum=accum)
    dc, ds = mxq.quantize_b128(wide(R, N, BF16, 33, False).to(DEV), "e5m2", "col", offsets=offsets)
    cc, cs = mxq.quantize_b128(wide(R, K, BF16, 34, False).to(DEV), "e4m3", "col", offsets=offsets)
    dw = mxq.moe_wgrad_b128(dc, ds, cc, cs, offsets, accum=accum)
    xc, xs, wc, ws, dc, ds, cc, cs, y, dw = (t.cpu() for t in (xc, xs, wc, ws, dc, ds, cc, cs, y, dw))
    first = block = 0
    for e, n in enumerate(sizes):
        if n:
            want, tol = ref.product(xc[first:first + n], xs[first:first + n], "e4m3", wc[e], ws[e], "e4m3", accum)
            ref.check(y[first:first + n], want, tol, "expert %d" % e)
        nb = ref.blocks(n)
        at = slice(128 * block, 128 * (block + nb))
        want, tol = ref.product(dc[:, at], ds[:, block:block + nb], "e5m2", cc[:, at], cs[:, block:block + nb], "e4m3", accum)
        ref.check(dw[e], want, tol, "gradient %d" % e)
        first += n
        block += nb
    assert bool((y[first:] == 5.0).all())


def test_wrong_offsets_stay_inside():
    """Offsets out of order or past the rows: unspecified results, but none outside the arrays."""
    R, N, K, E = 70, 40, 130, 4
    xc, xs = mxq.quantize_b128(wide(R, K, BF16, 1).to(DEV))
    wc, ws = mxq.quantize_b128(wide(E * N, K, BF16, 2).to(DEV))
    wc, ws = wc.view(E, N, -1), ws.t().contiguous().view(-1, E, N).permute(1, 2, 0)
    for o in ([0, 900, -5, 60, 70], [50, 10, 70, 0, 80], [-3, -2, -1, 0, 1]):
        off = torch.tensor(o, dtype=torch.int32, device=DEV)
        whole = torch.full((R + 64, N), 5.0, device=DEV)
        mxq.moe_gemm_b128(xc, xs, wc, ws, off, K, out=whole[:R])
        assert bool((whole[R:] == 5.0).all())
        rc, rs, cc, cs = mxq.quantize_b128_dual(wide(R, K, BF16, 3).to(DEV), offsets=off)
        mxq.moe_wgrad_b128(cc, cs, cc, cs, off, x_elem="e4m3")
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------------- streams, graphs

def test_side_stream_and_graph():
    """On a stream of its own, and captured: every replay on new inputs equals the eager result."""
    M, N, K, E = 300, 260, 400, 5
    x = wide(M, K, BF16, 1).to(DEV)
    w = wide(E * N, K, BF16, 2).to(DEV)
    wc, ws = mxq.quantize_b128(w)
    wc, ws = wc.view(E, N, -1), ws.t().contiguous().view(-1, E, N).permute(1, 2, 0)
    offsets = torch.tensor([0, 20, 20, 150, 290, 300], dtype=torch.int32, device=DEV)

    def step():
        rc, rs, cc, cs = mxq.quantize_b128_dual(x, offsets=offsets)
        y = mxq.moe_gemm_b128(rc, rs, wc, ws, offsets, K)
        dw = mxq.moe_wgrad_b128(cc, cs, cc, cs, offsets, x_elem="e4m3", accum="fp8")
        return y, dw, mxq.gemm_b128(rc, rs, wc[0], ws[0], K, accum="fp8")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs = step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (3, 4, 5):
        x.copy_(wide(M, K, BF16, seed).to(DEV))
        offsets.copy_(torch.tensor([0, 20 * seed, 20 * seed, 150, 290, 300], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


def test_results_do_not_change_from_run_to_run():
    M, N, K = 900, 1000, 2000
    xc, xs = mxq.quantize_b128(wide(M, K, BF16, 1).to(DEV))
    wc, ws = mxq.quantize_b128(wide(N, K, BF16, 2).to(DEV), axis="tile")
    y = mxq.gemm_b128(xc, xs, wc, ws, K, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(mxq.gemm_b128(xc, xs, wc, ws, K, out_dtype=F32), y)


def test_subnormal_and_extreme_codes():
    """Every finite code against every finite code, exactly: one product each in a block of its own."""
    for fx, fw in (("e4m3", "e4m3"), ("e5m2", "e5m2"), ("e4m3", "e5m2")):
        tx, tw = ref.decode_table(fx), ref.decode_table(fw)
        cx, cw = [torch.arange(256)[torch.isfinite(t)].to(torch.uint8) for t in (tx, tw)]
        x = torch.zeros((len(cx), 128), dtype=torch.uint8)
        w = torch.zeros((len(cw), 128), dtype=torch.uint8)
        x[:, 5], w[:, 5] = cx, cw
        one = [torch.ones((len(c), 1), device=DEV) for c in (cx, cw)]
        want = tx[cx.long()][:, None] * tw[cw.long()][None]
        for accum in ("fp32", "fp8"):
            got = mxq.gemm_b128(x.to(DEV), one[0], w.to(DEV), one[1], 128, fx, fw, accum=accum, out_dtype=F32)
            assert torch.equal(got.cpu().double(), want), (fx, fw, accum)
            big = [t.to(DEV).repeat(12, 1) for t in (x, w)]
            ones = [torch.ones((t.shape[0], 1), device=DEV) for t in big]
            got = mxq.gemm_b128(big[0], ones[0], big[1], ones[1], 128, fx, fw, accum=accum, out_dtype=F32)
            assert torch.equal(got.cpu().double(), want.repeat(12, 12)), (fx, fw, accum)


def test_nan_codes():
    """A NaN code under a finite scale makes its row and column NaN, in both modes and every kernel."""
    for M, N in ((3, 40), (100, 80), (700, 900), (4001, 4003)):
        for accum in ("fp32", "fp8"):
            x, w = torch.full((M, 128), 0x38, dtype=torch.uint8), torch.full((N, 128), 0x38, dtype=torch.uint8)
            x[2, 77], w[N - 1, 0] = 0x7F, 0xFF
            y = mxq.gemm_b128(x.to(DEV), torch.ones((M, 1), device=DEV), w.to(DEV), torch.ones((N, 1), device=DEV), 128,
                              accum=accum, out_dtype=F32).cpu()
            nan = torch.zeros((M, N), dtype=torch.bool)
            nan[2], nan[:, N - 1] = True, True
            assert torch.equal(torch.isnan(y), nan) and bool((y[~nan] == 128.0).all())


def test_rows_past_32_bit_offsets():
    """Codes and outputs whose byte offsets pass 2^32."""
    M, K, N = 70000, 65536, 40
    codes = torch.zeros((M, K), dtype=torch.uint8, device=DEV)
    codes[-3:] = torch.randint(1, 100, (3, K), device=DEV).to(torch.uint8)
    scales = torch.ones((K // 128, M), device=DEV).t()
    w, ws = mxq.quantize_b128(wide(N, K, BF16, 1, False).to(DEV))
    y = mxq.gemm_b128(codes, scales, w, ws, K, out_dtype=F32)
    few = mxq.gemm_b128(codes[-3:].clone(), scales[-3:].t().contiguous().t(), w, ws, K, out_dtype=F32)
    want, tol = ref.product(codes[-3:].cpu(), scales[-3:].cpu(), "e4m3", w.cpu(), ws.cpu(), "e4m3", "fp32")
    ref.check(y[-3:], want, tol, "last rows")
    ref.check(few, want, tol, "the same alone")
    assert bool((y[:-3] == 0).all())
    del codes, y
    x = torch.zeros((70000, 32768), dtype=BF16, device=DEV)        # 4.6e9 bytes
    x[-1] = wide(1, 32768, BF16, 2, False)[0].to(DEV)
    rc, rs, cc, cs = mxq.quantize_b128_dual(x)
    c, s = ref.quantize(x[-1:].cpu(), "e4m3")
    same(rc[-1:], rs[-1:], (c, s), "last row")
    assert bool((rc[:-1] == 0).all()) and bool((rs[:-1] == 1).all())
    amax = x[-1].float().abs().cpu().double()
    assert torch.equal(cs[:, -1].cpu().double(), torch.where(amax == 0, 1.0, (amax / 448).float().double()))


def test_broadcast_and_strided_operands():
    """Scales of one tile for all, weights of one expert for all, rows of a wider array."""
    M, N, K, E = 60, 70, 260, 3
    xw, xs = mxq.quantize_b128(wide(M, K, BF16, 1).to(DEV))
    wide_codes = torch.zeros((M, 640), dtype=torch.uint8, device=DEV)
    wide_codes[:, :384] = xw
    wc, ws = mxq.quantize_b128(wide(N, K, BF16, 2).to(DEV))
    one = torch.full((1, 1), 0.5, device=DEV).expand(1, 3)
    got = mxq.gemm_b128(wide_codes, xs, wc, one, K, out_dtype=F32)
    want, tol = ref.product(xw.cpu(), xs.cpu(), "e4m3", wc.cpu(), torch.full((N, 3), 0.5), "e4m3", "fp32")
    ref.check(got, want, tol, "one scale for all")
    offsets = torch.tensor([0, 10, 40, 60], dtype=torch.int32, device=DEV)
    y = mxq.moe_gemm_b128(wide_codes, xs, wc.expand(E, N, -1), ws.expand(E, N, 3), offsets, K, out_dtype=F32)
    want, tol = ref.product(xw.cpu(), xs.cpu(), "e4m3", wc.cpu(), ws.cpu(), "e4m3", "fp32")
    ref.check(y, want, tol, "one expert for all")


def test_two_streams_at_once():
    """The same operands on two streams, call beside call."""
    M, N, K, E = 500, 600, 700, 4
    xc, xs = mxq.quantize_b128(wide(M, K, BF16, 1).to(DEV))
    wc, ws = mxq.quantize_b128(wide(E * N, K, BF16, 2).to(DEV))
    wc, ws = wc.view(E, N, -1), ws.t().contiguous().view(-1, E, N).permute(1, 2, 0)
    offsets = torch.tensor([0, 100, 130, 131, 500], dtype=torch.int32, device=DEV)
    want = mxq.moe_gemm_b128(xc, xs, wc, ws, offsets, K), mxq.gemm_b128(xc, xs, wc[1], ws[1], K)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((mxq.moe_gemm_b128(xc, xs, wc, ws, offsets, K), mxq.gemm_b128(xc, xs, wc[1], ws[1], K)))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


# ---------------------------------------------------------------------------------- ends of the ranges

def test_product_bias_past_2_to_the_29_columns():
    """A bias whose later columns lie 2^31 bytes and more from its first: every column gets its own.  No blocks of K, so that
    the weights take no memory; y = fma(1, 0, bias) is the bias itself."""
    N = 2 ** 29 + 133
    assert mxq.mxq_gemm_b128_plan(0, 2, N, 0, 1, 128, 1, 256) == (64, 64, 0)
    bias = torch.randn(N, device=DEV)
    x, w = (torch.empty((n, 0), dtype=torch.uint8, device=DEV) for n in (2, N))
    y = mxq.gemm_b128(x, torch.empty((2, 0), device=DEV), w, torch.empty((ref.blocks(N), 0), device=DEV), 0, bias=bias,
                      out_dtype=F32)
    for m in range(2):
        assert torch.equal(y[m], bias)


def guarded(shape, dtype, ld=None):
    """A view [rows][cols] at pitch ld inside a buffer of its own, 4 KiB before it and behind it, and a check that all but the view
    is as it was."""
    rows, cols = shape
    ld = ld or cols
    es = torch.empty((), dtype=dtype).element_size()
    pad = 4096 // es
    buf = torch.full((2 * pad + rows * ld,), 0x5A, dtype=torch.uint8, device=DEV) if dtype is torch.uint8 else \
        torch.full((2 * pad + rows * ld,), 5.0, dtype=dtype, device=DEV)
    view = buf[pad:pad + rows * ld].view(rows, ld)[:, :cols]

    def untouched():
        rest = buf.clone()
        fill = buf[0].item()
        rest[pad:pad + rows * ld].view(rows, ld)[:, :cols] = fill
        return bool((rest == fill).all())
    return view, untouched


def wrong_offsets(E, R, seed):
    """Offsets out of order, before the first row and past the last one."""
    g = torch.Generator().manual_seed(seed)
    o = torch.randint(-R, 3 * R, (E + 1,), generator=g)
    o[::3] = torch.randint(0, R + 1, (len(o[::3]),), generator=g)
    return o.int().to(DEV)


@pytest.mark.parametrize("E", [1, 5, 64, 100])
def test_quantize_by_wrong_offsets_stays_inside(E):
    R, C = 700, 300
    x = wide(R, C, BF16, 3).to(DEV)
    nbr = (R + 127 * E) // 128
    for seed in range(3):
        off = wrong_offsets(E, R, seed)
        rc, rc_ok = guarded((R, 384), torch.uint8, 400)
        rs, rs_ok = guarded((3, R), F32, R + 5)
        cc, cc_ok = guarded((C, 128 * nbr), torch.uint8, 128 * nbr + 16)
        cs, cs_ok = guarded((nbr, C), F32, C + 3)
        stream = torch.cuda.current_stream().cuda_stream
        for row in (True, False):
            assert mxq.mxq_quantize_b128(
                x.data_ptr(), mxq.MXQ_BF16, R, C, C, mxq.MXQ_E4M3, mxq.MXQ_SCALE_AMAX, 0, rc.data_ptr() if row else None, 400,
                rs.data_ptr() if row else None, R + 5, cc.data_ptr(), 128 * nbr + 16, cs.data_ptr(), C + 3, off.data_ptr(), E,
                stream) == 0
        assert rc_ok() and rs_ok() and cc_ok() and cs_ok()


# plan, experts, rows, columns, K: the search for up to and for more than 64 experts, and every kernel
WRONG_ROWS = [((16, 64, 1), 100, 250, 200, 300), ((64, 64, 0), 100, 700, 200, 300), ((64, 64, 0), 6, 511, 900, 384),
              ((128, 128, 0), 4, 2011, 4100, 640), ((256, 256, 0), 3, 3811, 3000, 1280)]


@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("tile,E,R,N,K", WRONG_ROWS)
def test_experts_of_wrong_offsets_stay_inside(tile, E, R, N, K, accum):
    assert mxq.mxq_gemm_b128_plan(1, R, N, K, E, 1, 0 if accum == "fp8" else 1, 256) == tile
    xc, xs = mxq.quantize_b128(wide(R, K, BF16, 1).to(DEV))
    wc, ws = mxq.quantize_b128(wide(E * N, K, BF16, 2).to(DEV))
    wc, ws = wc.view(E, N, -1), ws.t().contiguous().view(-1, E, N).permute(1, 2, 0)
    for seed in range(3):
        y, y_ok = guarded((R, N), F32, N + 5)
        mxq.moe_gemm_b128(xc, xs, wc, ws, wrong_offsets(E, R, seed), K, out=y, accum=accum)
        assert y_ok()


WRONG_GRADS = [((64, 64, 0), 4, 470, 512, 500), ((64, 64, 0), 100, 700, 100, 90), ((128, 128, 0), 10, 166, 1999, 2003),
               ((256, 256, 0), 4, 15000, 8001, 2041)]


@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("tile,E,R,N,K", WRONG_GRADS)
def test_gradients_of_wrong_offsets_stay_inside(tile, E, R, N, K, accum):
    nb = (R + 127 * E) // 128
    assert mxq.mxq_gemm_b128_plan(2, N, K, 128 * nb + 127 - 127 * E, E, 1, 0 if accum == "fp8" else 1, 256) == tile
    codes = [torch.randint(0, 120, (n, 128 * nb), dtype=torch.uint8, device=DEV) for n in (N, K)]
    scales = [torch.ones((nb, n), device=DEV).t() for n in (N, K)]
    for seed in range(3):
        whole = torch.full((E + 2, N + 1, K + 3), 5.0, device=DEV)
        mxq.moe_wgrad_b128(codes[0], scales[0], codes[1], scales[1], wrong_offsets(E, R, seed), x_elem="e4m3",
                           out=whole[1:E + 1, :N, :K], accum=accum)
        for rest in (whole[0], whole[E + 1], whole[:, N], whole[:, :, K:]):
            assert bool((rest == 5.0).all())


@pytest.mark.parametrize("accum", ["fp32", "fp8"])
@pytest.mark.parametrize("M,N", [(9, 40), (700, 900), (1900, 2100)])
def test_codes_past_k_of_another_producer(M, N, accum):
    """Finite codes of any value behind K change nothing where the other operand has zeros there."""
    K = 300
    xc, xs = mxq.quantize_b128(wide(M, K, BF16, 1).to(DEV))
    wc, ws = mxq.quantize_b128(wide(N, K, BF16, 2).to(DEV))
    want = mxq.gemm_b128(xc, xs, wc, ws, K, accum=accum, out_dtype=F32)
    for codes in (xc, wc):
        kept = codes.clone()
        codes[:, K:] = torch.randint(0, 127, (codes.shape[0], 384 - K), device=DEV).to(torch.uint8)
        assert torch.equal(mxq.gemm_b128(xc, xs, wc, ws, K, accum=accum, out_dtype=F32), want)
        codes.copy_(kept)
