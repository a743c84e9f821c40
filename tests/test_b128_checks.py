"""Refusals of the entry points for blocks of 128 and for routing, in C and in Python, and the plans of the
product: host logic only."""
import pytest
import torch

import mxfp8_block_scaled_03_amd as mxq

# A 64 KiB-aligned non-null address.  Every call below must fail validation (or be an empty problem), so nothing is
# ever enqueued with it -- never add a case that passes.
FAKE = 0x10000
OK, NULL, SHAPE, LD, ALIGN, DTYPE, ARG, SCRATCH = 0, -1, -2, -3, -4, -5, -6, -8


def call(fn, order, base, kw):
    a = dict(base)
    unknown = set(kw) - set(a)
    assert not unknown, unknown
    a.update(kw)
    return fn(*[a[n] for n in order.split()], None)


def q(**kw):
    return call(mxq.mxq_quantize_b128, "src src_type rows cols ld_src elem rule tile rc ld_rc rs ld_rs cc ld_cc cs ld_cs offsets experts",
                dict(src=FAKE, src_type=mxq.MXQ_BF16, rows=200, cols=300, ld_src=300, elem=mxq.MXQ_E4M3,
                     rule=mxq.MXQ_SCALE_AMAX, tile=0, rc=FAKE, ld_rc=384, rs=FAKE, ld_rs=200, cc=FAKE, ld_cc=256, cs=FAKE,
                     ld_cs=300, offsets=None, experts=0), kw)


@pytest.mark.parametrize("kw,want", [
    (dict(src_type=mxq.MXQ_E4M3), DTYPE), (dict(elem=mxq.MXQ_E2M1), DTYPE), (dict(rule=mxq.MXQ_SCALE_OCP), ARG),
    (dict(tile=2), ARG), (dict(rows=-1), SHAPE), (dict(cols=2 ** 30, ld_src=2 ** 30), SHAPE), (dict(src=None), NULL),
    (dict(rc=None, cc=None), NULL), (dict(rs=None), NULL), (dict(cs=None), NULL), (dict(tile=1, rc=None), NULL),
    (dict(ld_src=299), LD), (dict(ld_rc=383), LD), (dict(ld_rs=199), LD), (dict(ld_cc=255), LD), (dict(ld_cs=299), LD),
    (dict(rc=FAKE + 8), ALIGN), (dict(ld_rc=392), ALIGN), (dict(cc=FAKE + 1), ALIGN), (dict(rs=FAKE + 2), ALIGN),
    (dict(src=FAKE + 1), ALIGN), (dict(tile=1, ld_rs=2), LD),
    (dict(tile=1, offsets=FAKE, experts=3), ARG), (dict(offsets=FAKE, experts=0), SHAPE),
    (dict(offsets=FAKE, experts=1025), SHAPE), (dict(offsets=FAKE, experts=3, cc=None), ARG),
    (dict(offsets=FAKE, experts=3), LD),                       # 200 rows of 3 experts take up to 4 blocks, not 2
    (dict(offsets=FAKE + 2, experts=3, ld_cc=512), ALIGN),
    (dict(rows=2 ** 29, cols=2 ** 29, ld_src=2 ** 29, ld_rc=2 ** 29, ld_rs=2 ** 29, ld_cc=2 ** 29, ld_cs=2 ** 29), SHAPE),
    (dict(rows=0, rc=FAKE), OK), (dict(cols=0), OK)])
def test_quantize_validation(kw, want):
    assert q(**kw) == want


def g(**kw):
    return call(mxq.mxq_gemm_b128, "M N K x ld_x xs ld_xs x_elem w ld_w ws ws_line ws_block w_block w_elem alpha bias act accum y y_type ld_y",
                dict(M=100, N=200, K=300, x=FAKE, ld_x=384, xs=FAKE, ld_xs=100, x_elem=mxq.MXQ_E4M3, w=FAKE, ld_w=384, ws=FAKE,
                     ws_line=3, ws_block=1, w_block=128, w_elem=mxq.MXQ_E4M3, alpha=1.0, bias=None, act=0, accum=1, y=FAKE,
                     y_type=mxq.MXQ_BF16, ld_y=200), kw)


PRODUCT = [
    (dict(x_elem=mxq.MXQ_BF16), DTYPE), (dict(w_elem=mxq.MXQ_E2M1), DTYPE), (dict(y_type=mxq.MXQ_E4M3), DTYPE),
    (dict(accum=2), ARG), (dict(w_block=32), ARG),
    (dict(K=-1), SHAPE), (dict(N=2 ** 30), SHAPE), (dict(K=2 ** 24), SHAPE), (dict(x=None), NULL),
    (dict(xs=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL), (dict(ld_x=383), LD),
    (dict(ld_x=2 ** 24), LD), (dict(ld_w=2 ** 24), LD), (dict(ld_w=256), LD), (dict(ld_xs=99), LD), (dict(ld_y=199), LD),
    (dict(ws_line=-1), LD), (dict(w_block=1), LD), (dict(w_block=1, ws_line=1, ws_block=199), LD), (dict(x=FAKE + 4), ALIGN),
    (dict(ld_w=392), ALIGN), (dict(ws=FAKE + 1), ALIGN), (dict(y=FAKE + 1), ALIGN), (dict(xs=FAKE + 3), ALIGN),
    (dict(ld_xs=2 ** 28), SHAPE), (dict(ws_block=2 ** 28), SHAPE)]


@pytest.mark.parametrize("kw,want", PRODUCT + [
    (dict(M=2 ** 30), SHAPE), (dict(act=2), ARG), (dict(alpha=float("inf")), ARG), (dict(bias=FAKE + 2), ALIGN),
    (dict(M=2 ** 29, N=2 ** 29, K=1, ld_xs=2 ** 29, ld_y=2 ** 29), SHAPE), (dict(M=0), OK), (dict(N=0), OK)])
def test_gemm_validation(kw, want):
    assert g(**kw) == want


@pytest.mark.parametrize("kw,want", PRODUCT + [
    (dict(rows=2 ** 30), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(offsets=None), NULL), (dict(offsets=FAKE + 1), ALIGN),
    (dict(expert_w=-16), LD), (dict(expert_ws=-1), LD), (dict(expert_w=24), ALIGN), (dict(expert_w=2 ** 62), SHAPE),
    (dict(rows=0), OK), (dict(N=0), OK)])
def test_moe_gemm_validation(kw, want):
    got = call(mxq.mxq_moe_gemm_b128, "rows N K E offsets x ld_x xs ld_xs x_elem w ld_w expert_w ws ws_line ws_block expert_ws w_block w_elem accum y y_type ld_y",
               dict(rows=100, N=200, K=300, E=4, offsets=FAKE, x=FAKE, ld_x=384, xs=FAKE, ld_xs=100, x_elem=mxq.MXQ_E4M3, w=FAKE,
                    ld_w=384, expert_w=76800, ws=FAKE, ws_line=3, ws_block=1, expert_ws=6, w_block=128, w_elem=mxq.MXQ_E4M3,
                    accum=1, y=FAKE, y_type=mxq.MXQ_BF16, ld_y=200), kw)
    assert got == want


@pytest.mark.parametrize("kw,want", [
    (dict(M=2 ** 30), SHAPE), (dict(rows=2 ** 24), SHAPE), (dict(E=0), SHAPE), (dict(offsets=None), NULL), (dict(x=None), NULL),
    (dict(ld_x=640), LD), (dict(ld_w=640), LD), (dict(ld_xs=99), LD), (dict(ld_ws=199), LD), (dict(ld_y=199), LD),
    (dict(expert_y=19999), LD), (dict(expert_y=2 ** 62), SHAPE), (dict(y_type=mxq.MXQ_E5M2), DTYPE), (dict(accum=-1), ARG),
    (dict(y=FAKE + 2), ALIGN), (dict(M=0), OK)])
def test_moe_wgrad_validation(kw, want):
    # 300 rows of 4 experts: up to (300 + 4 * 127) // 128 = 6 blocks
    got = call(mxq.mxq_moe_wgrad_b128, "M N rows E offsets x ld_x xs ld_xs x_elem w ld_w ws ld_ws w_elem accum y y_type ld_y expert_y",
               dict(M=100, N=200, rows=300, E=4, offsets=FAKE, x=FAKE, ld_x=768, xs=FAKE, ld_xs=100, x_elem=mxq.MXQ_E5M2, w=FAKE,
                    ld_w=768, ws=FAKE, ld_ws=200, w_elem=mxq.MXQ_E4M3, accum=1, y=FAKE, y_type=mxq.MXQ_F32, ld_y=200,
                    expert_y=20000), kw)
    assert got == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(E=1025), SHAPE), (dict(E=0), SHAPE), (dict(k=0), ARG), (dict(k=9), ARG), (dict(E=100, k=65, ld=100), ARG),
    (dict(T=2 ** 29, k=2), SHAPE), (dict(type=mxq.MXQ_E4M3), DTYPE), (dict(renorm=2), ARG), (dict(logits=None), NULL),
    (dict(experts=None), NULL), (dict(counts=None), NULL), (dict(loss=None), NULL), (dict(workspace=None), NULL), (dict(ld=7), LD),
    (dict(logits=FAKE + 2), ALIGN), (dict(order=FAKE + 1), ALIGN), (dict(workspace=FAKE + 128), ALIGN), (dict(bytes=64), SCRATCH)])
def test_route_validation(kw, want):
    T, E, k = kw.get("T", 1000), kw.get("E", 8), kw.get("k", 2)
    got = call(mxq.mxq_moe_route, "T E k renorm logits type ld mask experts shares counts offsets order loss slope workspace bytes",
               dict(T=T, E=E, k=k, renorm=1, logits=FAKE, type=mxq.MXQ_F32, ld=8, mask=None, experts=FAKE, shares=FAKE,
                    counts=FAKE, offsets=FAKE, order=FAKE, loss=FAKE, slope=FAKE, workspace=FAKE, bytes=2 ** 40), kw)
    assert got == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(k=0), ARG), (dict(type=mxq.MXQ_E4M3), DTYPE), (dict(renorm=-1), ARG), (dict(logits=None), NULL),
    (dict(d=None), NULL), (dict(experts=None), NULL), (dict(slope=None), NULL), (dict(ld=7), LD), (dict(ld_d=7), LD),
    (dict(ld_ds=1), LD), (dict(d=FAKE + 2), ALIGN), (dict(d_loss=FAKE + 1), ALIGN), (dict(T=0), OK)])
def test_route_grad_validation(kw, want):
    got = call(mxq.mxq_moe_route_grad, "T E k renorm logits type ld mask experts shares slope d_shares ld_ds d_loss d ld_d",
               dict(T=1000, E=8, k=2, renorm=1, logits=FAKE, type=mxq.MXQ_F32, ld=8, mask=None, experts=FAKE, shares=FAKE,
                    slope=FAKE, d_shares=FAKE, ld_ds=2, d_loss=FAKE, d=FAKE, ld_d=8), kw)
    assert got == want


def test_route_workspace():
    assert mxq.mxq_moe_route_workspace(64, 64, 8) == 0            # one workgroup
    assert mxq.mxq_moe_route_workspace(0, 8, 2) == 0
    assert mxq.mxq_moe_route_workspace(257, 8, 2) > 0
    assert mxq.mxq_moe_route_workspace(10, 300, 2) > 0
    for bad in ((10, 8, 9), (10, 0, 1), (-1, 8, 2)):
        with pytest.raises(mxq.MxqError):
            mxq.mxq_moe_route_workspace(*bad)


# ------------------------------------------------------------------------------------- plans

def plan(mode, M, N, K, E=1, block=128, accum=1, cus=256):
    return mxq.mxq_gemm_b128_plan(mode, M, N, K, E, block, accum, cus)


@pytest.mark.parametrize("mode,M,N,K,E,block,accum,want", [
    (0, 16, 4096, 4096, 1, 128, 0, (16, 16, 8)), (0, 32, 4096, 4096, 1, 128, 0, (32, 16, 8)),
    (0, 128, 4096, 4096, 1, 128, 1, (64, 32, 8)), (0, 512, 4096, 4096, 1, 128, 0, (64, 64, 0)),
    (0, 2048, 4096, 4096, 1, 128, 1, (128, 128, 0)), (0, 8192, 4096, 4096, 1, 128, 0, (256, 256, 0)),
    (0, 4096, 4096, 4096, 1, 1, 1, (256, 256, 0)), (1, 128, 4096, 2048, 64, 128, 0, (16, 64, 1)),
    (1, 512, 4096, 2048, 64, 128, 0, (64, 64, 0)), (1, 8192, 4096, 2048, 64, 128, 0, (128, 128, 0)),
    (1, 512, 8192, 5120, 8, 128, 0, (256, 256, 0)), (2, 4096, 2048, 8192, 16, 1, 1, (128, 128, 0))])
def test_plans(mode, M, N, K, E, block, accum, want):
    assert plan(mode, M, N, K, E, block, accum) == want


def test_plans_are_kernels_that_there_are():
    there = {(16, 16, 8), (32, 16, 8), (64, 32, 8), (16, 64, 1), (64, 64, 0), (128, 128, 0), (256, 256, 0)}
    got = set()
    sizes = (1, 3, 17, 64, 100, 300, 1000, 5000, 100000, 2 ** 20)
    for mode in (0, 1, 2):
        for M in sizes:
            for N in sizes:
                for K in (0, 1, 200, 5000, 2 ** 20):
                    for accum in (0, 1):
                        p = plan(mode, M, N, K, 7 if mode else 1, 1 if mode == 2 else 128, accum)
                        assert p in there and (p[2] != 1 or mode == 1)
                        got.add(p)
    assert got == there


def test_plan_validation():
    for bad in ((3, 1, 1, 1, 1, 128, 1, 256), (0, 0, 1, 1, 1, 128, 1, 256), (0, 1, 1, -1, 1, 128, 1, 256),
                (0, 1, 1, 1, 1, 64, 1, 256), (0, 1, 1, 1, 1, 128, 1, 0), (1, 1, 1, 1, 1025, 128, 1, 256)):
        with pytest.raises(mxq.MxqError):
            mxq.mxq_gemm_b128_plan(*bad)


# -------------------------------------------------------------------------- torch conveniences

def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def lines(n, nb):
    return torch.zeros((nb, n)).t()


@pytest.mark.parametrize("run,says", [
    (lambda: mxq.quantize_b128(torch.zeros(3, 4)), "CUDA"),
    (lambda: mxq.quantize_b128(torch.zeros(3, 4), "e3m4"), "e4m3"),
    (lambda: mxq.quantize_b128(torch.zeros(3, 4), axis="both"), "axis"),
    (lambda: mxq.quantize_b128(torch.zeros(3, 4), rule="ocp"), "rule"),
    (lambda: mxq.quantize_b128(torch.zeros(3, 4), offsets=torch.zeros(3, dtype=torch.int32)), "axis='col'"),
    (lambda: mxq.quantize_b128(torch.zeros(3, 4), axis="col", offsets=torch.zeros(3)), "offsets"),
    (lambda: mxq.quantize_b128(torch.zeros(3, 4).half()), "float32 or bfloat16"),
    (lambda: mxq.quantize_b128(torch.zeros(3, 4, 5)), "2-D"),
    (lambda: mxq.quantize_b128(torch.zeros(30, 4).t()), "stride"),
    (lambda: mxq.quantize_b128_dual(torch.zeros(3, 4), tile=True, offsets=torch.zeros(3, dtype=torch.int32)), "tiles"),
    (lambda: mxq.quantize_b128_dual(torch.zeros(3, 4)), "CUDA"),
    (lambda: mxq.gemm_b128(u8(5, 128), lines(5, 1), u8(7, 128), lines(7, 1), 100), "CUDA"),
    (lambda: mxq.gemm_b128(u8(5, 128), lines(5, 1), u8(7, 128), lines(7, 1), 200), "x_codes"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(4, 2), u8(7, 256), lines(7, 2), 200), "x_scales"),
    (lambda: mxq.gemm_b128(u8(5, 256), torch.zeros(5, 2), u8(7, 256), lines(7, 2), 200), "block by block"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(5, 2), u8(7, 256), torch.zeros(7, 2), 200), "block by block"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(5, 2), u8(300, 256), torch.zeros(2, 2), 200), "w_scales"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(5, 2).double(), u8(7, 256), lines(7, 2), 200), "float32"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(5, 2), u8(7, 256), lines(7, 2), 200, accum="tf32"), "accum"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(5, 2), u8(7, 256), lines(7, 2), 200, act="gelu"), "act"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(5, 2), u8(7, 256), lines(7, 2), 200, bias=torch.zeros(6)), "bias"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(5, 2), u8(7, 256), lines(7, 2), 200, x_elem="e2m1"), "formats"),
    (lambda: mxq.gemm_b128(u8(5, 256), lines(5, 2), u8(7, 256), lines(7, 2), -1), "K"),
    (lambda: mxq.moe_gemm_b128(u8(5, 128), lines(5, 1), u8(2, 7, 128), torch.zeros(2, 1, 1), torch.zeros(4, dtype=torch.int32), 9), "E = 3"),
    (lambda: mxq.moe_gemm_b128(u8(5, 128), lines(5, 1), u8(3, 7, 128), torch.zeros(2, 1, 1), torch.zeros(4, dtype=torch.int32), 9), "E = 3"),
    (lambda: mxq.moe_gemm_b128(u8(5, 128), lines(5, 1), u8(3, 7, 128), torch.zeros(3, 1, 1), torch.zeros(4), 9), "offsets"),
    (lambda: mxq.moe_gemm_b128(u8(5, 128), lines(5, 1), u8(3, 7, 128), torch.zeros(3, 1, 1), torch.zeros(4, dtype=torch.int32), 9), "CUDA"),
    (lambda: mxq.moe_wgrad_b128(u8(5, 128), lines(5, 1), u8(7, 128), lines(6, 1), torch.zeros(2, dtype=torch.int32)), "x_scales"),
    (lambda: mxq.moe_wgrad_b128(u8(5, 128), lines(5, 1), u8(7, 128), lines(7, 1), torch.zeros(2, dtype=torch.int32)), "CUDA"),
    (lambda: mxq.moe_route(torch.zeros(4, 8), 9), "k must"),
    (lambda: mxq.moe_route(torch.zeros(4, 8), 2, mask=torch.zeros(3, dtype=torch.bool)), "mask"),
    (lambda: mxq.moe_route(torch.zeros(4, 8), 2), "CUDA"),
    (lambda: mxq.moe_route(torch.zeros(4, 8).half(), 2), "float32 or bfloat16"),
])
def test_torch_refusals(run, says):
    with pytest.raises(ValueError, match=says):
        run()


def test_route_grad_refusals():
    i32, z = torch.int32, torch.zeros(4, 8)
    r = mxq.MoeRoute(torch.zeros((4, 2), dtype=i32), torch.zeros(4, 2), torch.zeros(8, dtype=i32), torch.zeros(9, dtype=i32),
                     torch.zeros(8, dtype=i32), torch.zeros(1), torch.zeros(8))
    with pytest.raises(ValueError, match="other sizes"):
        mxq.moe_route_grad(torch.zeros(5, 8), r)
    with pytest.raises(ValueError, match="d_shares"):
        mxq.moe_route_grad(z, r, d_shares=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="d_loss"):
        mxq.moe_route_grad(z, r, d_loss=torch.zeros(2))
    with pytest.raises(ValueError, match="contiguous"):
        mxq.moe_route_grad(z, r._replace(experts=torch.zeros((4, 2))))
    with pytest.raises(ValueError, match="CUDA"):
        mxq.moe_route_grad(z, r)
