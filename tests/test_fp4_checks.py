"""CPU tests of the MXFP4 entry points' argument checks: the C ABI rejects on the host before
any HIP call, the torch functions before any call at all."""
import pytest
import torch

import mxfp8_block_scaled_03_amd as mxq

# A 64 KiB-aligned non-null address: every call below fails validation or is an empty problem,
# so nothing is ever enqueued with it -- never add a case that passes.
FAKE = 0x10000


def q(fn=None, **kw):
    a = dict(src=FAKE, src_type=mxq.MXQ_BF16, rows=4, cols=80, ld_src=80, axis=mxq.MXQ_ROWWISE, opt=0, codes=FAKE,
             ld_codes=48, scales=FAKE, ld_scales=3)
    a.update(kw)
    return (fn or mxq.mxq_quantize_fp4)(a["src"], a["src_type"], a["rows"], a["cols"], a["ld_src"], a["axis"], a["opt"],
                                        a["codes"], a["ld_codes"], a["scales"], a["ld_scales"], None)


@pytest.mark.parametrize("fn", [mxq.mxq_quantize_fp4, mxq.mxq_quantize_fp4_sr])
def test_quantize(fn):
    assert q(fn, src_type=mxq.MXQ_E2M1) == -5
    assert q(fn, axis=2) == -6
    assert q(fn, rows=-1) == -2
    assert q(fn, cols=1 << 31) == -2
    assert q(fn, src=None) == -1 and q(fn, codes=None) == -1 and q(fn, scales=None) == -1
    assert q(fn, ld_src=79) == -3
    assert q(fn, ld_codes=32) == -3                   # 3 blocks need 48 bytes
    assert q(fn, ld_scales=2) == -3
    assert q(fn, ld_codes=56) == -4
    assert q(fn, codes=FAKE + 8) == -4
    assert q(fn, src=FAKE + 1) == -4
    assert q(fn, axis=mxq.MXQ_COLWISE, rows=40, ld_codes=16) == -3
    assert q(fn, ld_src=(1 << 62)) == -2
    assert q(fn, rows=0, src=None, codes=None, scales=None) == 0
    assert q(fn, cols=0, src=None, codes=None, scales=None) == 0


def test_quantize_rule():
    assert q(opt=2) == -6 and q(opt=-1) == -6


def test_quantize_dual():
    def d(**kw):
        a = dict(src=FAKE, t=mxq.MXQ_F32, rows=40, cols=80, ld=80, rc=FAKE, ld_rc=48, rs=FAKE, ld_rs=3, cc=FAKE,
                 ld_cc=32, cs=FAKE, ld_cs=2)
        a.update(kw)
        return mxq.mxq_quantize_fp4_dual(a["src"], a["t"], a["rows"], a["cols"], a["ld"], a["rc"], a["ld_rc"], a["rs"],
                                         a["ld_rs"], a["cc"], a["ld_cc"], a["cs"], a["ld_cs"], None)
    assert d(t=mxq.MXQ_E4M3) == -5
    assert d(rows=-1) == -2
    for name in ("src", "rc", "rs", "cc", "cs"):
        assert d(**{name: None}) == -1
    assert d(ld=79) == -3 and d(ld_rc=32) == -3 and d(ld_rs=2) == -3 and d(ld_cc=16) == -3 and d(ld_cs=1) == -3
    assert d(ld_rc=56) == -4 and d(ld_cc=40) == -4 and d(rc=FAKE + 8) == -4 and d(cc=FAKE + 4) == -4
    assert d(src=FAKE + 2) == -4
    assert d(rows=0, src=None, rc=None) == 0


def test_dequantize():
    def d(**kw):
        a = dict(c=FAKE, ld=48, s=FAKE, ld_s=3, L=4, K=70, dst=FAKE, t=mxq.MXQ_BF16, ld_dst=70)
        a.update(kw)
        return mxq.mxq_dequantize_fp4(a["c"], a["ld"], a["s"], a["ld_s"], a["L"], a["K"], a["dst"], a["t"], a["ld_dst"],
                                      None)
    assert d(t=mxq.MXQ_E2M1) == -5
    assert d(L=-1) == -2
    assert d(c=None) == -1 and d(s=None) == -1 and d(dst=None) == -1
    assert d(ld=32) == -3 and d(ld_s=2) == -3 and d(ld_dst=69) == -3
    assert d(ld=56) == -4 and d(c=FAKE + 4) == -4 and d(dst=FAKE + 1) == -4
    assert d(K=0, c=None) == 0


def test_gemm():
    def g(**kw):
        a = dict(M=8, N=8, K=80, x=FAKE, xt=mxq.MXQ_BF16, ld_x=80, xs=None, ld_xs=0, w=FAKE, ld_w=48, ws=FAKE, ld_ws=3,
                 alpha=1.0, bias=None, act=0, y=FAKE, yt=mxq.MXQ_F32, ld_y=8)
        a.update(kw)
        return mxq.mxq_gemm_fp4(a["M"], a["N"], a["K"], a["x"], a["xt"], a["ld_x"], a["xs"], a["ld_xs"], a["w"],
                                a["ld_w"], a["ws"], a["ld_ws"], a["alpha"], a["bias"], a["act"], a["y"], a["yt"],
                                a["ld_y"], None)
    fp4 = dict(xt=mxq.MXQ_E2M1, ld_x=48, xs=FAKE, ld_xs=3)
    assert g(xt=mxq.MXQ_F32) == -5 and g(xt=mxq.MXQ_E4M3) == -5 and g(yt=mxq.MXQ_E2M1) == -5
    assert g(act=2) == -6 and g(alpha=float("nan")) == -6 and g(alpha=float("inf")) == -6
    assert g(M=-1) == -2 and g(K=1 << 24) == -2 and g(N=1 << 31) == -2
    assert g(x=None) == -1 and g(w=None) == -1 and g(ws=None) == -1 and g(y=None) == -1
    assert g(**{**fp4, "xs": None}) == -1
    assert g(ld_x=79) == -3 and g(ld_w=32) == -3 and g(ld_ws=2) == -3 and g(ld_y=7) == -3
    assert g(ld_w=1 << 24) == -3 and g(ld_ws=1 << 24) == -3
    assert g(**{**fp4, "ld_x": 32}) == -3 and g(**{**fp4, "ld_xs": 2}) == -3
    assert g(w=FAKE + 8) == -4 and g(ld_w=56) == -4 and g(x=FAKE + 1) == -4 and g(y=FAKE + 2) == -4
    assert g(**{**fp4, "x": FAKE + 2}) == -4 and g(**{**fp4, "ld_x": 56}) == -4 and g(bias=FAKE + 2) == -4
    assert g(M=0, x=None, y=None) == 0 and g(N=0, w=None) == 0


def test_moe():
    def m(**kw):
        a = dict(T=2, H=80, I=40, E=4, k=2, rn=1, x=FAKE, ld_x=80, lg=FAKE, ld_lg=4, w13=FAKE, l13=48, e13=48 * 80,
                 s13=FAKE, ls13=3, es13=240, w2=FAKE, l2=32, e2=32 * 80, s2=FAKE, ls2=2, es2=160, y=FAKE,
                 yt=mxq.MXQ_BF16, ld_y=80, ws=FAKE, n=1 << 30)
        a.update(kw)
        return mxq.mxq_moe_fp4(a["T"], a["H"], a["I"], a["E"], a["k"], a["rn"], a["x"], a["ld_x"], a["lg"], a["ld_lg"],
                               a["w13"], a["l13"], a["e13"], a["s13"], a["ls13"], a["es13"], a["w2"], a["l2"], a["e2"],
                               a["s2"], a["ls2"], a["es2"], a["y"], a["yt"], a["ld_y"], a["ws"], a["n"], None)
    assert m(T=-1) == -2 and m(T=1025) == -2 and m(E=0) == -2 and m(E=1025) == -2 and m(I=-1) == -2 and m(I=0) == -2
    assert m(k=0) == -6 and m(k=5) == -6 and m(rn=2) == -6
    assert m(yt=mxq.MXQ_E4M3) == -5
    for name in ("x", "lg", "w13", "s13", "w2", "s2", "y", "ws"):
        assert m(**{name: None}) == -1, name
    assert m(ld_x=79) == -3 and m(ld_lg=3) == -3 and m(ld_y=79) == -3
    assert m(l13=32) == -3 and m(ls13=2) == -3 and m(l2=16) == -3 and m(ls2=1) == -3
    assert m(e13=48 * 79) == -3 and m(es13=100) == -3 and m(e2=32) == -3 and m(es2=2) == -3
    assert m(w13=FAKE + 8) == -4 and m(l13=56) == -4 and m(e13=48 * 80 + 8) == -4 and m(w2=FAKE + 4) == -4
    assert m(x=FAKE + 1) == -4 and m(lg=FAKE + 2) == -4 and m(y=FAKE + 1) == -4 and m(ws=FAKE + 128) == -4
    assert m(I=1 << 20, l13=1 << 13, l2=1 << 20, ls2=1 << 16, e13=1 << 50, e2=1 << 50, es13=1 << 50, es2=1 << 50) == -2
    assert m(n=mxq.mxq_moe_fp4_workspace(2, 80, 40, 4, 2, mxq.MXQ_BF16) - 1) == -8
    assert m(T=0, x=None, y=None) == 0 and m(H=0, x=None) == 0


def test_moe_workspace():
    small = mxq.mxq_moe_fp4_workspace(1, 4096, 2048, 64, 4, mxq.MXQ_BF16)
    assert 0 < small < mxq.mxq_moe_fp4_workspace(64, 4096, 2048, 64, 8, mxq.MXQ_BF16)
    assert 0 < mxq.mxq_moe_fp4_workspace(1, 4096, 2048, 64, 4, mxq.MXQ_F32)
    assert mxq.mxq_moe_fp4_workspace(0, 4096, 2048, 64, 4, mxq.MXQ_BF16) == 0
    with pytest.raises(mxq.MxqError):
        mxq.mxq_moe_fp4_workspace(1, 4096, 2048, 64, 65, mxq.MXQ_BF16)


# ---------------------------------------------------------------- the torch functions

U8 = torch.uint8


def z(*shape, dtype=U8):
    return torch.zeros(shape, dtype=dtype)


def refuses(fn, *a, match, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


@pytest.mark.parametrize("fn", [mxq.quantize_fp4, lambda x, **kw: mxq.quantize_fp4_sr(x, 1, **kw)])
def test_quantize_function(fn):
    x = z(4, 80, dtype=torch.float32)
    refuses(fn, x.double(), match="float32 or bfloat16")
    refuses(fn, x[0], match="2-D")
    refuses(fn, x.T, match="unit stride")
    refuses(fn, x, axis="diag", match="axis")
    refuses(fn, x, codes=z(4, 47), match="columns")
    refuses(fn, x, codes=z(3, 48), match="rows")
    refuses(fn, x, codes=z(4, 48, dtype=torch.int8), match="uint8")
    refuses(fn, x, scales=z(4, 2), match="columns")
    refuses(fn, x, match="CUDA")


def test_other_functions():
    x = z(4, 80, dtype=torch.float32)
    refuses(mxq.quantize_fp4, x, rule="floor", match="rule")
    refuses(mxq.quantize_fp4_dual, x.int(), match="float32 or bfloat16")
    refuses(mxq.quantize_fp4_dual, x, match="CUDA")
    c, s = z(4, 48), z(4, 3)
    refuses(mxq.dequantize_fp4, c, s, 70, out_dtype=torch.float16, match="out_dtype")
    refuses(mxq.dequantize_fp4, c, s, -1, match="K must")
    refuses(mxq.dequantize_fp4, c, s, 97, match="codes")
    refuses(mxq.dequantize_fp4, c, s[:, :2], 70, match="scales")
    refuses(mxq.dequantize_fp4, c, s, 70, match="CUDA")


def test_one_row_with_steps():
    """A single row whose elements are not neighbours."""
    x = z(1, 160, dtype=torch.bfloat16)[:, ::2]
    refuses(mxq.quantize_fp4, x, match="unit stride")
    refuses(mxq.gemm_fp4, x, None, z(8, 48), z(8, 3), 80, match="unit stride")
    refuses(mxq.dequantize_fp4, z(1, 96)[:, ::2], z(1, 3), 70, match="unit stride")
    refuses(mxq.moe_fp4, x, z(1, 4, dtype=torch.float32), z(4, 80, 48), z(4, 80, 3), z(4, 80, 32), z(4, 80, 2), 2,
            match="unit stride")


def test_gemm_function():
    w, ws, xc, xs, xb = z(8, 48), z(8, 3), z(4, 48), z(4, 3), z(4, 80, dtype=torch.bfloat16)
    g = mxq.gemm_fp4
    refuses(g, xb, None, w, ws, -1, match="K must")
    refuses(g, xb, None, w[:, :32], ws, 80, match="w_codes")
    refuses(g, xb, None, w, ws[:, :2], 80, match="w_scales")
    refuses(g, xb[:, :79], None, w, ws, 80, match="columns")
    refuses(g, xb.float(), None, w, ws, 80, match="bfloat16")
    refuses(g, xb, xs, w, ws, 80, match="uint8")
    refuses(g, xc[:, :32], xs, w, ws, 80, match="x has")
    refuses(g, xc, xs[:3], w, ws, 80, match="x_scales")
    refuses(g, xc, xs, w, ws, 80, bias=z(7, dtype=torch.float32), match="bias")
    refuses(g, xc, xs, w, ws, 80, bias=z(16, dtype=torch.float32)[::2], match="bias")
    refuses(g, xc, xs, w, ws, 80, act="gelu", match="act")
    refuses(g, xc, xs, w, ws, 80, out_dtype=torch.float16, match="out_dtype")
    refuses(g, xc, xs, w, ws, 80, out=z(4, 7, dtype=torch.float32), match="out must")
    refuses(g, xc, xs, w, ws, 80, match="CUDA")


def test_moe_function():
    x, lg = z(2, 80, dtype=torch.bfloat16), z(2, 4, dtype=torch.float32)
    w13, s13, w2, s2 = z(4, 80, 48), z(4, 80, 3), z(4, 80, 32), z(4, 80, 2)
    f = mxq.moe_fp4
    refuses(f, x.float(), lg, w13, s13, w2, s2, 2, match="bfloat16")
    refuses(f, x, lg.double(), w13, s13, w2, s2, 2, match="float32")
    refuses(f, x, lg[:1], w13, s13, w2, s2, 2, match="logits")
    refuses(f, x, lg, w13[:, :79], s13, w2, s2, 2, match="even")
    refuses(f, x, lg, w13, s13, w2, s2, 0, match="k must")
    refuses(f, x, lg, w13, s13, w2, s2, 5, match="k must")
    refuses(f, x, lg, w13[:3], s13, w2, s2, 2, match="w13_codes")
    refuses(f, x, lg, w13[..., :32], s13, w2, s2, 2, match="w13_codes")
    refuses(f, x, lg, w13, s13[..., :2], w2, s2, 2, match="w13_scales")
    refuses(f, x, lg, w13, s13, w2[:, :79], s2, 2, match="w2_codes")
    refuses(f, x, lg, w13, s13, w2, s2[..., :1], 2, match="w2_scales")
    refuses(f, x, lg, w13, s13, w2.transpose(0, 1).contiguous().transpose(0, 1)[..., ::2], s2, 2, match="w2_codes")
    refuses(f, x, lg, w13, s13, w2, s2, 2, out=z(2, 79, dtype=torch.float32), match="out must")
    refuses(f, x, lg, w13, s13, w2, s2, 2, out_dtype=torch.float16, match="out_dtype")
    refuses(f, x, lg, w13, s13, w2, s2, 2, match="CUDA")
