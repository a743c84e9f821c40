"""The plans of the MXFP4 product and the expert layer (host logic, no device needed): what they refuse, the
choices that the kernels' comments explain, and that every plan names a kernel that there is."""
import ctypes
import itertools

import numpy as np
import pytest

import mxfp8_block_scaled_03_amd as mxq

FP4, B16, F32 = mxq.MXQ_E2M1, mxq.MXQ_BF16, mxq.MXQ_F32
SPLITS = {(64, 64, w) for w in (1, 2, 4, 8)} | {(32, 64, 4), (32, 64, 8), (32, 32, 4), (32, 32, 8), (32, 16, 8), (16, 32, 4),
                                                (16, 32, 8), (16, 16, 4), (16, 16, 8)}


def product(M, N, K, x=FP4, aligned=True, cus=256):
    return mxq.mxq_gemm_fp4_plan(M, N, K, x, aligned, cus)


def experts(T, H, I, E, k, y=B16, aligned=True, cus=256):
    return mxq.mxq_moe_fp4_plan(T, H, I, E, k, y, aligned, cus)


def test_refusals():
    def status(fn, n, *a, null=False):
        out = [ctypes.c_int() for _ in range(n)]
        return fn(*a, *(None if null else ctypes.byref(v) for v in out))
    g = lambda M=8, N=8, K=64, x=FP4, a=1, cus=256, **kw: status(mxq.lib().mxq_gemm_fp4_plan, 3, M, N, K, x, a, cus, **kw)  # noqa: E731
    assert g() == 0 and g(K=0) == 0
    assert g(null=True) == -1 and g(x=F32) == -5 and g(cus=0) == -6 and g(a=2) == -6
    assert g(M=0) == -2 and g(N=0) == -2 and g(K=-1) == -2 and g(M=1 << 31) == -2 and g(N=1 << 31) == -2 and g(K=1 << 24) == -2
    m = lambda T=2, H=80, I=40, E=4, k=2, y=B16, a=1, cus=256, **kw: status(  # noqa: E731
        mxq.lib().mxq_moe_fp4_plan, 4, T, H, I, E, k, y, a, cus, **kw)
    assert m() == 0
    assert m(null=True) == -1 and m(y=FP4) == -5 and m(k=0) == -6 and m(k=5) == -6 and m(cus=0) == -6 and m(a=-1) == -6
    assert m(T=0) == -2 and m(T=1025) == -2 and m(H=0) == -2 and m(I=0) == -2 and m(E=0) == -2 and m(E=1025) == -2
    assert m(H=1 << 24) == -2 and m(I=1 << 24) == -2
    with pytest.raises(mxq.MxqError):
        product(0, 1, 1)
    with pytest.raises(mxq.MxqError):
        experts(1, 1, 1, 1, 2)


def test_product_choices():
    assert product(8192, 4096, 4096) == (256, 256, 8) and product(8192, 4096, 4096, aligned=False) == (64, 64, 1)
    assert product(4096, 2048, 4096) == (256, 256, 8) and product(1000, 4096, 4096) == (64, 64, 2)
    assert product(1000, 1000, 4001) == (64, 64, 8) and product(2000, 1000, 3000) == (64, 64, 4)
    assert product(3000, 1500, 800) == (64, 32, 2) and product(3000, 1500, 800, B16) == (64, 64, 1)
    assert product(30, 32768, 4096, B16) == (32, 64, 4) and product(1, 65536, 4096, B16) == (16, 32, 8)
    assert product(300, 300, 7, B16) == (1, 4, 0) and product(300, 300, 8, B16) != (1, 4, 0)
    # the tile kernel's bias has 32-bit offsets
    assert product(1, (1 << 29) - 1, 64) == (256, 256, 8) and product(1, 1 << 29, 64) == (16, 32, 4)


def test_products_have_a_kernel():
    rng = np.random.default_rng(0)
    for _ in range(4000):
        M, N, K = (int(2 ** rng.uniform(0, b)) for b in (30.9, 30.9, 23.9))
        x, aligned, cus = int(rng.choice((FP4, B16))), bool(rng.integers(2)), int(rng.choice((1, 64, 256, 304)))
        p = product(M, N, K, x, aligned, cus)
        assert p in SPLITS or (x == FP4 and (p == (64, 32, 2) or (p == (256, 256, 8) and aligned))) or (x == B16 and K < 8 and p == (1, 4, 0)), \
            (M, N, K, x, aligned, cus, p)


def test_expert_choices():
    assert experts(1, 4096, 2048, 64, 4) == (2, 0, 0, 0)                   # one token: two launches
    assert experts(16, 5120, 8192, 8, 2) == (4, 128, 256, 8)               # large matrices: persistent workgroups
    assert experts(16, 5120, 8192, 8, 2, aligned=False) == (4, 64, 128, 1)
    assert experts(16, 5121, 8192, 8, 2)[1] == 64                          # rows of x that are no whole pieces
    assert experts(1, 64, 64, 257, 4)[0] == 4 and experts(1, 64, 64, 256, 4)[0] == 2


def test_expert_layers_have_kernels_and_room():
    """Plans name kernels that there are, and the workspace holds what they need: h in the fragment order and a
    row of y for each (token, rank, range)."""
    rng = np.random.default_rng(1)
    for _ in range(2000):
        T, E = int(rng.integers(1, 1025)), int(rng.integers(1, 1025))
        H, I, k = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 14)), int(rng.integers(1, min(E, 64) + 1))
        for y, aligned in itertools.product((B16, F32), (True, False)):
            launches, up, down, parts = experts(T, H, I, E, k, y, aligned)
            assert (launches == 2 and E <= 256 and up == down == parts == 0) or (
                launches == 4 and up in ((16, 32, 64, 128) if aligned and H % 8 == 0 else (16, 32, 64))
                and (down == 256 and aligned and parts in (1, 2, 4, 8) or down in ((32,) if y == F32 else (32, 64, 128)) and parts == 1))
    for T, H, I, E, k, y in ((16, 5120, 8192, 8, 2, B16), (16, 5120, 8192, 8, 2, F32), (300, 70, 700, 3, 2, B16)):
        parts, planes = experts(T, H, I, E, k, y)[3], 2 if y == B16 else 3
        h = E * -(-T // 16) * 16 * -(-I // 512) * 512 * 2 * planes
        need = mxq.mxq_moe_fp4_workspace(T, H, I, E, k, y)
        assert h + 4 * T * k * parts * H <= need <= h + 4 * T * k * (parts * H + 2) + 2 * E * T + 4 * 256
