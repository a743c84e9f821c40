"""CPU pins of the MXFP4 reference that the GPU tests compare with."""
from fractions import Fraction

import numpy as np
import pytest

import fp4_reference as ref
import oracle


def test_format_facts():
    codes = np.arange(16, dtype=np.uint8)
    c = np.zeros((1, 16), np.uint8)
    c[0, :8] = codes[0::2] | (codes[1::2] << 4)
    v = ref.values(c, np.array([[127]], np.uint8), 16)[0]
    assert v[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and v[8:].tolist() == [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
    assert np.signbit(v[8])
    assert np.isnan(ref.values(c, np.array([[255]], np.uint8), 16)).all()
    assert ref.values(c, np.array([[0]], np.uint8), 2)[0, 1] == 2.0 ** -128


@pytest.mark.parametrize("rule,amax,byte", [
    ("ceil", 6.0, 127), ("ceil", 6.0001, 128), ("ceil", 3.0, 126), ("ceil", 3.0001, 127), ("ceil", 1.0, 125),
    ("ceil", 2.0 ** -140, 0), ("ceil", 3.4e38, 253), ("ocp", 6.0, 127), ("ocp", 7.9, 127), ("ocp", 8.0, 128),
    ("ocp", 4.0, 127), ("ocp", 3.99, 126), ("ocp", 2.0 ** -149, 0), ("ceil", 0.0, 127), ("ocp", 0.0, 127)])
def test_scale_byte(rule, amax, byte):
    x = np.zeros((1, 32))
    x[0, 5] = -np.float64(np.float32(amax))
    assert ref.quantize(x, rule)[1][0, 0] == byte


def test_codes_round_to_the_nearest_even_neighbour():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 70)).astype(np.float32).astype(np.float64) * np.exp2(rng.integers(-30, 30, (40, 1)))
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    for rule in ("ceil", "ocp"):
        codes, scales = ref.quantize(x, rule)
        v = ref.values(codes, scales, 70)
        for l in range(40):
            for k in range(70):
                s = Fraction(2) ** (int(scales[l, k // 32]) - 127)
                a = min(abs(Fraction(float(x[l, k]))) / s, Fraction(6))
                best = min(range(8), key=lambda i: (abs(a - Fraction(float(ref.MAG[i]))), i % 2))
                assert abs(Fraction(float(v[l, k]))) == Fraction(float(ref.MAG[best])) * s
    assert ref.values(*ref.quantize(x[:1, :8], "ceil"), 8)[0].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]


def test_special_values():
    x = np.zeros((1, 96))
    x[0, 3], x[0, 40], x[0, 70] = -0.0, np.inf, np.nan
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127, 255, 255]]
    assert codes[0, 1] == 0x80 and (codes[0, 16:] == 0x77).all()


def test_philox_matches_the_oracle_and_rounding_is_unbiased():
    seed = 0x123456789ABCDEF0
    r = ref.philox24(64, seed)
    for c in range(16):
        w = oracle.philox4x32_10((c, 0, 0, 0), (seed & 0xFFFFFFFF, seed >> 32))
        assert [int(v) >> 8 for v in w] == r[4 * c:4 * c + 4].tolist()
    n = 1 << 16
    x = np.full((1, n), 2.2)
    x[0, ::32] = 6.0                                      # scale 1
    v = ref.values(*ref.quantize(x, seed=7), n)[0]
    v = v[np.arange(n) % 32 != 0]
    assert set(np.unique(v)) == {2.0, 3.0}
    p = (v == 3.0).mean()
    assert abs(p - 0.2) < 5 * np.sqrt(0.2 * 0.8 / len(v))


def test_product_and_experts_agree_with_plain_sums():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((3, 40)), rng.standard_normal((5, 40))
    y, b = ref.product(x, w, 2.0, np.arange(5.0), "silu")
    for i in range(3):
        for j in range(5):
            v = 2.0 * sum(x[i] * w[j]) + j
            assert abs(y[i, j] - v / (1 + np.exp(-v))) < 1e-12 and 0 < b[i, j] < 1e-2
    # one expert, share 1: a plain gated layer; a masked expert is not taken
    w13, w2 = rng.standard_normal((2, 12, 40)), rng.standard_normal((2, 40, 6))
    logits = np.array([[0.0, -np.inf]] * 3)
    y, b = ref.moe(x, logits, w13, w2, 2, True, False)
    g, u = x @ w13[0, :6].T, x @ w13[0, 6:].T
    assert np.allclose(y, (g / (1 + np.exp(-g)) * u) @ w2[0].T, rtol=0, atol=1e-12)
    assert (ref.moe(x, np.full((3, 2), -np.inf), w13, w2, 1, False, True)[0] == 0).all()
    assert ref.order(np.array([[1.0, 2.0, 2.0, 0.0]])).tolist() == [[1, 2, 0, 3]]
