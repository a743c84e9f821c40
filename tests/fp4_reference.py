"""MXFP4 in 64 bits, from the definition: quantize by search over the eight magnitudes,
decode by the bit fields, products and the mixture-of-experts layer in float64 with the
error bounds that the GPU tests assert.  numpy only; shares no code with the library.

Error bounds.  u = 2^-23 bounds a rounding to FP32 whether it rounds or truncates.
  product  every product of the operands is exact in FP32 (E2M1 x E2M1: 6 bits; bf16 x
           E2M1: 10 bits), so an output is off by at most one u of sum |x w| for each addition that a
           product passes through: at most 32 inside a matrix instruction, one for each
           instruction of K / 32, 8 for the waves: (K / 32 + 40) u T
  epilogue alpha and bias one fma: u |v|; SiLU: slope at most 1.1, 2^-20 relative for its own
           evaluation; rounding to bf16 half a step, 2^-8 relative
  experts  the bounds of the gate and up products carried through silu(g) * u * share, the
           split of h into 2 or 3 bf16 terms (2^-16 or 2^-24 relative), the down product, and
           the k additions of the sum
"""
import numpy as np

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U = 2.0 ** -23


def blocks(k):
    return (k + 31) // 32


def _scale_exponent(amax, rule):
    if rule == "ocp":
        return max(-127, int(np.frexp(amax)[1]) - 1 - 2)
    e = -127
    if amax > 6.0 * 2.0 ** -127:
        e = int(np.frexp(amax)[1]) - 5                      # certainly low enough
        while amax > 6.0 * 2.0 ** e:
            e += 1
    return max(-127, e)


def philox24(n, seed):
    """Top 24 bits of word i % 4 of Philox4x32-10(counter i / 4, key seed), i = 0 .. n-1."""
    c = (n + 3) // 4
    i = np.arange(c, dtype=np.uint64)
    lo32 = np.uint64(0xFFFFFFFF)
    x = [i & lo32, i >> np.uint64(32), np.zeros(c, np.uint64), np.zeros(c, np.uint64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(q >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), q & lo32, (p >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]),
             p & lo32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return (np.stack(x, 1).reshape(-1)[:n] >> np.uint64(8)).astype(np.int64)


def quantize(x, rule="ceil", seed=None):
    """x [L][K] float64 (values of fp32 or bf16) along its rows -> codes [L][16 nb], scales
    [L][nb] as bytes."""
    L, K = x.shape
    nb = blocks(K)
    b = np.zeros((L, nb * 32))
    b[:, :K] = x
    b = b.reshape(L, nb, 32)
    codes = np.zeros((L, nb, 32), np.uint8)
    scales = np.zeros((L, nb), np.uint8)
    rnd = None if seed is None else philox24(L * nb * 32, seed).reshape(L, nb, 32)
    for l in range(L):
        for j in range(nb):
            v = b[l, j]
            if not np.isfinite(v).all():
                scales[l, j], codes[l, j] = 255, 7
                continue
            amax = np.abs(v).max()
            e = 0 if amax == 0 else _scale_exponent(amax, rule)
            scales[l, j] = e + 127
            a = np.minimum(np.ldexp(np.abs(v), -e), 6.0)
            lo = np.searchsorted(MAG, a, side="right") - 1
            hi = np.minimum(lo + 1, 7)
            if rnd is None:
                mid = (MAG[lo] + MAG[hi]) / 2
                up = (a > mid) | ((a == mid) & (hi % 2 == 0))
            else:
                up = rnd[l, j] * (MAG[hi] - MAG[lo]) < (a - MAG[lo]) * 2.0 ** 24
            c = np.where(up & (hi != lo), hi, lo).astype(np.uint8)
            codes[l, j] = c | (np.signbit(v).astype(np.uint8) << 3)
    codes = codes.reshape(L, nb * 32)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def values(codes, scales, K):
    """The float64 values that codes and scales stand for (NaN under byte 255)."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)[:, :32 * scales.shape[1]]
    v = MAG[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * np.repeat(s, 32, 1))[:, :K]


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def product(x, w, alpha=1.0, bias=None, act=None, bf16=False):
    """Y of x [M][K], w [N][K] float64 and the bound of each element's error."""
    K = x.shape[1]
    y = alpha * (x @ w.T)
    bound = abs(alpha) * (K / 32 + 40) * U * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        y = y + bias
    bound = bound + U * np.abs(y)
    if act == "silu":
        y = silu(y)
        bound = 1.1 * bound + 2.0 ** -20 * np.abs(y) + 2.0 ** -126
    if bf16:
        bound = bound + 2.0 ** -8 * (np.abs(y) + bound)
    return y, bound + 2.0 ** -149


def order(logits):
    """Experts of each token from the greatest logit down, ties to the lower index."""
    return np.argsort(-logits, axis=1, kind="stable")


def moe(x, logits, w13, w2, k, renormalize, bf16):
    """y [T][H] of x [T][H], logits [T][E], w13 [E][2I][H], w2 [E][H][I] float64, with bounds."""
    T, H = x.shape
    I = w2.shape[2]
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    total = np.zeros((T, H))
    split = 2.0 ** -16 if bf16 else 2.0 ** -24
    rank = order(logits)
    for t in range(T):
        ids = rank[t, :k]
        if logits[t].max() == -np.inf:
            continue
        p = np.exp(logits[t] - logits[t].max())
        share = p / (p[ids].sum() if renormalize else p.sum())
        for e in ids:
            if logits[t, e] == -np.inf:
                continue
            g, dg = product(x[t:t + 1], w13[e, :I])
            u, du = product(x[t:t + 1], w13[e, I:])
            h = share[e] * silu(g) * u
            dh = share[e] * (1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du) + (2.0 ** -19 + split) * np.abs(h)
            part = h @ w2[e].T
            size = (np.abs(h) + dh) @ np.abs(w2[e]).T
            y[t] += part[0]
            total[t] += size[0]
            bound[t] += (dh @ np.abs(w2[e]).T)[0] + (I / 32 + 40) * U * size[0]
    bound += k * U * total
    if bf16:
        bound = bound + 2.0 ** -8 * (np.abs(y) + bound)
    return y, bound + 2.0 ** -149
