"""FP8 in blocks of 128 and expert routing in 64 bits, from the definitions, with the error bounds
that the GPU tests assert.  torch on the CPU; shares no code with the library.

Error bounds.  u = 2^-23 bounds a rounding to FP32 whether it rounds or truncates.
  product  products of two FP8 codes are exact in FP32 (8 bits).  Exact accumulation: a product passes
           at most 32 additions inside its matrix instruction, 3 more instructions of its block, the product of
           two scales and the multiply-add of the block, nb blocks, 8 waves: (nb + 48) u T with
           T = |alpha| sum |s x w|.  FP8 matrix cores: at most 16 groups of 8 in its block instead,
           (nb + 32) u T, and the truncation of each group of 8 consecutive codes, at most
           7 * 2^-12 of the largest binade product times the scales.
  epilogue alpha and bias one fma: u |v|; SiLU: slope at most 1.1, 2^-20 relative for its own evaluation;
           rounding to bf16 half a step, 2^-8 relative
  routing  exp, two sums of E terms and two divisions: (E / 64 + 24) u relative for p and shares (a wave sums E / 64
           terms a lane and then six steps; exp is good to a few u, its argument's rounding adds |x - m| u); p below
           exp(-40) is held to u absolutely
"""
import torch

B = 128
U = 2.0 ** -23
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F64 = torch.float64


def blocks(k):
    return (k + B - 1) // B


def decode_table(elem):
    bits, bias = (3, 7) if elem == "e4m3" else (2, 15)
    v = torch.zeros(256, dtype=F64)
    for c in range(256):
        e, m = (c & 127) >> bits, c & (2 ** bits - 1)
        x = 2.0 ** (1 - bias) * m / 2 ** bits if e == 0 else 2.0 ** (e - bias) * (1 + m / 2 ** bits)
        v[c] = -x if c & 128 else x
        if (elem == "e4m3" and c & 127 == 127) or (elem == "e5m2" and e == 31):
            v[c] = float("nan") if elem == "e4m3" or m else (float("-inf") if c & 128 else float("inf"))
    return v


def binade_table(elem):
    bits, bias = (3, 7) if elem == "e4m3" else (2, 15)
    return torch.tensor([2.0 ** (max((c & 127) >> bits, 1) - bias) for c in range(256)], dtype=F64)


def encode(q, elem):
    """Codes of finite values |q| <= fmax: the nearest number by search, ties to the even code."""
    grid = decode_table(elem)[:127 if elem == "e4m3" else 124]
    a = q.abs()
    lo = (torch.searchsorted(grid, a.contiguous(), right=True) - 1).clamp(0, len(grid) - 1)
    hi = (lo + 1).clamp(max=len(grid) - 1)
    mid = (grid[lo] + grid[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return (torch.where(up, hi, lo) | (torch.signbit(q).long() << 7)).to(torch.uint8)


def quantize(x, elem, rule="amax", tile=False):
    """Codes [L][128 nb] and scales [L or tiles][nb] of x [L][K] along its rows."""
    L, K = x.shape
    nb, t = blocks(K), B if tile else 1
    nl = -(-L // t)
    w = torch.zeros((nl * t, nb * B), dtype=F64)
    w[:L, :K] = x.double()
    inside = torch.zeros(w.shape, dtype=torch.bool)
    inside[:L, :K] = True
    w, inside = w.view(nl, t, nb, B), inside.view(nl, t, nb, B)
    amax = w.abs().amax(3).amax(1) if w.numel() else torch.zeros((nl, nb), dtype=F64)
    bad = ~torch.isfinite(amax)
    a = torch.where(bad, torch.ones_like(amax), amax).clamp(min=2.0 ** -100)
    f = torch.full_like(a, FMAX[elem])
    if rule == "amax":
        s, r = (a / f).float().double(), (f / a).float().double()
    else:
        m, ex = torch.frexp(a / f)                       # a / f = m 2^ex: the next power of two, itself if it is one
        s = torch.ldexp(torch.ones_like(a), torch.where(m == 0.5, ex - 1, ex))
        r = 1 / s
    zero = amax == 0
    s, r = torch.where(zero, 1.0, s), torch.where(zero, 1.0, r)
    q = torch.where(torch.isfinite(w), w, 0.0) * r[:, None, :, None]
    q = q.float().double().clamp(-FMAX[elem], FMAX[elem])
    c = encode(q, elem)
    c = torch.where(bad[:, None, :, None] & inside, torch.full_like(c, 0x7F), c)
    s = torch.where(bad, float("nan"), s)
    return c.view(nl * t, nb * B)[:L], s


def values(codes, scales, elem):
    """[L][128 nb] codes and [L or tiles][nb] scales -> float64 values."""
    L, nb = codes.shape[0], scales.shape[1]
    s = scales.double()
    if s.shape[0] != L:
        s = s.repeat_interleave(B, 0)[:L]
    return decode_table(elem)[codes[:, :B * nb].long()] * s.repeat_interleave(B, 1)


def truncation(xc, xs, fx, wc, ws, fw):
    """sum over groups of 8 of 7 * 2^-12 * S * (largest binade product), [M][N]."""
    def binades(c, s, f):
        L, nb = c.shape[0], s.shape[1]
        s = s.double().abs()
        if s.shape[0] != L:
            s = s.repeat_interleave(B, 0)[:L]
        return (binade_table(f)[c[:, :B * nb].long()] * s.repeat_interleave(B, 1)).view(L, -1, 8)
    bx, bw = binades(xc, xs, fx), binades(wc, ws, fw)
    out = torch.zeros((bx.shape[0], bw.shape[0]), dtype=F64)
    for m in range(bx.shape[0]):
        out[m] = (bx[m][None] * bw).amax(2).sum(1)
    return 7 * 2.0 ** -12 * out


def product(xc, xs, fx, wc, ws, fw, accum, alpha=1.0, bias=None, act=None, out=torch.float32):
    """y [M][N] in 64 bits and the bound on a result's distance from it."""
    nb = xs.shape[1]
    x, w = values(xc, xs, fx), values(wc, ws, fw)
    y, t = alpha * (x @ w.T), abs(alpha) * (x.abs() @ w.abs().T)
    tol = (nb + (48 if accum == "fp32" else 32)) * U * t
    if accum == "fp8":
        tol = tol + abs(alpha) * truncation(xc, xs, fx, wc, ws, fw)
    if bias is not None:
        y = y + bias.double()
    tol = tol + U * (y.abs() + tol)
    if act == "silu":
        y = y * torch.sigmoid(y)
        tol = 1.1 * tol + 2.0 ** -20 * y.abs()
    if out == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (y.abs() + tol)
    return y, tol


def check(got, want, tol, what=""):
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what
    off = torch.where(nan, 0.0, (got - want).abs() - tol)
    assert not bool((off > 0).any()), "%s: %d of %d outside the bound, worst by %.3g (bound %.3g)" % (
        what, int((off > 0).sum()), off.numel(), float(off.max()), float(tol.flatten()[off.argmax()]))


def route(logits, k, renorm, mask=None, d_shares=None, d_loss=None):
    """The router in 64 bits, from the definition; the gradient from one-hot rows of the choice."""
    T, E = logits.shape
    z = logits.double()
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    nan = torch.isnan(z).any(1)
    none = (z == float("-inf")).all(1) | ~live
    p = torch.exp(z - torch.where(none, 0.0, z.amax(1))[:, None])
    p = torch.where(none[:, None], 0.0, p / p.sum(1, keepdim=True))
    p = torch.where((nan & live)[:, None], float("nan"), p)
    # NaN first, then falling, ties to the lower index (a stable sort keeps them)
    rank = torch.where(torch.isnan(z), float("inf"), z)
    order = torch.sort(rank + torch.zeros_like(rank), dim=1, descending=True, stable=True)[1]
    if bool(nan.any()):
        assert not bool((z == float("inf")).any()), "a NaN beside an infinity needs an order of its own"
    ids = order[:, :k]
    taken = live[:, None] & ~(torch.gather(z, 1, ids) == float("-inf"))
    experts = torch.where(taken, ids, -1)
    shares = torch.where(taken, torch.gather(p, 1, ids), 0.0)
    if renorm:
        total = shares.sum(1, keepdim=True)
        shares = torch.where(taken, shares / torch.where(total == 0, 1.0, total), 0.0)
    flat = experts.flatten()
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), counts.cumsum(0)))
    slots = torch.full((T * k,), -1)
    n_slots = int(offsets[-1])
    slots[:n_slots] = torch.sort(torch.where(flat < 0, E, flat), stable=True)[1][:n_slots]
    n = max(int(live.sum()), 1)
    slope = E * counts.double() / (n * k) / n
    out = {"experts": experts, "shares": shares, "counts": counts, "offsets": offsets, "order": slots,
           "loss": (slope * p.sum(0)).sum(), "slope": slope, "p": p}
    if d_shares is not None or d_loss is not None:
        ds = torch.where(taken, torch.zeros((T, k), dtype=F64) if d_shares is None else d_shares.double(), 0.0)
        g = (slope * (0.0 if d_loss is None else float(d_loss))).expand(T, E).clone()
        d = torch.zeros((T, E), dtype=F64)
        size = torch.zeros((T, E), dtype=F64)                 # what the gradient is made of, for its bound
        at = torch.where(taken, ids, 0)
        if renorm:
            dot = (shares * ds).sum(1, keepdim=True)
            d.scatter_add_(1, at, torch.where(taken, shares * (ds - dot), 0.0))
            size.scatter_add_(1, at, shares * (ds.abs() + (shares * ds.abs()).sum(1, keepdim=True)))
        else:
            g.scatter_add_(1, at, ds)
        d += p * (g - (p * g).sum(1, keepdim=True))
        d = torch.where(live[:, None], d, 0.0)
        out["d"], out["size"] = d, size + p * (g.abs() + (p * g.abs()).sum(1, keepdim=True))
    return out
