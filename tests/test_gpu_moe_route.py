"""Expert routing on the GPU against 64 bits (b128_reference.route): choices, counts and order exactly, shares,
loss and gradients within derived bounds and against differences."""
import pytest
import torch

import b128_reference as ref
import mxfp8_block_scaled_03_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def logits_of(T, E, dtype, seed, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((T, E), generator=g) * 2
    if masked:
        z = z.masked_fill(torch.rand((T, E), generator=g) < masked, float("-inf"))
    return z.to(dtype)


def check(z, k, renorm, mask=None, seed=0, strided=False):
    T, E = z.shape
    g = torch.Generator().manual_seed(seed)
    ds, dl = torch.randn((T, k), generator=g), torch.tensor([0.7])
    want = ref.route(z, k, renorm, mask, ds, dl)
    d = z.to(DEV)
    if strided:
        d = torch.cat((d, d), 1)[:, :E]
    m = None if mask is None else mask.to(DEV)
    r = mxq.moe_route(d, k, renormalize=renorm, mask=m)
    for name in ("experts", "counts", "offsets", "order"):
        assert torch.equal(getattr(r, name).cpu().long(), want[name]), name
    # relative error of p and shares: the sums, exp and its argument (|x - m| < 40 where p matters)
    rel = (E / 64 + 24 + 40) * ref.U
    ref.check(r.shares, want["shares"], rel * want["shares"].abs() + ref.U, "shares")
    # the loss sums T positive terms: unit by unit, then over at most 1024 units
    add = (T / 1024 + 1024) * ref.U
    ref.check(r.slope, want["slope"], 8 * ref.U * want["slope"], "slope")
    ref.check(r.loss, want["loss"].reshape(1), (rel + add) * want["loss"].abs().reshape(1), "loss")
    half = 2.0 ** -8 if z.dtype == BF16 else 0.0
    for ds_, dl_ in ((ds, dl), (ds, None), (None, dl)):
        w = ref.route(z, k, renorm, mask, ds_, dl_)
        got = mxq.moe_route_grad(d, r, None if ds_ is None else ds_.to(DEV), None if dl_ is None else dl_.to(DEV),
                                 renormalize=renorm, mask=m)
        assert got.dtype == z.dtype
        # both factors of a product are off by rel, the sums over E and k by (E / 64 + 70) u
        tol = (3 * rel + 70 * ref.U) * w["size"] + ref.U * 1e-3
        ref.check(got, w["d"], tol + half * (w["d"].abs() + tol), "d_logits")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (7, 5, 5), (64, 64, 8), (100, 65, 3), (256, 256, 16), (33, 200, 64),
                                   (257, 8, 2), (300, 130, 7), (70, 257, 4), (1500, 40, 6), (40, 1024, 9), (50, 600, 64)])
def test_route(T, E, k, dtype, renorm):
    check(logits_of(T, E, dtype, T + E), k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(60, 33, 4), (400, 70, 5), (1, 3, 2)])
def test_route_masked_tokens_and_experts(T, E, k, renorm):
    """Padding tokens; experts at -inf, some tokens with fewer than k left and some with none."""
    z = logits_of(T, E, F32, 5, masked=0.8)
    z[T // 2] = float("-inf")
    g = torch.Generator().manual_seed(1)
    for mask in (None, torch.rand(T, generator=g) < 0.7, torch.zeros(T, dtype=torch.bool), torch.ones(T, dtype=torch.bool)):
        check(z, k, renorm, mask, strided=True)


def test_route_ties_go_to_the_lower_index():
    z = torch.tensor([[0.0, 1.0, 1.0, -0.0, 0.0, 1.0]]).repeat(300, 1)
    for part in (z[:20], z):
        r = mxq.moe_route(part.to(DEV), 5)
        assert r.experts.cpu().tolist() == [[1, 2, 5, 0, 3]] * len(part)


def test_route_lowest_values_are_not_masked():
    """The type's lowest finite value is a logit like any other; -inf is not."""
    z = torch.full((9, 4), torch.finfo(F32).min)
    z[:, 1] = float("-inf")
    z[3] = torch.finfo(F32).min
    check(z, 4, True)
    check(z, 4, False)


def test_route_nan():
    """A NaN logit is taken first and makes the token's shares, the loss and its gradients NaN; other tokens keep theirs."""
    for T in (10, 300):
        z = logits_of(T, 20, F32, 2)
        clean = mxq.moe_route(z.to(DEV), 3)
        z[4, 7] = float("nan")
        z[5, 2] = -z[4, 7]
        r = mxq.moe_route(z.to(DEV), 3)
        assert r.experts[4, 0] == 7 and r.experts[5, 0] == 2
        assert bool(torch.isnan(r.shares[4:6]).all()) and bool(torch.isnan(r.loss).all())
        keep = torch.tensor([t for t in range(T) if t not in (4, 5)], device=DEV)
        assert torch.equal(r.shares[keep], clean.shares[keep])
        d = mxq.moe_route_grad(z.to(DEV), r, torch.ones_like(r.shares), torch.ones(1, device=DEV))
        assert bool(torch.isnan(d[4:6]).all()) and not bool(torch.isnan(d[keep]).any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), torch.finfo(F32).min])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_padding_of_any_value(renorm, bad):
    """What a padded token holds, logits and incoming gradients, changes nothing, and its own gradients are zero."""
    for T in (40, 700):
        z, mask = logits_of(T, 48, F32, 6), torch.arange(T) % 3 != 1
        clean, filled = z.to(DEV), z.clone()
        filled[~mask] = bad
        filled = filled.to(DEV)
        m, up = mask.to(DEV), torch.ones(1, device=DEV)
        want, got = (mxq.moe_route(x, 5, renormalize=renorm, mask=m) for x in (clean, filled))
        for name in want._fields:
            assert torch.equal(getattr(got, name), getattr(want, name)), name
        ds = torch.randn((T, 5), device=DEV)
        d = mxq.moe_route_grad(clean, want, ds, up, renormalize=renorm, mask=m)
        ds[~m] = bad
        assert torch.equal(mxq.moe_route_grad(filled, got, ds, up, renormalize=renorm, mask=m), d)
        assert bool((d[~m] == 0).all()) and bool((d[m] != 0).any())


def test_route_slots_of_no_expert_pass_nothing_back():
    """Incoming gradients of slots without an expert are not read into the token's own."""
    z = logits_of(90, 20, F32, 7, masked=0.85).to(DEV)
    for renorm in (True, False):
        r = mxq.moe_route(z, 6, renormalize=renorm)
        assert bool((r.experts < 0).any())
        ds = torch.randn((90, 6), device=DEV)
        d = mxq.moe_route_grad(z, r, ds, renormalize=renorm)
        ds[r.experts < 0] = float("nan")
        assert torch.equal(mxq.moe_route_grad(z, r, ds, renormalize=renorm), d)


def test_route_no_tokens():
    r = mxq.moe_route(torch.empty((0, 6), device=DEV), 2)
    assert r.counts.tolist() == [0] * 6 and r.offsets.tolist() == [0] * 7 and r.loss.item() == 0 and r.slope.tolist() == [0] * 6
    assert mxq.moe_route_grad(torch.empty((0, 6), device=DEV), r).shape == (0, 6)


def test_route_many_tokens():
    """More tokens than units: invariants that need no loop over tokens."""
    T, E, k = 50001, 100, 6
    z = torch.randn((T, E), device=DEV)
    mask = torch.rand(T, device=DEV) < 0.9
    r = mxq.moe_route(z, k, mask=mask)
    ids = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k]
    want = torch.where(mask[:, None], ids, -1)
    assert torch.equal(r.experts.long(), want)
    flat = torch.where(want < 0, E, want).flatten()
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    assert torch.equal(r.counts.long(), counts)
    n = int(counts.sum())
    order = torch.sort(flat, stable=True)[1]
    assert torch.equal(r.order[:n].long(), order[:n]) and bool((r.order[n:] == -1).all())
    p = torch.softmax(z.double(), 1) * mask[:, None]
    live = mask.sum()
    loss = (E * counts / (live * k) / live * p.sum(0)).sum()
    assert abs(r.loss.item() - loss.item()) <= (66 + 1.6 + 49 + 1024) * ref.U * loss.item()


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    """The gradient of sum(shares * c) + loss against central differences of the 64-bit forward pass, the choice
    (and with it f) held."""
    T, E, k = 6, 12, 3
    z = logits_of(T, E, F32, 8)
    c = torch.randn((T, k), generator=torch.Generator().manual_seed(3))
    r = mxq.moe_route(z.to(DEV), k, renormalize=renorm)
    got = mxq.moe_route_grad(z.to(DEV), r, c.to(DEV), torch.ones(1, device=DEV), renormalize=renorm).cpu().double()
    ids, slope = r.experts.cpu().long(), r.slope.cpu().double()

    def value(z):
        p = torch.softmax(z, 1)
        s = torch.gather(p, 1, ids)
        s = s / s.sum(1, keepdim=True) if renorm else s
        return (s * c.double()).sum() + (slope * p.sum(0)).sum()

    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = z.double().clone(), z.double().clone()
            up[t, e] += h
            down[t, e] -= h
            # differences are off by h^2 times a third derivative below 10, and 64-bit rounding over h
            assert abs((value(up) - value(down)) / (2 * h) - got[t, e]) < 1e-6 + 1e-9


def test_route_graph_and_side_stream():
    """Captured together (three launches, a workspace each), replayed on new logits."""
    for T in (50, 700):
        z, z2 = torch.randn((T, 32), device=DEV), torch.randn((T, 32), device=DEV)
        up = torch.ones(1, device=DEV)

        def step():
            out = []
            for x in (z, z2):
                r = mxq.moe_route(x, 4)
                out += list(r) + [mxq.moe_route_grad(x, r, r.shares, up)]
            return out
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs = step()
        torch.cuda.current_stream().wait_stream(side)
        for seed in range(3):
            z.normal_()
            z2.normal_()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, step()):
                assert torch.equal(a, b)


@pytest.mark.parametrize("E,k", [(6, 2), (257, 4), (600, 64), (1024, 1)])
def test_route_no_tokens_writes_its_sums(E, k):
    """Without tokens counts, offsets, loss and slope are zeros, written, however many experts there are."""
    i32 = torch.full((2 * E + 1,), 7, dtype=torch.int32, device=DEV)
    f32 = torch.full((E + 1,), 7.0, device=DEV)
    need = mxq.mxq_moe_route_workspace(0, E, k)
    work = torch.full((need + 256,), 7, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    assert mxq.mxq_moe_route(0, E, k, 1, None, mxq.MXQ_F32, E, None, None, None, i32.data_ptr(), i32.data_ptr() + 4 * E, None,
                             f32.data_ptr(), f32.data_ptr() + 4, work.data_ptr() if need else None, need, stream) == 0
    assert bool((i32 == 0).all()) and bool((f32 == 0).all()) and bool((work[need:] == 7).all())
    z = torch.empty((0, E), device=DEV)
    r = mxq.moe_route(z, k)
    assert r.counts.tolist() == [0] * E and r.offsets.tolist() == [0] * (E + 1) and r.loss.item() == 0
    assert mxq.moe_route_grad(z, r).shape == (0, E)


@pytest.mark.parametrize("T", [2 ** 25, 2 ** 25 + 4099, 2 ** 27])
def test_route_loss_of_very_many_tokens(T):
    """All logits equal: p = fl(1 / 5) of every token, all tokens to expert 0, so f = (1, 0, ..) and the loss is 1.  A sum of
    equal terms one after the other rounds the same way each time (2^25 tokens, 8192 a wave: 6e-5 off); as it is taken, a term passes
    256 additions, one for each 256 of its wave's T / 4096 tokens, and those of 8 waves, 4 groups and 7 steps,
    2^-24 each; p, f, slope, its product and the last sums take fewer than 16 roundings more."""
    z = torch.zeros((T, 5), device=DEV)
    r = mxq.moe_route(z, 1)
    assert r.counts.tolist() == [T, 0, 0, 0, 0]
    adds = 256 + (T // 4096 + 255) // 256 + 1 + 8 + 4 + 7
    assert abs(r.loss.item() - 1.0) <= (adds + 16) * 2.0 ** -24


def test_route_infinite_logit():
    """+inf is taken first (after a NaN), the lower index of two; the token's shares and gradients and the loss are NaN, and
    other tokens keep theirs."""
    for T in (10, 700):
        z = logits_of(T, 20, F32, 2)
        clean = mxq.moe_route(z.to(DEV), 3)
        z[4, 7] = z[5, 2] = z[5, 11] = float("inf")
        z[6, 3], z[6, 1] = float("nan"), float("inf")
        r = mxq.moe_route(z.to(DEV), 3)
        assert r.experts[4, 0] == 7 and r.experts[5, :2].tolist() == [2, 11] and r.experts[6, :2].tolist() == [3, 1]
        assert bool(torch.isnan(r.shares[4:7]).all()) and bool(torch.isnan(r.loss).all())
        keep = torch.tensor([t for t in range(T) if not 4 <= t <= 6], device=DEV)
        assert torch.equal(r.shares[keep], clean.shares[keep])
        d = mxq.moe_route_grad(z.to(DEV), r, torch.ones_like(r.shares), torch.ones(1, device=DEV))
        assert bool(torch.isnan(d[4:7]).all()) and not bool(torch.isnan(d[keep]).any())
