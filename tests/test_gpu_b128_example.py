"""The FP8 mixture-of-experts layer of examples/fp8_moe_layer.py: its functions' results and gradients against 64 bits
on the very operands that they quantize, and the whole layer against a layer without quantization."""
import importlib.util
import os

import pytest
import torch

import b128_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("fp8_moe_layer", os.path.join(ROOT, "examples", "fp8_moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("sizes", [[40, 0, 130], [1, 1, 300, 0, 5]])
def test_expert_linear(ex, sizes):
    E, N, K, R = len(sizes), 256, 384, sum(sizes)
    x, w, dy = normal(1, R, K).to(BF16), normal(2, E, N, K), normal(3, R, N).to(BF16)
    offsets = torch.tensor([0] + sizes).cumsum(0).int()
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    y = ex.ExpertLinear.apply(xd, wd, offsets.to(DEV))
    y.backward(dy.to(DEV))
    first = 0
    for e, n in enumerate(sizes):
        at = slice(first, first + n)
        first += n
        if n == 0:
            assert bool((wd.grad[e] == 0).all())
            continue
        wc, ws = ref.quantize(w[e], "e4m3", tile=True)
        want, tol = ref.product(*ref.quantize(x[at], "e4m3"), "e4m3", wc, ws, "e4m3", "fp8", out=BF16)
        ref.check(y[at], want, tol, "y")
        tc, ts = ref.quantize(w[e].T, "e4m3", tile=True)
        want, tol = ref.product(*ref.quantize(dy[at], "e5m2"), "e5m2", tc, ts, "e4m3", "fp8", out=BF16)
        ref.check(xd.grad[at], want, tol, "dx")
        want, tol = ref.product(*ref.quantize(dy[at].T, "e5m2"), "e5m2", *ref.quantize(x[at].T, "e4m3"), "e4m3", "fp32")
        ref.check(wd.grad[e], want, tol, "dw")


def test_router(ex):
    T, E, k = 300, 16, 3
    z, c = normal(4, T, E), normal(5, T, k)
    zd = z.to(DEV).requires_grad_()
    shares, loss, experts, offsets, order = ex.Router.apply(zd, k)
    ((shares * c.to(DEV)).sum() + 0.5 * loss.sum()).backward()
    want = ref.route(z, k, True, None, c, torch.tensor(0.5))
    assert torch.equal(experts.cpu().long(), want["experts"]) and torch.equal(order.cpu().long(), want["order"])
    ref.check(zd.grad, want["d"], 300 * ref.U * want["size"] + 1e-10, "logits")


def test_layer_against_an_unquantized_one(ex):
    """Every operand of a product is off by at most 2^-4 (E4M3) or 2^-3 (E5M2) of its value, evenly spread: 3.6 and 7.2 % root
    mean square.  A result of one product of random operands is off by the root of the two squares' sum, and two
    products and the nonlinearity follow one another: up to 8 % for y, 14 % for gradients, and as much again as room."""
    T, H, I, E, k = 400, 256, 128, 6, 2
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    layer = ex.MoeLayer(H, I, E, k, DEV, g)
    x = normal(8, T, H).to(BF16)
    xd = x.to(DEV).requires_grad_()
    c = normal(9, T, H)
    y, balance = layer(xd)
    ((y.float() * c.to(DEV)).sum() + balance.sum()).backward()
    p = {n: t.detach().cpu().double().requires_grad_() for n, t in layer.named_parameters()}
    xr = x.double().requires_grad_()
    logits = xr @ p["router"].T
    prob = torch.softmax(logits, 1)
    ids = ref.route((x.to(DEV).float() @ layer.router.detach().T).cpu(), k, True)["experts"]
    share = torch.gather(prob, 1, ids)
    share = share / share.sum(1, keepdim=True)
    out = torch.zeros((T, H), dtype=F64)
    for j in range(k):
        w13, w2 = p["w13"][ids[:, j]], p["w2"][ids[:, j]]
        gu = (w13 @ xr[:, :, None])[:, :, 0]
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        out = out + share[:, j, None] * (w2 @ h[:, :, None])[:, :, 0]
    f = torch.bincount(ids.flatten(), minlength=E).double() / (T * k)
    loss = E * (f * prob.mean(0)).sum()
    ((out * c.double()).sum() + loss).backward()
    assert abs(balance.item() - loss.item()) < 1e-4 * loss.item()

    def off(a, b):
        return float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm())
    assert off(y, out) < 0.16
    for name, a, b in [("x", xd.grad, xr.grad)] + [(n, t.grad, p[n].grad) for n, t in layer.named_parameters()]:
        assert off(a, b) < 0.28, name


def test_train_runs(ex):
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    layer = ex.MoeLayer(128, 128, 5, 2, DEV, g)
    said = ex.train(3, 300, layer, DEV, g)
    assert len(said) == 3 and all(abs(a) < 1e6 and 0.9 < b < 5 for a, b in said)


def test_captured_gradients(ex):
    """Forward and backward of the experts' product in one graph, replayed on new rows and offsets with eager work
    between the replays."""
    E, N, K, R = 4, 256, 128, 300
    x, w = normal(1, R, K).to(BF16).to(DEV).requires_grad_(), normal(2, E, N, K).to(DEV).requires_grad_()
    dy = normal(3, R, N).to(BF16).to(DEV)
    offsets = torch.tensor([0, 100, 100, 250, 300], dtype=torch.int32, device=DEV)

    def step():
        y = ex.ExpertLinear.apply(x, w, offsets)
        return [y.detach(), *torch.autograd.grad(y, (x, w), dy)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (3, 4, 5):
        with torch.no_grad():
            x.copy_(normal(seed, R, K).to(BF16))
            offsets.copy_(torch.tensor([0, 10 * seed, 10 * seed, 250, 300], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
