"""examples/mxfp4_layer.py: its serving layer against the same layer in float64 on the dequantized
weights, its training gradients against products of the quantized values, its loss."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp4_reference as ref
import mxfp8_block_scaled_03_amd as mxq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_layer.py")
    spec = importlib.util.spec_from_file_location("mxfp4_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def values(q, K):
    codes, scales = (t.cpu().numpy() for t in q)
    return ref.values(codes.reshape(-1, codes.shape[-1]), scales.reshape(-1, scales.shape[-1]), K)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_decoder_layer(example, T):
    H, I, E, k = 160, 72, 6, 2
    layer = example.DecoderLayer(H, I, E, k, DEV, generator(1))
    x = torch.randn((T, H), generator=generator(2), device=DEV).to(torch.bfloat16)
    h = mxq.gemm_fp4(x, None, *layer.projection, H)
    want, bound = ref.product(x.cpu().double().numpy(), values(layer.projection, H), bf16=True)
    assert (np.abs(h.cpu().double().numpy() - want) <= bound).all()
    logits = (h @ layer.router.T).float()
    moe, bound = ref.moe(h.cpu().double().numpy(), logits.cpu().double().numpy(), values(layer.w13, H).reshape(E, 2 * I, H),
                         values(layer.w2, I).reshape(E, H, I), k, True, True)
    y = x.cpu().double().numpy() + moe
    # the sum with x is rounded to bf16 once more
    bound = bound + 2.0 ** -8 * (np.abs(y) + bound)
    assert (np.abs(layer(x).cpu().double().numpy() - y) <= bound).all()


def test_gradients(example):
    M, N, K, seed = 96, 64, 160, 11
    x = torch.randn((M, K), generator=generator(3), device=DEV).to(torch.bfloat16).requires_grad_()
    w = torch.randn((N, K), generator=generator(4), device=DEV).requires_grad_()
    dy = (torch.randn((M, N), generator=generator(5), device=DEV) * 1e-3).to(torch.bfloat16)
    y = example.LinearFp4.apply(x, w, seed)
    y.backward(dy)
    xr, xs, xc, xcs = mxq.quantize_fp4_dual(x.detach())
    wr, ws, wc, wcs = mxq.quantize_fp4_dual(w.detach())
    row, col = mxq.quantize_fp4_sr(dy, seed, "row"), mxq.quantize_fp4_sr(dy, seed + 1, "col")
    for got, a, b, depth, bf16 in ((y, (xr, xs), (wr, ws), K, True), (x.grad, row, (wc, wcs), N, True),
                                   (w.grad, col, (xc, xcs), M, False)):
        want, bound = ref.product(values(a, depth), values(b, depth), bf16=bf16)
        assert (np.abs(got.detach().cpu().double().numpy() - want) <= bound).all()


def test_training_learns(example):
    """The target's mean square is 1 at the start; what remains is the rounding of x and w to 4 bits:
    a relative error of at most 1/4 of each value (half a step of 0.5 below 1, of 1 below 2 ...), with
    values spread over the codes well below 1/4 in the mean square."""
    losses = example.train(25, 512, 256, 128, DEV, generator(6))
    assert 0.5 < losses[0] < 2.0 and all(np.isfinite(losses)) and losses[-1] < 0.25 * losses[0]
