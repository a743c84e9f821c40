"""The MXFP4 operators as a program uses them.

    python examples/mxfp4_layer.py

`DecoderLayer` serves: a projection and a mixture-of-experts layer whose weights were quantized once,
for the few tokens of a decoding step.  `LinearFp4` trains: a linear layer whose three products run on
MXFP4 operands, the gradient rounded stochastically.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_03_amd as mxq  # noqa: E402


def quantize_stack(w):
    """Codes [E][rows][..] and scales [E][rows][..] of weights [E][rows][K], along K."""
    E, rows, K = w.shape
    codes, scales = mxq.quantize_fp4(w.reshape(E * rows, K))
    return codes.view(E, rows, -1), scales.unflatten(0, (E, rows))


class DecoderLayer:
    """x + experts(router(h), h) with h = x W_p: all large weights in MXFP4 (4.25 bits each)."""

    def __init__(self, hidden, inner, experts, top, device, generator):
        def normal(*shape):
            return (torch.randn(shape, generator=generator, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)
        self.hidden, self.top = hidden, top
        self.projection = mxq.quantize_fp4(normal(hidden, hidden))
        self.router = normal(experts, hidden)
        self.w13 = quantize_stack(normal(experts, 2 * inner, hidden))
        self.w2 = quantize_stack(normal(experts, hidden, inner))

    def __call__(self, x):
        h = mxq.gemm_fp4(x, None, *self.projection, self.hidden)
        logits = (h @ self.router.T).float()
        return x + mxq.moe_fp4(h, logits, *self.w13, *self.w2, self.top)


class LinearFp4(torch.autograd.Function):
    """y = x w^T: x [M][K] bf16, w [N][K] fp32.  Both are quantized along K for y, and from the same
    read along the other axis for the gradients."""

    @staticmethod
    def forward(ctx, x, w, seed):
        xr, xr_s, xc, xc_s = mxq.quantize_fp4_dual(x)
        wr, wr_s, wc, wc_s = mxq.quantize_fp4_dual(w)
        ctx.save_for_backward(xc, xc_s, wc, wc_s)
        ctx.seed = seed
        return mxq.gemm_fp4(xr, xr_s, wr, wr_s, x.shape[1])

    @staticmethod
    def backward(ctx, dy):
        xc, xc_s, wc, wc_s = ctx.saved_tensors
        dy = dy.contiguous()
        M, N = dy.shape
        rows = mxq.quantize_fp4_sr(dy, ctx.seed, "row")
        cols = mxq.quantize_fp4_sr(dy, ctx.seed + 1, "col")
        return (mxq.gemm_fp4(*rows, wc, wc_s, N), mxq.gemm_fp4(*cols, xc, xc_s, M, out_dtype=torch.float32), None)


def train(steps, tokens, inputs, outputs, device, generator, rate=0.25):
    """Fits a linear map from noisy samples; the loss before each step."""
    target = torch.randn((outputs, inputs), generator=generator, device=device) * inputs ** -0.5
    w = torch.zeros_like(target, requires_grad=True)
    losses = []
    for step in range(steps):
        x = torch.randn((tokens, inputs), generator=generator, device=device).to(torch.bfloat16)
        y = LinearFp4.apply(x, w, 2 * step).float()
        loss = (y - x.float() @ target.T).square().mean()
        loss.backward()
        with torch.no_grad():
            w -= rate * outputs * w.grad / 2
            w.grad = None
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def main():
    device = "cuda:0"
    generator = torch.Generator(device=device)
    generator.manual_seed(0)
    layer = DecoderLayer(2048, 1024, 32, 4, device, generator)
    x = torch.randn((4, 2048), generator=generator, device=device).to(torch.bfloat16)
    for _ in range(4):
        x = layer(x)
    print("decoded 4 steps of 4 tokens, root mean square %.3f" % x.float().square().mean().sqrt().item())
    losses = train(30, 1024, 512, 256, device, generator)
    print("trained: loss %.4f -> %.4f" % (losses[0], losses[-1]))


if __name__ == "__main__":
    main()
