"""A mixture-of-experts layer trained in FP8: routing with its balance loss, and the experts' products and gradients in
blocks of 128.

    python examples/fp8_moe_layer.py

The tokens' rows are gathered by expert, quantized once for both orientations (along the row for the product, along the
expert's rows for the weight gradient) and multiplied expert by expert; the weights are quantized in tiles, whose
transposed codes serve the gradient of the rows.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_03_amd as mxq  # noqa: E402

B = 128


def quantize_experts(w):
    """Weights [E][N][K], N and K multiples of 128, in tiles: (codes, scales) of the matrices and of their transposes."""
    E, N, K = w.shape
    rc, rs, cc, _ = mxq.quantize_b128_dual(w.reshape(E * N, K), tile=True)
    rs = rs.view(E, N // B, K // B)
    # column k of the stack holds every expert's transposed line k in turn: views, nothing is copied
    return (rc.view(E, N, K), rs), (cc.view(K, E, N).transpose(0, 1), rs.transpose(1, 2))


class ExpertLinear(torch.autograd.Function):
    """y[r] = w_e x[r] for the rows r of expert e: x [R][K] bf16 sorted by expert, w [E][N][K], offsets [E + 1]."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        rc, rs, cc, cs = mxq.quantize_b128_dual(x, offsets=offsets)
        (wc, ws), (wt, wts) = quantize_experts(w)
        ctx.save_for_backward(cc, cs, wt, wts, offsets)
        ctx.dtype = w.dtype
        return mxq.moe_gemm_b128(rc, rs, wc, ws, offsets, x.shape[1], accum="fp8")

    @staticmethod
    def backward(ctx, dy):
        cc, cs, wt, wts, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        rc, rs, dc, ds = mxq.quantize_b128_dual(dy, "e5m2", offsets=offsets)
        dx = mxq.moe_gemm_b128(rc, rs, wt, wts, offsets, dy.shape[1], x_elem="e5m2", accum="fp8")
        return dx, mxq.moe_wgrad_b128(dc, ds, cc, cs, offsets, out_dtype=ctx.dtype), None


class Router(torch.autograd.Function):
    """(shares, balance loss, experts, offsets, order) of logits [T][E]; gradients through the first two."""

    @staticmethod
    def forward(ctx, logits, k):
        r = mxq.moe_route(logits, k)
        ctx.save_for_backward(logits, *r)
        ctx.mark_non_differentiable(r.experts, r.offsets, r.order)
        return r.shares, r.loss, r.experts, r.offsets, r.order

    @staticmethod
    def backward(ctx, d_shares, d_loss, *_):
        logits, *r = ctx.saved_tensors
        return mxq.moe_route_grad(logits, mxq.MoeRoute(*r), d_shares.contiguous(), d_loss), None


class MoeLayer(torch.nn.Module):
    """sum over a token's experts of share * W2_e (silu(W1_e x) * (W3_e x)), weights in FP32, products in FP8."""

    def __init__(self, hidden, inner, experts, top, device, generator):
        super().__init__()
        def normal(*shape):
            return torch.nn.Parameter(torch.randn(shape, generator=generator, device=device) * shape[-1] ** -0.5)
        self.top = top
        self.router, self.w13, self.w2 = normal(experts, hidden), normal(experts, 2 * inner, hidden), normal(experts, hidden, inner)

    def forward(self, x):
        """x [T][hidden] bf16 -> (y, balance loss)."""
        T, H = x.shape
        shares, balance, _, offsets, order = Router.apply(x.float() @ self.router.T, self.top)
        slots = order.long()                                       # every slot has an expert: no token is masked
        rows = x[slots // self.top]
        gate, up = ExpertLinear.apply(rows, self.w13, offsets).float().chunk(2, 1)
        h = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
        out = ExpertLinear.apply(h, self.w2, offsets).float() * shares.flatten()[slots][:, None]
        back = torch.empty_like(slots)
        back[slots] = torch.arange(len(slots), device=x.device)    # a slot's row
        return out[back].view(T, self.top, H).sum(1).to(torch.bfloat16), balance


def train(steps, tokens, layer, device, generator, rate=0.05, weight=0.01):
    """Fits a fixed map of the tokens; the loss and the balance loss before each step."""
    target = torch.randn((layer.w2.shape[1],) * 2, generator=generator, device=device) * layer.w2.shape[1] ** -0.5
    optimizer = torch.optim.SGD(layer.parameters(), lr=rate)
    said = []
    for _ in range(steps):
        x = torch.randn((tokens, target.shape[0]), generator=generator, device=device).to(torch.bfloat16)
        y, balance = layer(x)
        loss = (y.float() - x.float() @ target.T).square().sum(1).mean()
        optimizer.zero_grad()
        (loss + weight * balance.sum()).backward()
        optimizer.step()
        said.append((loss.detach(), balance.detach().sum()))
    return [(a.item(), b.item()) for a, b in said]


def main():
    device = "cuda:0"
    generator = torch.Generator(device=device)
    generator.manual_seed(0)
    layer = MoeLayer(256, 256, 8, 2, device, generator)
    said = train(30, 2048, layer, device, generator)
    (loss, balance), (last, last_balance) = said[0], said[-1]
    print("loss %.3f -> %.3f, balance loss %.3f -> %.3f" % (loss, last, balance, last_balance))


if __name__ == "__main__":
    main()
