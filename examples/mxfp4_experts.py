"""An expert layer on MXFP4 products: trained with all three products in 4 bits, then served.

A two-layer network of experts, y = relu(x W1[e]^T) W2[e]^T, each token going to the expert a fixed
router names.  Tokens are sorted by expert once a batch; after that every product is one call
over all experts, whose row offsets never leave the GPU:

  forward          mxfp4_gemm_grouped on the rowwise copies of x and W
  input gradient   mxfp4_gemm_grouped on dy's rowwise and W's columnwise copy
  weight gradient  mxfp4_gemm_grouped_wgrad on the columnwise copies of dy and x
  serving          mxfp4_linear on packed weights, a few tokens at a time

Gradients are quantized with stochastic rounding under the scale rule that never saturates, as
NVFP4 training does it.  Run on the GPU:  python examples/mxfp4_experts.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_quantize_amd as nv  # noqa: E402


class GroupedLinear(torch.autograd.Function):
    """y[rows of g] = x[rows of g] W[g]^T with MXFP4 operands; W is kept in float32."""

    @staticmethod
    def forward(ctx, x, w, offsets, seed):
        both = nv.mxfp4_quant_params(True, True, nv.MXFP4_SCALE_CEIL)
        xr, xc = nv.mxfp4_quantize(x, both, offsets=offsets)
        wr, wc = nv.mxfp4_quantize(w, both)
        ctx.copies = xc, wc, offsets, seed
        return nv.mxfp4_gemm_grouped(xr, wr, offsets, out_dtype=torch.bfloat16)

    @staticmethod
    def backward(ctx, dy):
        xc, wc, offsets, seed = ctx.copies
        p = nv.mxfp4_quant_params(True, True, nv.MXFP4_SCALE_CEIL, nv.NVFP4_SR, nv.NVFP4_SR, seed)
        dyr, dyc = nv.mxfp4_quantize(dy.contiguous(), p, offsets=offsets)
        dx = nv.mxfp4_gemm_grouped(dyr, wc, offsets, out_dtype=torch.bfloat16)
        return dx, nv.mxfp4_gemm_grouped_wgrad(dyc, xc, offsets), None, None


def by_expert(expert, n_experts):
    """Token order sorted by expert, and the experts' row offsets (both on the GPU)."""
    order = torch.argsort(expert, stable=True)
    ends = torch.searchsorted(expert[order], torch.arange(n_experts, device=expert.device), right=True)
    return order, torch.cat([ends.new_zeros(1), ends]).int()


def serve(x, experts, w1, w2, n_experts):
    """The layer on packed weights, for any number of tokens."""
    order, offsets = by_expert(experts, n_experts)
    h = nv.mxfp4_linear(x[order], w1, offsets=offsets).relu_()
    y = nv.mxfp4_linear(h, w2, offsets=offsets)
    out = torch.empty_like(y)
    out[order] = y
    return out


def main(steps=60, tokens=2048, width=256, hidden=512, n_experts=8, device="cuda:0", log=print):
    gen = torch.Generator(device=device).manual_seed(0)

    def rand(*shape, std=1.0):
        return std * torch.randn(shape, generator=gen, device=device)

    # the function to learn: a random layer of the same form; a router that leaves an expert idle
    t1, t2 = rand(n_experts, hidden, width, std=width ** -0.5), rand(n_experts, width, hidden, std=hidden ** -0.5)
    router = rand(width, n_experts)
    router[:, -1] = 0
    w1 = rand(n_experts, hidden, width, std=width ** -0.5).requires_grad_()
    w2 = rand(n_experts, width, hidden, std=hidden ** -0.5).requires_grad_()
    opt = torch.optim.Adam([w1, w2], lr=2e-3)

    def target(x, expert):
        h = torch.bmm(t1[expert], x.float().unsqueeze(2)).relu()
        return torch.bmm(t2[expert], h).squeeze(2)

    losses = []
    for step in range(steps):
        x = rand(tokens, width).bfloat16()
        expert = (x.float() @ router)[:, :-1].argmax(1)
        order, offsets = by_expert(expert, n_experts)
        x, expert = x[order], expert[order]
        h = GroupedLinear.apply(x, w1, offsets, 2 * step).relu()
        y = GroupedLinear.apply(h, w2, offsets, 2 * step + 1)
        want = target(x, expert)
        loss = (y.float() - want).square().mean() / want.square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step}: relative squared error {losses[-1]:.4f}")

    row = nv.mxfp4_quant_params()
    packed = [nv.mxfp4_quantize(w.detach(), row)[0] for w in (w1, w2)]
    x = rand(5, width).bfloat16()
    expert = (x.float() @ router)[:, :-1].argmax(1)
    few = serve(x, expert, *packed, n_experts)
    many = serve(x.repeat(200, 1), expert.repeat(200), *packed, n_experts)[:5]
    log(f"served 5 tokens; the same among 1000 differ by {(few.float() - many.float()).abs().max().item():.2g}")
    return losses, few, many


if __name__ == "__main__":
    main()
