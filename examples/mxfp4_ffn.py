"""A gated feed-forward block on MXFP4 products: trained with its activations kept in 8 bits, then served.

y = (silu(x Wg^T) * (x Wu^T)) W2^T, W1 = [Wg; Wu].  What a training step runs:

  forward          mxfp8_quantize keeps x; mxfp8_to_mxfp4 makes its rowwise copy; mxfp4_gated gives H packed
                   and the checkpoint of G and U; mxfp4_gemm gives y
  backward         mxfp4_gated_backward: dH = dy W2, [dG dU] and H from the checkpoint, in one kernel;
                   mxfp8_to_mxfp4 makes the columnwise copy of x; three mxfp4_gemm give dx, dW1, dW2
  serving          mxfp4_gated_linear and mxfp4_linear on packed weights, a few tokens at a time

Between forward and backward a token costs 33/32 bytes for each element of x, G and U.  Gradients are quantized
with stochastic rounding under the scale rule that never saturates.  Run on the GPU:  python
examples/mxfp4_ffn.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_quantize_amd as nv  # noqa: E402

CEIL = nv.MXFP4_SCALE_CEIL
ROW, COL = nv.mxfp4_quant_params(True, False, CEIL), nv.mxfp4_quant_params(False, True, CEIL)
BOTH = nv.mxfp4_quant_params(True, True, CEIL)


class GatedBlock(torch.autograd.Function):
    """The block with MXFP4 operands; x is bfloat16, weights are kept in float32."""

    @staticmethod
    def forward(ctx, x, w1, w2, seed):
        (w1r, w1c), (w2r, w2c) = nv.mxfp4_quantize(w1, BOTH), nv.mxfp4_quantize(w2, BOTH)
        x8 = nv.mxfp8_quantize(x)
        xr, _ = nv.mxfp8_to_mxfp4(x8, ROW)
        _, h, kept = nv.mxfp4_gated(xr, w1r, out_dtype=None, packed=True, scale_rule=CEIL, checkpoint=True)
        ctx.kept = x8, kept, w1c, w2c, seed
        return nv.mxfp4_gemm(h, w2r, out_dtype=torch.bfloat16)

    @staticmethod
    def backward(ctx, dy):
        x8, kept, w1c, w2c, seed = ctx.kept
        def stochastic(i):
            return nv.mxfp4_quant_params(True, True, CEIL, nv.NVFP4_SR, nv.NVFP4_SR, 2 * seed + i)
        dyr, dyc = nv.mxfp4_quantize(dy.contiguous(), stochastic(0))
        dgu, h = nv.mxfp4_gated_backward(dyr, w2c, kept, h=True)
        dr, dc = nv.mxfp4_quantize(dgu, stochastic(1))
        _, hc = nv.mxfp4_quantize(h, COL)
        _, xc = nv.mxfp8_to_mxfp4(x8, COL)
        return nv.mxfp4_gemm(dr, w1c, out_dtype=torch.bfloat16), nv.mxfp4_gemm(dc, xc), nv.mxfp4_gemm(dyc, hc), None


def serve(x, w1, w2):
    """The block on packed weights, for any number of tokens."""
    return nv.mxfp4_linear(nv.mxfp4_gated_linear(x, w1), w2)


def main(steps=60, tokens=2048, width=256, hidden=512, device="cuda:0", log=print):
    gen = torch.Generator(device=device).manual_seed(0)

    def rand(*shape, std=1.0):
        return std * torch.randn(shape, generator=gen, device=device)

    # the function to learn: a random block of the same form
    t1, t2 = rand(2 * hidden, width, std=2 * width ** -0.5), rand(width, hidden, std=hidden ** -0.5)
    w1 = rand(2 * hidden, width, std=2 * width ** -0.5).requires_grad_()
    w2 = rand(width, hidden, std=hidden ** -0.5).requires_grad_()
    opt = torch.optim.Adam([w1, w2], lr=2e-3)
    losses = []
    for step in range(steps):
        x = rand(tokens, width).bfloat16()
        g, u = (x.float() @ t1.t()).chunk(2, dim=1)
        want = (torch.nn.functional.silu(g) * u) @ t2.t()
        y = GatedBlock.apply(x, w1, w2, step)
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
    few, many = serve(x, *packed), serve(x.repeat(200, 1), *packed)[:5]
    log(f"served 5 tokens; the same among 1000 differ by {(few.float() - many.float()).abs().max().item():.2g}")
    return losses, few, many


if __name__ == "__main__":
    main()
