"""A residual block of a language model (layer norm, gated projection, activation, projection back) whose
training step keeps nothing but 8-bit operands between its forward and its backward pass:

    layer norm -> product -> gated activation -> product -> plus the residual stream

What the backward pass reads are the codes the forward pass made: the norm's input and output (2.1 bytes per
token and column of the stream, 4 in bf16) and the activation's (3.1 per hidden column, 6 in bf16).

    python examples/checkpointed_block.py [--steps N]
"""
import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mx_microscaling_quantize_gb300 as mxq  # noqa: E402


class Block(torch.autograd.Function):
    """x + act_gated(norm(x) @ up^T) @ down^T: x bf16 [T, D], up fp32 [2 H, D], down fp32 [D, H] (D and H
    multiples of 128)."""

    @staticmethod
    def forward(ctx, x, weight, bias, up, down, kind):
        uc, us, uct, ust = mxq.mx_quantize_b128_blocks(up.bfloat16(), transpose=True)
        dc, ds, dct, dst = mxq.mx_quantize_b128_blocks(down.bfloat16(), transpose=True)
        n, ns, mean, rstd, kept, kept_s = mxq.mx_layer_norm_b128(x, weight, bias, stats=True, checkpoint=True)
        h, hs, u, u_s = mxq.mx_activation_b128(mxq.mx_gemm_b128(n, ns, uc, us), kind, checkpoint=True)
        ctx.save_for_backward(n, ns, mean, rstd, kept, kept_s, h, hs, u, u_s, uct, ust, dct, dst, weight)
        ctx.kind = kind
        return mxq.mx_gemm_b128(h, hs, dc, ds).add_(x)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        n, ns, mean, rstd, kept, kept_s, h, hs, u, u_s, uct, ust, dct, dst, weight = ctx.saved_tensors
        dy = dy.contiguous()
        dup = ddown = None
        dh = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(dy), dct, dst)
        if ctx.needs_input_grad[4]:
            ddown = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_cols(dy), *mxq.mx_requantize_b128_cols(h, hs),
                                     mxq.B128_ROWS, out_dtype=torch.float32)
        want_up = ctx.needs_input_grad[3]
        du = mxq.mx_activation_backward(dh, u, ctx.kind, u_scales=u_s, grad=want_up, operand=True)
        if want_up:
            dup = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_cols(du[0]), *mxq.mx_requantize_b128_cols(n, ns),
                                   mxq.B128_ROWS, out_dtype=torch.float32)
        dn = mxq.mx_gemm_b128(*du[-2:], uct, ust)
        dx, dweight, dbias = mxq.mx_layer_norm_backward(
            dn, kept, mean, rstd, weight, x_scales=kept_s, weight_grad=ctx.needs_input_grad[1],
            bias_grad=ctx.needs_input_grad[2])
        return dx.add_(dy), dweight, dbias, dup, ddown, None


class ResidualBlock(torch.nn.Module):
    def __init__(self, width=512, hidden=1024, kind=mxq.SILU):
        super().__init__()
        self.kind = kind
        self.weight = torch.nn.Parameter(torch.ones(width))
        self.bias = torch.nn.Parameter(torch.zeros(width))
        self.up = torch.nn.Parameter(torch.randn(2 * hidden, width) / width ** 0.5)
        self.down = torch.nn.Parameter(torch.randn(width, hidden) / hidden ** 0.5)

    def forward(self, x):  # bf16 [T, width]
        return Block.apply(x, self.weight, self.bias, self.up, self.down, self.kind)


def train(steps=20, tokens=1024, width=512, hidden=1024):
    """Fits a random block of the same kind; returns (block, losses)."""
    torch.manual_seed(0)
    block, teacher = ResidualBlock(width, hidden).cuda(), ResidualBlock(width, hidden).cuda()
    optimizer = torch.optim.Adam(block.parameters(), lr=3e-3)
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    with torch.no_grad():
        target = teacher(x).float()
    losses = []
    for _ in range(steps):
        loss = (block(x).float() - target).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    return block, losses


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=20)
    args = parser.parse_args(argv)
    _, losses = train(args.steps)
    for i, loss in enumerate(losses):
        print(f"step {i:3d}  loss {loss:.4f}")
    assert mxq.mx_device_errors() == 0


if __name__ == "__main__":
    main()
