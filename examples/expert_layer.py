"""A layer of routed experts beside a shared linear layer, trained and then served, with every product
in E4M3 with a scale per block of 128:

    route -> order the choices by expert -> quantise the experts' rows -> products by expert
          -> activation -> products by expert -> join the experts' rows

    python examples/expert_layer.py [--steps N]

The autograd functions below are what a model's own layer needs; the weights are fp32 masters that are
quantised once per step (and once in all for serving).
"""
import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mx_microscaling_quantize_gb300 as mxq  # noqa: E402


class Route(torch.autograd.Function):
    """logits [T, E] -> (experts [T, k], weights [T, k])."""

    @staticmethod
    def forward(ctx, logits, k):
        experts, weights = mxq.mx_route(logits, k, mxq.SOFTMAX)
        ctx.save_for_backward(logits, experts)
        ctx.mark_non_differentiable(experts)
        return experts, weights

    @staticmethod
    @once_differentiable
    def backward(ctx, _, grad_weights):
        logits, experts = ctx.saved_tensors
        return mxq.mx_route_backward(grad_weights.contiguous(), logits, experts, mxq.SOFTMAX), None


class Combine(torch.autograd.Function):
    """Experts' rows [R, N] -> tokens [T, N], weighted."""

    @staticmethod
    def forward(ctx, y, slots, weights):
        ctx.save_for_backward(y, slots, weights)
        return mxq.mx_combine(y, slots, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        dy, dweights = mxq.mx_combine_backward(dout.contiguous(), *ctx.saved_tensors)
        return dy, None, dweights


class Linear(torch.autograd.Function):
    """bf16 [M, K] times the transpose of fp32 [N, K] -> bf16 [M, N]."""

    @staticmethod
    def forward(ctx, x, w):
        codes, scales, codes_t, scales_t = mxq.mx_quantize_b128_blocks(w.bfloat16(), transpose=True)
        ctx.save_for_backward(x, codes_t, scales_t)
        return mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(x), codes, scales)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, codes_t, scales_t = ctx.saved_tensors
        dy, dx, dw = dy.contiguous(), None, None
        if ctx.needs_input_grad[0]:
            dx = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(dy), codes_t, scales_t)
        if ctx.needs_input_grad[1]:
            dw = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_cols(dy), *mxq.mx_quantize_b128_cols(x),
                                  mxq.B128_ROWS, out_dtype=torch.float32)
        return dx, dw


class ExpertLinear(torch.autograd.Function):
    """Rows by expert times that expert's fp32 [N, K]. With tokens and slots the rows are gathered from
    x [T, K] on the way (and their gradients added up); without, x is [R, K] already."""

    @staticmethod
    def forward(ctx, x, w, row_offsets, tokens=None, slots=None):
        codes, scales, codes_t, scales_t = mxq.mx_quantize_b128_blocks(w.bfloat16(), transpose=True)
        ctx.save_for_backward(x, codes_t, scales_t, row_offsets, tokens, slots)
        return mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(x, tokens), codes, scales, row_offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, codes_t, scales_t, row_offsets, tokens, slots = ctx.saved_tensors
        dy, dx, dw = dy.contiguous(), None, None
        if ctx.needs_input_grad[0]:
            dx = mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(dy), codes_t, scales_t, row_offsets)
            if slots is not None:
                dx = mxq.mx_combine(dx, slots)  # weights of one: the sum of a token's rows
        if ctx.needs_input_grad[1]:
            dw = mxq.mx_gemm_b128_grouped_wgrad(*mxq.mx_quantize_b128_cols(dy, None, row_offsets),
                                                *mxq.mx_quantize_b128_cols(x, tokens, row_offsets),
                                                row_offsets)
        return dx, dw, None, None, None


class ExpertLayer(torch.nn.Module):
    def __init__(self, width=512, hidden=256, experts=16, k=4):
        super().__init__()
        self.k = k
        self.router = torch.nn.Parameter(torch.randn(experts, width) / width ** 0.5)
        self.up = torch.nn.Parameter(torch.randn(experts, hidden, width) / width ** 0.5)
        self.down = torch.nn.Parameter(torch.randn(experts, width, hidden) / hidden ** 0.5)
        self.shared = torch.nn.Parameter(torch.randn(width, width) / width ** 0.5)

    def forward(self, x):  # bf16 [T, width]
        experts, weights = Route.apply(x.float() @ self.router.t(), self.k)
        row_offsets, tokens, slots = mxq.mx_route_plan(experts, self.router.shape[0])
        h = ExpertLinear.apply(x, self.up, row_offsets, tokens, slots)
        y = ExpertLinear.apply(torch.nn.functional.silu(h), self.down, row_offsets)
        return Combine.apply(y, slots, weights) + Linear.apply(x, self.shared)

    def serving(self):
        """The forward pass alone, with the weights quantised once: a function of x."""
        up, down, shared = (mxq.mx_quantize_b128_blocks(w.detach().bfloat16())
                            for w in (self.up, self.down, self.shared))
        router = self.router.detach().t()
        E, k = self.router.shape[0], self.k

        def step(x):
            experts, weights = mxq.mx_route(x.float() @ router, k)
            row_offsets, tokens, slots = mxq.mx_route_plan(experts, E)
            h = mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(x, tokens), *up, row_offsets)
            h = torch.nn.functional.silu(h)
            y = mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(h), *down, row_offsets)
            return mxq.mx_combine(y, slots, weights).add_(
                mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(x), *shared))

        return step


def train(steps=20, tokens=1024, width=512):
    """Fits a random layer of the same kind; returns (layer, losses)."""
    torch.manual_seed(0)
    layer, teacher = ExpertLayer(width).cuda(), ExpertLayer(width).cuda()
    optimizer = torch.optim.Adam(layer.parameters(), lr=3e-3)
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    with torch.no_grad():
        target = teacher(x).float()
    losses = []
    for _ in range(steps):
        loss = (layer(x).float() - target).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    return layer, losses


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=20)
    args = parser.parse_args(argv)
    layer, losses = train(args.steps)
    for i, loss in enumerate(losses):
        print(f"step {i:3d}  loss {loss:.4f}")

    # serving one token at a time, captured once and replayed on each new token
    step, x = layer.serving(), torch.zeros(1, 512, device="cuda", dtype=torch.bfloat16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(x)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(x)
    for i in range(4):
        x.copy_(torch.randn_like(x))
        graph.replay()
        print(f"token {i}  |y| {y.float().norm().item():.3f}")
    assert mxq.mx_device_errors() == 0


if __name__ == "__main__":
    main()
