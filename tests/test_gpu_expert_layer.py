"""The example layer: its forward pass and every gradient against the same layer in plain fp64, its
single-token form against its batched one, and that it learns."""
import importlib.util
import os

import pytest
import torch

import mx_microscaling_quantize_gb300 as mxq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(layer, x):
    """The layer in fp64, every expert on every token."""
    logits = x @ layer["router"].t()
    p = torch.softmax(logits, -1)
    top, experts = p.topk(layer["k"], dim=-1)
    w = torch.zeros_like(p).scatter(1, experts, top / top.sum(-1, keepdim=True))
    h = torch.nn.functional.silu(torch.einsum("tk,enk->ten", x, layer["up"]))
    y = torch.einsum("ten,ekn->tek", h, layer["down"])
    return torch.einsum("tek,te->tk", y, w) + x @ layer["shared"].t()


# A quantised element is off by at most 2^-4 of itself (three mantissa bits), and a bf16 one by 2^-9;
# the errors of different elements are independent, so a product of two quantised operands with
# elements of random sign is off, in norm, by at most 2^-4 sqrt(2) of itself. The output has four
# quantised operands behind it (x, up, h, down), a gradient of the experts' weights or of x at most eight
# (those, dy, dh and the operands of its own product).
OUTPUT, GRADIENT = 2.0 ** -4 * 4 ** 0.5, 2.0 ** -4 * 8 ** 0.5


@pytest.mark.parametrize("tokens,width,hidden,experts,k", [(1, 128, 64, 4, 1), (300, 256, 160, 8, 3),
                                                           (1024, 512, 256, 16, 4)])
def test_layer_against_plain(example, tokens, width, hidden, experts, k):
    torch.manual_seed(tokens)
    layer = example.ExpertLayer(width, hidden, experts, k).cuda()
    x = torch.randn(tokens, width, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(tokens, width, device="cuda").bfloat16()
    y = layer(x)
    y.backward(dy)
    names = ["router", "up", "down", "shared"]
    ref = {n: getattr(layer, n).detach().double().requires_grad_() for n in names}
    xr = x.detach().double().requires_grad_()
    yr = plain({**ref, "k": k}, xr)
    yr.backward(dy.double())

    def close(got, want, bound):
        got, want = got.detach().double(), want.detach()
        assert (got - want).norm() <= bound * want.norm() + 1e-12

    close(y, yr, OUTPUT)
    close(x.grad, xr.grad, GRADIENT)
    for n in names:
        if k > 1 or n != "router":  # a single weight, made one, has no gradient
            close(getattr(layer, n).grad, ref[n].grad, GRADIENT)
    serving = layer.serving()
    assert torch.equal(serving(x.detach()), y.detach())
    assert mxq.mx_device_errors() == 0


def test_single_tokens_agree_with_the_batch(example):
    torch.manual_seed(3)
    layer = example.ExpertLayer(256, 128, 8, 2).cuda()
    step = layer.serving()
    x = torch.randn(9, 256, device="cuda").bfloat16()
    y = step(x)
    for t in range(9):
        one = step(x[t:t + 1]).double()
        # the same codes and products; the sums' order and the router's rounding may differ
        assert (one - y[t:t + 1].double()).norm() <= 2.0 ** -7 * y[t].double().norm()


def test_training_learns(example):
    _, losses = example.train(steps=12)
    assert losses[-1] < 0.8 * losses[0]
