"""The example block that keeps 8 bits: its forward pass and every gradient against the same block in plain
fp64, frozen parameters, and its training."""
import importlib.util
import os

import pytest
import torch

import mx_microscaling_quantize_gb300 as mxq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "checkpointed_block.py")
    spec = importlib.util.spec_from_file_location("checkpointed_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain(p, x, kind):
    act = {mxq.SILU: torch.nn.functional.silu, mxq.GELU: torch.nn.functional.gelu,
           mxq.GELU_TANH: lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[kind]
    n = torch.nn.functional.layer_norm(x, x.shape[1:], p["weight"], p["bias"])
    gate, up = (n @ p["up"].t()).chunk(2, 1)
    return x + (act(gate) * up) @ p["down"].t()


# A quantised element is off by at most 2^-4 of itself and a bf16 one by 2^-8, the errors of different elements
# independent, so that a product of operands with elements of random sign is off, in norm, by at most 2^-4 times
# the root of the roundings behind it: of the block's output four (norm, up, activation, down), of a
# gradient at most nine (dy, down, the checkpoint of the activation's input, which itself has two behind it, du, up,
# the norm's checkpoint, and the operand of the gradient's own product).
OUTPUT, GRADIENT = 2.0 ** -4 * 4 ** 0.5, 2.0 ** -4 * 9 ** 0.5


@pytest.mark.parametrize("tokens,width,hidden", [(1, 128, 128), (300, 256, 384), (1024, 512, 1024)])
@pytest.mark.parametrize("kind", [mxq.SILU, mxq.GELU, mxq.GELU_TANH])
def test_block_against_plain(example, tokens, width, hidden, kind):
    torch.manual_seed(tokens)
    block = example.ResidualBlock(width, hidden, kind).cuda()
    with torch.no_grad():
        block.weight.add_(0.1 * torch.randn_like(block.weight))
        block.bias.add_(0.1 * torch.randn_like(block.bias))
    x = torch.randn(tokens, width, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(tokens, width, device="cuda").bfloat16()
    y = block(x)
    y.backward(dy)
    ref = {n: p.detach().double().requires_grad_() for n, p in block.named_parameters()}
    xr = x.detach().double().requires_grad_()
    yr = plain(ref, xr, kind)
    yr.backward(dy.double())

    def close(got, want, less, bound):
        got, want = got.detach().double() - less, want.detach() - less
        assert (got - want).norm() <= bound * want.norm() + 2.0 ** -8 * float(torch.as_tensor(less).norm())

    close(y, yr, xr.detach(), OUTPUT)  # without the stream, whose rounding to bf16 is allowed for
    close(x.grad, xr.grad, dy.double(), GRADIENT)
    for name, p in block.named_parameters():
        close(p.grad, ref[name].grad, 0.0, GRADIENT)
    assert mxq.mx_device_errors() == 0


@pytest.mark.parametrize("frozen", [("up",), ("down", "bias"), ("weight", "bias", "up", "down")])
def test_frozen_parameters_have_no_gradient_and_change_no_other(example, frozen):
    torch.manual_seed(3)
    block = example.ResidualBlock(128, 128).cuda()
    x = torch.randn(200, 128, device="cuda").bfloat16().requires_grad_()
    block(x).sum().backward()
    want = {n: p.grad for n, p in block.named_parameters()}
    want_x, x.grad = x.grad, None
    for n, p in block.named_parameters():
        p.grad = None
        p.requires_grad_(n not in frozen)
    block(x).sum().backward()
    assert torch.equal(x.grad, want_x)
    for n, p in block.named_parameters():
        assert p.grad is None if n in frozen else torch.equal(p.grad, want[n])


def test_second_derivatives_are_refused(example):
    block = example.ResidualBlock(128, 128).cuda()
    x = torch.randn(8, 128, device="cuda").bfloat16().requires_grad_()
    g, = torch.autograd.grad(block(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().square().sum().backward()


def test_example_trains(example):
    _, losses = example.train(steps=3)
    assert len(losses) == 3 and all(torch.isfinite(torch.tensor(v)) for v in losses)


def test_example_runs(example, capsys):
    example.main(["--steps", "2"])
    assert capsys.readouterr().out.count("step") == 2
