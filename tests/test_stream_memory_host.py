"""Under which stream the binding takes memory, on the CPU: tensors that say they are on the device, a
library that accepts everything, and an allocator that notes the stream it was called under."""

import contextlib

import pytest
import torch

import mx_microscaling_quantize_gb300 as mxq

SIDE = 0x5510  # a raw handle, never dereferenced


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def on_device(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


class Library:
    """Every entry point succeeds; sizes are asked of the real shapes' formulas."""

    def __getattr__(self, name):
        def call(*args):
            if name == "mx_route_plan_workspace":
                args[3]._obj.value = 4096
            return 0
        return call


@pytest.fixture
def noted(monkeypatch):
    """The (stream, bytes) of every allocation, and the streams that outputs were recorded on."""
    state = {"stream": "current", "taken": [], "recorded": []}
    real = torch.empty

    def empty(*args, **kwargs):
        t = real(*args, **kwargs)
        state["taken"].append((state["stream"], t.numel() * t.element_size()))
        return t

    @contextlib.contextmanager
    def under(stream):
        before, state["stream"] = state["stream"], stream
        try:
            yield
        finally:
            state["stream"] = before

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state["stream"])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state["recorded"].append(s))
    monkeypatch.setattr(mxq, "_lib", Library())
    monkeypatch.setattr(mxq, "_raw_stream", lambda device: 0)
    sizes = mxq.mx_route_plan_workspace  # remembers what the library answered
    sizes.cache_clear()
    yield state
    sizes.cache_clear()


def test_the_plans_workspace_is_of_the_stream_it_is_used_on(noted):
    experts = on_device(4096, 2, dtype=torch.int32)
    out = dict(row_offsets=on_device(9, dtype=torch.int64), tokens=on_device(8192, dtype=torch.int32),
               slots=on_device(4096, 2, dtype=torch.int32))
    mxq.mx_route_plan(experts, 8, **out, stream=SIDE)
    assert noted["taken"] == [(SIDE, 4096)]
    mxq.mx_route_plan(experts, 8, **out)
    assert noted["taken"][1:] == [("current", 4096)]
    mxq.mx_route_plan(experts, 8, **out, stream=1)  # the default stream's other handle
    assert noted["taken"][2:] == [(0, 4096)]


def calls():
    """(name, a call with every output left to the binding)."""
    bf16, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    x, H, gs = on_device(128, 256, dtype=bf16), on_device(32, 32, dtype=bf16), on_device(1)
    codes, scales = on_device(128, 256, dtype=u8), on_device(128, 8, dtype=u8)
    offsets = on_device(2, dtype=torch.int64)
    logits, experts, weights = on_device(16, 8), on_device(16, 2, dtype=i32), on_device(16, 2)
    rows = codes, on_device(2, 128)  # scales [K / 128, rows]
    blocks = codes, on_device(1, 2)
    y, slots = on_device(32, 256, dtype=bf16), on_device(16, 2, dtype=i32)
    dout = on_device(16, 256, dtype=bf16)
    return [
        ("quantize", lambda **s: mxq.mx_quantize(x, mxq.E4M3, **s)),
        ("qdq", lambda **s: mxq.mx_qdq(x, mxq.E4M3, **s)),
        ("rotate_quantize", lambda **s: mxq.mx_rotate_quantize(x, H, mxq.E4M3, **s)),
        ("quantize_grouped", lambda **s: mxq.mx_quantize_grouped(x, offsets, mxq.E4M3, **s)),
        ("dequantize", lambda **s: mxq.mx_dequantize(codes, scales, 256, mxq.E4M3, **s)),
        ("quantize_nvfp4", lambda **s: mxq.mx_quantize_nvfp4(x, gs, **s)),
        ("qdq_nvfp4", lambda **s: mxq.mx_qdq_nvfp4(x, gs, **s)),
        ("quantize_nvfp4_grouped", lambda **s: mxq.mx_quantize_nvfp4_grouped(x, offsets, gs, **s)),
        ("dequantize_nvfp4", lambda **s: mxq.mx_dequantize_nvfp4(
            on_device(128, 128, dtype=u8), on_device(128, 16, dtype=u8), 256, gs, **s)),
        ("rotate_debug", lambda **s: mxq.mx_rotate_debug(x, H, **s)),
        ("gemm", lambda **s: mxq.mx_gemm(codes, scales, codes, scales, 256, mxq.E4M3, **s)),
        ("route", lambda **s: mxq.mx_route(logits, 2, **s)),
        ("route_backward", lambda **s: mxq.mx_route_backward(weights, logits, experts, **s)),
        ("route_plan", lambda **s: mxq.mx_route_plan(experts, 8, **s)),
        ("b128_rows", lambda **s: mxq.mx_quantize_b128_rows(x, **s)),
        ("b128_cols", lambda **s: mxq.mx_quantize_b128_cols(x, **s)),
        ("b128_blocks", lambda **s: mxq.mx_quantize_b128_blocks(x, transpose=True, **s)),
        ("gemm_b128", lambda **s: mxq.mx_gemm_b128(*rows, *blocks, **s)),
        ("gemm_b128_grouped", lambda **s: mxq.mx_gemm_b128_grouped(
            *rows, blocks[0][None], blocks[1][None], offsets, **s)),
        ("gemm_b128_grouped_wgrad", lambda **s: mxq.mx_gemm_b128_grouped_wgrad(
            *rows, *rows, offsets, **s)),
        ("combine", lambda **s: mxq.mx_combine(y, slots, **s)),
        ("combine_backward", lambda **s: mxq.mx_combine_backward(dout, y, slots, weights, **s)),
    ]


# shapes whose queries the accepting library answers with nothing are asked of these
SHAPES = {"mx_scales_shape": (128, 8), "mx_grouped_scales_shape": (128, 8),
          "mx_nvfp4_scales_shape": (128, 16), "mx_nvfp4_grouped_scales_shape": (128, 16),
          "mx_b128_padded_rows": 128}


@pytest.mark.parametrize("i", range(22))
def test_outputs_are_of_the_stream_they_are_written_on(noted, monkeypatch, i):
    for query, shape in SHAPES.items():
        monkeypatch.setattr(mxq, query, lambda *a, shape=shape, **k: shape)
    every = calls()
    assert len(every) == 22
    name, call = every[i]
    noted["taken"].clear()
    call(stream=SIDE)
    taken = noted["taken"]
    assert taken and all(stream == SIDE for stream, _ in taken), name
    # the caller's stream is recorded on each output (a workspace is not the caller's)
    outputs = len(taken) - (name in ("route_plan", "combine_backward"))
    assert noted["recorded"] == ["current"] * outputs
    noted["taken"].clear()
    call()
    assert [stream for stream, _ in noted["taken"]] == ["current"] * len(taken)
