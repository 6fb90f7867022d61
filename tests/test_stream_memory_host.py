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
    for cached in (mxq.mx_route_plan_workspace, mxq.mx_b128_padded_rows):
        cached.cache_clear()
    yield state
    for cached in (mxq.mx_route_plan_workspace, mxq.mx_b128_padded_rows):
        cached.cache_clear()


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
