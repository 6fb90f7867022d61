"""Give-ups of the layer norm's kernels: the limit reaches them, and a wait that runs out costs the call no time beyond
what it had asked for, whichever threads it runs out for."""

import time

import pytest
import torch

import __graft_entry__
import mx_microscaling_quantize_gb300 as mxq
from test_gpu_train import BF16, rows
from test_gpu_train_edges import same

pytestmark = pytest.mark.gpu

# Rows that all go by kernels that wait for them (more than 8 a multiprocessor). A call takes about 0.1 ms, copies that
# are on their way land within as long; a wait for one that never lands takes the 2 s of the last wait before the end.
SHAPES = [(3000, 8192), (5000, 1024), (3000, 16384), (9000, 256), (4000, 1056)]
SOON = 0.5  # s


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    yield
    assert mxq.mx_device_errors() == 0


def calls(M, K):
    """(a call with limited waits, the call, what it gives) of each kernel."""
    x, dy = rows(M, M, K, BF16), rows(M + 1, M, K, BF16, 0.0)
    _, mean, rstd = mxq.mx_layer_norm(x, stats=True)
    kept, kept_scales = mxq.mx_quantize_b128_rows(x)
    out = [(lambda ns: mxq.mx_selftest_layer_norm_give_up(x, ns), lambda: mxq.mx_layer_norm(x)),
           (lambda ns: mxq.mx_selftest_layer_norm_backward_give_up(dy, x, mean, rstd, ns),
            lambda: mxq.mx_layer_norm_backward(dy, x, mean, rstd)[0]),
           (lambda ns: mxq.mx_selftest_layer_norm_backward_give_up(dy, kept, mean, rstd, ns, x_scales=kept_scales),
            lambda: mxq.mx_layer_norm_backward(dy, kept, mean, rstd, x_scales=kept_scales)[0])]
    return [(give_up, call, call()) for give_up, call in out]


@pytest.mark.parametrize("M,K", SHAPES)
def test_a_limit_of_1_ns_is_a_give_up(M, K):
    """Rows from memory take hundreds of ns: with nothing of them in the caches some wait is too short. Not in every
    call: a row that has landed before it is waited for is no give-up, and the GPU's clock, by which a limit is
    measured, goes in steps that are longer than a wait of the shortest rows. One call of ten and more does at every
    size here, so that 200 of them without are less likely than 1e-9."""
    beside = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")  # twice the L2

    def gives_up(call):
        beside.fill_(1)
        torch.cuda.synchronize()
        assert mxq.mx_device_errors() == 0
        call(1)
        return mxq.mx_device_errors() == 1
    for give_up, call, want in calls(M, K):
        assert any(gives_up(give_up) for _ in range(200))
        assert same(call(), want) and mxq.mx_device_errors() == 0


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("limit", [1, 100, 500, 1000, 2000, 5000, 20000, 100000])
def test_a_give_up_ends_soon(M, K, limit):
    """Limits about the time that a row takes, so that waits run out for some threads of a group and not for others."""
    for give_up, call, want in calls(M, K):
        give_up(limit)  # what is made once, outside of the time
        for _ in range(10):
            torch.cuda.synchronize()
            start = time.perf_counter()
            give_up(limit)
            torch.cuda.synchronize()
            assert time.perf_counter() - start < SOON
        mxq.mx_device_errors()
        assert same(call(), want) and mxq.mx_device_errors() == 0
