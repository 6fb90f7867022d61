"""Host-side checks that go with test_gpu_expert_edges.py: refusals before any launch (fake pointers are
never dereferenced)."""

import os
import re

import pytest

import mx_microscaling_quantize_gb300 as mxq
from mx_microscaling_quantize_gb300 import _build

OK, NULL, SHAPE, ALIGN = 0, 1, 2, 3
P = 1 << 20


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mxq.lib()


def test_combine_backward_whole(L):
    # (dout, y, slots, weights, T, k, R, N, dy, dweights, workspace, stream)
    def f(d=P, y=P, s=P, w=P, T=4, k=2, R=8, N=64, dy=P, dw=P, ws=P):
        return L.mx_combine_backward_whole(d, y, s, w, T, k, R, N, dy, dw, ws, None)
    assert f(k=0) == SHAPE and f(N=4) == SHAPE and f(R=-1) == SHAPE and f(T=-1) == SHAPE
    for name in ("d", "y", "s", "dy", "ws"):
        assert f(**{name: None}) == NULL
    assert f(T=0, dy=None) == NULL and f(T=0, ws=None) == NULL  # rows are still zeroed
    assert f(d=P + 8) == ALIGN and f(dy=P + 2) == ALIGN and f(dw=P + 2) == ALIGN and f(ws=P + 2) == ALIGN
    assert f(T=0, R=0, d=None, y=None, s=None, dy=None, dw=None, ws=None) == OK


def test_kernels_read_their_inputs_through_the_coherent_loads():
    """A kernel's arrays are read by the load functions (asm volatile, after the wait for the kernel before)
    and never by subscript, which the compiler may turn into a non-coherent or an earlier load."""
    csrc = os.path.join(os.path.dirname(mxq.__file__), "csrc")
    for name in ("mx_route.cu", "mx_b128_quant.cu", "mx_b128_gemm.cu", "mx_combine.cu"):
        for number, line in enumerate(open(os.path.join(csrc, name)), 1):
            line = line.split("//")[0]
            for use in re.finditer(r"\ba\.\w+\[", line):
                # what is written: the subscript's end is followed by an assignment
                assert re.match(r"[^=]*\] = ", line[use.end():]), f"{name}:{number}: {line.strip()}"


def test_grouped_give_up(L):
    # (a, sa, b, sb, offsets, E, M, N, K, c, limit, stream)
    def f(limit=1000, M=128, off=P, c=P, E=4):
        return L.mx_selftest_gemm_b128_grouped_give_up(P, P, P, P, off, E, M, 128, 128, c, limit, None)
    assert f(limit=0) == SHAPE and f(limit=100_000_001) == SHAPE and f(M=0) == SHAPE and f(E=0) == SHAPE
    assert f(off=None) == NULL and f(c=None) == NULL and f(c=P + 8) == ALIGN


def test_no_rows_need_no_index(L):
    """An empty index has no address: without rows there is nothing that it could name."""
    r = L.mx_quantize_b128_rows  # (x, M, K, index, R, codes, scales, stream)
    assert r(P, 4, 64, None, 0, None, None, None) == OK
    assert r(P, 4, 64, None, 3, P, P, None) == SHAPE
    c = L.mx_quantize_b128_cols  # (x, M, K, index, R, offsets, E, codes, scales, stream)
    assert c(P, 4, 64, None, 0, None, 1, None, None, None) == OK
    assert c(P, 4, 64, None, 3, P, 2, P, P, None) == SHAPE
