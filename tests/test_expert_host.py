"""Host-side checks of the expert-layer entry points: arguments are refused before any launch, empty
calls launch nothing. No call here reaches a kernel, so fake pointers are never dereferenced."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import expert_ref as R
import mx_microscaling_quantize_gb300 as mxq
from mx_microscaling_quantize_gb300 import _build

OK, NULL, SHAPE, ALIGN, UNSUP = 0, 1, 2, 3, 4
P = 1 << 20  # a fake device address, never dereferenced
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mxq.h")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mxq.lib()


def test_macros_match_binding():
    macros = dict(re.findall(r"#define (MX_\w+) (\d+)", open(HEADER).read()))
    assert int(macros["MX_SCORE_SOFTMAX"]) == mxq.SOFTMAX
    assert int(macros["MX_SCORE_SIGMOID"]) == mxq.SIGMOID
    assert int(macros["MX_B128_BLOCKS"]) == mxq.B128_BLOCKS
    assert int(macros["MX_B128_ROWS"]) == mxq.B128_ROWS
    assert int(macros["MX_TYPE_BF16"]) == mxq._TYPES[torch.bfloat16]
    assert int(macros["MX_TYPE_FP32"]) == mxq._TYPES[torch.float32]


def test_route(L):
    # (logits, type, bias, T, E, k, score, groups, top_groups, renorm, scale, experts, weights, stream)
    def f(logits=P, ty=1, bias=None, T=4, E=8, k=2, score=0, g=1, tg=1, experts=P, weights=P):
        return L.mx_route(logits, ty, bias, T, E, k, score, g, tg, 1, 1.0, experts, weights, None)
    assert f(T=-1) == SHAPE and f(E=0) == SHAPE and f(E=1025, k=2) == SHAPE
    assert f(k=0) == SHAPE and f(k=9) == SHAPE and f(E=64, k=33) == SHAPE
    assert f(T=1 << 31, k=1) == SHAPE and f(T=1 << 30, k=4) == SHAPE
    assert f(ty=2) == UNSUP and f(score=2) == UNSUP
    assert f(g=0) == SHAPE and f(g=3) == SHAPE and f(E=66, g=33) == SHAPE
    assert f(g=4, tg=0) == SHAPE and f(g=4, tg=5) == SHAPE and f(g=4, tg=1, k=3) == SHAPE
    assert f(logits=None) == NULL and f(experts=None) == NULL and f(weights=None) == NULL
    assert f(logits=P + 2) == ALIGN and f(logits=P + 1, ty=0) == ALIGN and f(bias=P + 2) == ALIGN
    assert f(experts=P + 2) == ALIGN and f(weights=P + 1) == ALIGN
    assert f(T=0, logits=None, experts=None, weights=None) == OK


def test_route_backward(L):
    # (grad, logits, type, experts, T, E, k, score, renorm, scale, grad_logits, stream)
    def f(g=P, l=P, ty=1, e=P, T=4, E=8, k=2, score=0, out=P):
        return L.mx_route_backward(g, l, ty, e, T, E, k, score, 1, 1.0, out, None)
    assert f(T=-1) == SHAPE and f(k=9) == SHAPE and f(ty=3) == UNSUP and f(score=-1) == UNSUP
    for name in ("g", "l", "e", "out"):
        assert f(**{name: None}) == NULL and f(**{name: P + 1}) == ALIGN
    assert f(T=0, g=None, l=None, e=None, out=None) == OK


def test_route_plan(L):
    n = ctypes.c_int64()
    assert L.mx_route_plan_workspace(4, 2, 8, None) == NULL
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 2, 0), (4, 2, 1025), (1 << 31, 1, 8)):
        assert L.mx_route_plan_workspace(*bad, ctypes.byref(n)) == SHAPE
    assert mxq.mx_route_plan_workspace(4, 2, 8) == 0
    big = mxq.mx_route_plan_workspace(1 << 20, 8, 256)
    assert 0 < big <= 512 * 256 * 4
    f = L.mx_route_plan  # (experts, T, k, E, offsets, tokens, slots, workspace, stream)
    assert f(None, 4, 2, 8, P, P, P, None, None) == NULL
    assert f(P, 4, 2, 8, None, P, P, None, None) == NULL
    assert f(P, 4, 2, 8, P, None, P, None, None) == NULL
    assert f(P, 4, 2, 8, P, P, None, None, None) == NULL
    assert f(P, 1 << 20, 8, 256, P, P, P, None, None) == NULL  # needs its workspace
    assert f(P, 4, 2, 8, P + 4, P, P, None, None) == ALIGN
    assert f(P + 2, 4, 2, 8, P, P, P, None, None) == ALIGN
    assert f(P, 4, 2, 1025, P, P, P, None, None) == SHAPE


def test_b128_quantize(L):
    assert mxq.mx_b128_padded_rows(0, 1) == 0 and mxq.mx_b128_padded_rows(1, 1) == 128
    assert mxq.mx_b128_padded_rows(128, 1) == 128 and mxq.mx_b128_padded_rows(300, 4) == 768
    counts = [1] * 127 + [16384 - 127]  # the bound holds for any split
    assert sum(R.up(c) for c in counts) <= mxq.mx_b128_padded_rows(16384, 128)
    n = ctypes.c_int64()
    assert L.mx_b128_padded_rows(-1, 1, ctypes.byref(n)) == SHAPE
    assert L.mx_b128_padded_rows(1, 0, ctypes.byref(n)) == SHAPE
    assert L.mx_b128_padded_rows(1, 1, None) == NULL
    r = L.mx_quantize_b128_rows  # (x, M, K, index, R, codes, scales, stream)
    assert r(P, -1, 64, None, -1, P, P, None) == SHAPE and r(P, 4, 48, None, 4, P, P, None) == SHAPE
    assert r(P, 4, 64, None, 5, P, P, None) == SHAPE and r(P, 4, 64, P, -2, P, P, None) == SHAPE
    assert r(P, 1 << 31, 64, None, 1 << 31, P, P, None) == SHAPE
    assert r(None, 4, 64, None, 4, P, P, None) == NULL and r(P, 4, 64, None, 4, None, P, None) == NULL
    assert r(P, 4, 64, None, 4, P, None, None) == NULL
    assert r(P + 16, 4, 64, None, 4, P, P, None) == ALIGN
    assert r(P, 4, 64, None, 4, P + 16, P, None) == ALIGN
    assert r(P, 4, 64, P + 2, 4, P, P, None) == ALIGN and r(P, 4, 64, None, 4, P, P + 2, None) == ALIGN
    assert r(None, 0, 64, None, 0, None, None, None) == OK
    assert r(None, 4, 0, None, 4, None, None, None) == OK
    c = L.mx_quantize_b128_cols  # (x, M, K, index, R, offsets, E, codes, scales, stream)
    assert c(P, 4, 48, None, 4, None, 1, P, P, None) == SHAPE
    assert c(P, 4, 64, None, 4, None, 2, P, P, None) == SHAPE  # experts without offsets
    assert c(P, 4, 64, None, 4, P, 1025, P, P, None) == SHAPE
    assert c(P, 4, 64, None, 4, P + 4, 2, P, P, None) == ALIGN
    assert c(None, 4, 64, None, 4, None, 1, P, P, None) == NULL
    assert c(None, 0, 64, None, 0, None, 1, None, None, None) == OK
    b = L.mx_quantize_b128_blocks  # (x, batch, M, K, codes, scales, codes_t, scales_t, stream)
    assert b(P, -1, 4, 64, P, P, None, None, None) == SHAPE
    assert b(P, 65536, 4, 64, P, P, None, None, None) == SHAPE
    assert b(P, 1, 4, 40, P, P, None, None, None) == SHAPE
    assert b(P, 1, 4, 64, P, P, P, None, None) == NULL and b(P, 1, 4, 64, P, None, None, None, None) == NULL
    assert b(P, 1, 4, 64, P, P, P + 16, P, None) == ALIGN
    assert b(None, 0, 4, 64, None, None, None, None, None) == OK


def test_b128_products(L):
    # (a, sa, b, sb, M, N, K, b_form, c_type, c, stream)
    def f(a=P, sa=P, b=P, sb=P, M=128, N=128, K=128, form=0, ty=0, c=P):
        return L.mx_gemm_b128(a, sa, b, sb, M, N, K, form, ty, c, None)
    assert f(K=0) == SHAPE and f(K=48) == SHAPE and f(N=100) == SHAPE and f(M=-1) == SHAPE
    assert f(M=1 << 31) == SHAPE and f(M=1 << 30, N=1 << 20) == SHAPE
    assert f(form=2) == UNSUP and f(ty=2) == UNSUP
    for name in ("a", "sa", "b", "sb", "c"):
        assert f(**{name: None}) == NULL
    for name in ("a", "b", "c"):
        assert f(**{name: P + 8}) == ALIGN
    assert f(sa=P + 2) == ALIGN and f(sb=P + 1) == ALIGN
    assert f(M=0, a=None, c=None) == OK and f(N=0, b=None, c=None) == OK
    # (a, sa, b, sb, offsets, E, M, N, K, c_type, c, stream)
    def g(off=P, E=4, M=128, N=128, K=128, ty=0, c=P, a=P):
        return L.mx_gemm_b128_grouped(a, P, P, P, off, E, M, N, K, ty, c, None)
    assert g(E=0) == SHAPE and g(E=1025) == SHAPE and g(K=40) == SHAPE and g(N=4) == SHAPE
    assert g(E=1024, N=1 << 22) == SHAPE and g(K=0) == SHAPE and g(ty=5) == UNSUP
    assert g(off=None) == NULL and g(off=P + 4) == ALIGN and g(a=None) == NULL and g(c=P + 8) == ALIGN
    assert g(M=0, off=None, a=None, c=None) == OK
    # (a, sa, b, sb, offsets, E, M, N, R_padded, c_type, c, stream)
    def w(off=P, E=4, M=128, N=128, R=128, ty=1, c=P, a=P):
        return L.mx_gemm_b128_grouped_wgrad(a, P, P, P, off, E, M, N, R, ty, c, None)
    assert w(R=64) == SHAPE and w(E=0) == SHAPE and w(N=12) == SHAPE and w(R=-128) == SHAPE
    assert w(off=None) == NULL and w(off=P + 1) == ALIGN and w(a=None) == NULL
    assert w(R=0, c=None) == NULL and w(M=0, c=None) == OK
    s = L.mx_selftest_gemm_b128_give_up  # (a, sa, b, sb, M, N, K, form, c, limit, stream)
    assert s(P, P, P, P, 128, 128, 128, 0, P, 0, None) == SHAPE
    assert s(P, P, P, P, 128, 128, 128, 0, P, 100_000_001, None) == SHAPE
    assert s(P, P, P, P, 0, 128, 128, 0, P, 1000, None) == SHAPE


def test_combine(L):
    # (y, slots, weights, T, k, R, N, out, stream)
    def f(y=P, s=P, w=P, T=4, k=2, R=8, N=64, out=P):
        return L.mx_combine(y, s, w, T, k, R, N, out, None)
    assert f(T=-1) == SHAPE and f(k=0) == SHAPE and f(k=65) == SHAPE and f(N=12) == SHAPE
    assert f(R=-1) == SHAPE and f(T=1 << 30, k=2) == SHAPE
    assert f(y=None) == NULL and f(s=None) == NULL and f(out=None) == NULL
    assert f(y=P + 8) == ALIGN and f(out=P + 8) == ALIGN and f(s=P + 2) == ALIGN and f(w=P + 2) == ALIGN
    assert f(T=0, y=None, s=None, out=None) == OK and f(N=0, y=None, s=None, out=None) == OK
    # (dout, y, slots, weights, T, k, R, N, dy, dweights, stream)
    def b(d=P, y=P, s=P, w=P, T=4, k=2, R=8, N=64, dy=P, dw=P):
        return L.mx_combine_backward(d, y, s, w, T, k, R, N, dy, dw, None)
    assert b(k=0) == SHAPE and b(N=4) == SHAPE
    assert b(d=None) == NULL and b(y=None) == NULL and b(s=None) == NULL and b(dy=None) == NULL
    assert b(d=P + 8) == ALIGN and b(dy=P + 2) == ALIGN and b(dw=P + 2) == ALIGN
    assert b(T=0, d=None, s=None, dy=None, dw=None) == OK


def test_binding_refuses_cpu_tensors():
    with pytest.raises(TypeError):
        mxq.mx_route(torch.zeros(2, 4), 1)
    with pytest.raises(TypeError):
        mxq.mx_quantize_b128_rows(torch.zeros(2, 32, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        mxq.mx_combine(torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32))


# the reference itself, against hand-worked values
def test_reference_quantize():
    x = np.zeros((1, 256), np.float32)
    x[0, :3] = [448.0, -1.0, 17.0]  # 17 lies halfway between 16 and 18: to the even code, 16
    codes, s = R.quantize(x, 1, 128)
    assert s.tolist() == [[1.0, np.float32(2.0 ** -100) / np.float32(448)]]
    assert R.decode(codes)[0, :4].tolist() == [448.0, -1.0, 16.0, 0.0]
    assert R.encode(np.array([500.0, np.nan, 0.0009765625, -0.0], np.float32)).tolist() == \
        [0x7E, 0x7F, 0x00, 0x80]  # saturates; NaN; half the least value goes to even; sign of zero


def test_reference_route_and_plan():
    l = np.array([[0.0, 2.0, 1.0, 2.0], [-np.inf] * 4])
    e, w = R.route(l, 3, "softmax", renorm=False)
    assert e.tolist() == [[1, 3, 2], [-1, -1, -1]] and (w[1] == 0).all()
    p = np.exp(l[0]) / np.exp(l[0]).sum()
    assert np.allclose(w[0], p[[1, 3, 2]])
    offsets, tokens, slots = R.plan(np.array([[2, 0], [0, -1]], np.int32), 3)
    assert offsets.tolist() == [0, 2, 2, 3] and tokens.tolist() == [0, 1, 0, -1]
    assert slots.tolist() == [[2, 0], [1, -1]]
