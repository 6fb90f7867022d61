"""Host-side checks of layer norm, activation and checkpoint entry points: arguments are refused before any
launch, empty calls launch nothing, and memory comes from the stream it is used on. No call here reaches a
kernel, so fake pointers are never dereferenced."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import expert_ref as R
import mx_microscaling_quantize_gb300 as mxq
import train_ref as T
from mx_microscaling_quantize_gb300 import _build
from test_stream_memory_host import SIDE, noted, on_device  # noqa: F401

OK, NULL, SHAPE, ALIGN, UNSUP = 0, 1, 2, 3, 4
P = 1 << 20  # a fake device address, never dereferenced
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mxq.h")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mxq.lib()


def test_macros_match_binding():
    macros = dict(re.findall(r"#define (MX_\w+) (\d+)", open(HEADER).read()))
    assert int(macros["MX_ACT_SILU"]) == mxq.SILU
    assert int(macros["MX_ACT_GELU"]) == mxq.GELU
    assert int(macros["MX_ACT_GELU_TANH"]) == mxq.GELU_TANH
    assert int(macros["MX_TYPE_E4M3_B128"]) == mxq._CHECKPOINT


def test_layer_norm(L):
    # (x, x_type, weight, bias, w_type, M, K, eps, center, y, y_type, mean, rstd, stream)
    def f(x=P, xt=0, w=P, b=P, wt=1, M=4, K=64, y=P, yt=0, mean=None, rstd=None):
        return L.mx_layer_norm(x, xt, w, b, wt, M, K, 1e-5, 1, y, yt, mean, rstd, None)
    assert f(M=-1) == SHAPE and f(K=-8) == SHAPE and f(K=16392) == SHAPE and f(M=1 << 31) == SHAPE
    assert f(xt=2) == UNSUP and f(wt=2) == UNSUP and f(yt=-1) == UNSUP
    assert f(x=None) == NULL and f(y=None) == NULL
    assert f(x=P + 1) == ALIGN and f(x=P + 2, xt=1) == ALIGN and f(y=P + 1) == ALIGN and f(y=P + 2, yt=1) == ALIGN
    assert f(w=P + 2) == ALIGN and f(b=P + 2) == ALIGN and f(w=P + 1, wt=0) == ALIGN
    assert f(mean=P + 2) == ALIGN and f(rstd=P + 1) == ALIGN
    assert f(M=0, x=None, y=None) == OK and f(K=0, x=None, y=None) == OK


def test_layer_norm_b128(L):
    # (x, x_type, weight, bias, w_type, M, K, eps, center, codes, scales, x_codes, x_scales, mean, rstd, stream)
    def f(x=P, xt=0, w=P, b=P, wt=1, M=4, K=64, c=P, s=P, xc=None, xs=None, mean=None, rstd=None):
        return L.mx_layer_norm_b128(x, xt, w, b, wt, M, K, 1e-5, 1, c, s, xc, xs, mean, rstd, None)
    assert f(K=40) == SHAPE and f(K=16416) == SHAPE and f(M=-1) == SHAPE
    assert f(xt=2) == UNSUP and f(wt=3) == UNSUP
    assert f(x=None) == NULL and f(c=None) == NULL and f(s=None) == NULL and f(xc=P) == NULL and f(xs=P) == NULL
    for name in ("x", "c", "w", "b"):
        assert f(**{name: P + 16}) == ALIGN
    assert f(s=P + 2) == ALIGN and f(xc=P + 16, xs=P) == ALIGN and f(xc=P, xs=P + 2) == ALIGN
    assert f(mean=P + 2) == ALIGN and f(rstd=P + 2) == ALIGN
    assert f(M=0, x=None, c=None, s=None) == OK and f(K=0, x=None, c=None, s=None) == OK


def test_layer_norm_backward(L):
    n = ctypes.c_int64()
    assert L.mx_layer_norm_backward_workspace(4, 64, None) == NULL
    for bad in ((-1, 64), (4, -1), (4, 16385)):
        assert L.mx_layer_norm_backward_workspace(*bad, ctypes.byref(n)) == SHAPE
    assert mxq.mx_layer_norm_backward_workspace(0, 64) == 0
    assert 0 < mxq.mx_layer_norm_backward_workspace(1 << 20, 8192) <= 64 << 20
    # (dy, dy_type, x, x_type, x_scales, mean, rstd, weight, w_type, M, K, dx, dx_type, dw, db, workspace, stream)

    def f(dy=P, dyt=0, x=P, xt=0, xs=None, mean=P, rstd=P, w=P, wt=1, M=4, K=64, dx=P, dxt=0, dw=P, db=P, ws=P):
        return L.mx_layer_norm_backward(dy, dyt, x, xt, xs, mean, rstd, w, wt, M, K, dx, dxt, dw, db, ws, None)
    assert f(M=-1) == SHAPE and f(K=16385) == SHAPE and f(xt=2, xs=P, K=40) == SHAPE
    assert f(dyt=2) == UNSUP and f(xt=3) == UNSUP and f(dxt=2) == UNSUP and f(wt=2) == UNSUP
    for name in ("dy", "x", "rstd", "dx", "ws"):
        assert f(**{name: None}) == NULL
    assert f(xt=2) == NULL  # no scales
    for name, by in (("dy", 1), ("x", 1), ("dx", 1), ("mean", 2), ("rstd", 2), ("w", 2), ("dw", 2), ("db", 1),
                     ("ws", 2)):
        assert f(**{name: P + by}) == ALIGN
    assert f(xt=2, xs=P + 2) == ALIGN
    assert f(K=0, dy=None, x=None, dx=None, rstd=None, ws=None) == OK
    assert f(M=0, dy=None, x=None, dx=None, rstd=None, dw=None, db=None, ws=None) == OK


def test_activation(L):
    # (u, R, H, kind, gated, codes, scales, u_codes, u_scales, stream)
    def f(u=P, R_=4, H=128, kind=0, gated=1, c=P, s=P, uc=None, us=None):
        return L.mx_activation_b128(u, R_, H, kind, gated, c, s, uc, us, None)
    assert f(R_=-1) == SHAPE and f(H=-32) == SHAPE and f(H=40) == SHAPE and f(H=(1 << 27) + 32) == SHAPE
    assert f(H=96, uc=P, us=P) == SHAPE  # blocks of gate and up would share a scale
    assert f(kind=3) == UNSUP and f(kind=-1) == UNSUP
    assert f(u=None) == NULL and f(c=None) == NULL and f(s=None) == NULL and f(uc=P) == NULL and f(us=P) == NULL
    assert f(u=P + 16) == ALIGN and f(c=P + 16) == ALIGN and f(s=P + 2) == ALIGN
    assert f(uc=P + 16, us=P) == ALIGN and f(uc=P, us=P + 1) == ALIGN
    assert f(R_=0, u=None, c=None, s=None) == OK and f(H=0, u=None, c=None, s=None) == OK


def test_activation_backward(L):
    # (dh, u, u_type, u_scales, R, H, kind, gated, du, du_codes, du_scales, stream)
    def f(dh=P, u=P, ut=0, us=None, R_=4, H=128, kind=0, gated=1, du=P, c=None, s=None):
        return L.mx_activation_backward(dh, u, ut, us, R_, H, kind, gated, du, c, s, None)
    assert f(ut=1) == UNSUP and f(ut=3) == UNSUP and f(kind=5) == UNSUP
    assert f(R_=-1) == SHAPE and f(H=33) == SHAPE
    assert f(H=96, ut=2, us=P) == SHAPE and f(H=96, c=P, s=P) == SHAPE
    assert f(dh=None) == NULL and f(u=None) == NULL and f(ut=2) == NULL
    assert f(du=None) == NULL and f(c=P) == NULL and f(s=P) == NULL  # nothing wanted; half an operand
    for name in ("dh", "u", "du"):
        assert f(**{name: P + 16}) == ALIGN
    assert f(ut=2, us=P + 2) == ALIGN and f(c=P + 16, s=P) == ALIGN and f(c=P, s=P + 2) == ALIGN
    assert f(R_=0, dh=None, u=None, du=None) == OK


def test_requantize_cols(L):
    # (codes, scales, M, K, index, R, row_offsets, E, out_codes, out_scales, stream)
    def f(c=P, s=P, M=4, K=64, i=None, R_=4, off=None, E=1, oc=P, os_=P):
        return L.mx_requantize_b128_cols(c, s, M, K, i, R_, off, E, oc, os_, None)
    assert f(M=-1) == SHAPE and f(K=40) == SHAPE and f(R_=5) == SHAPE and f(E=2) == SHAPE
    assert f(off=P, E=1025) == SHAPE and f(i=P, R_=-1) == SHAPE
    assert f(c=None) == NULL and f(s=None) == NULL and f(oc=None) == NULL and f(os_=None) == NULL
    assert f(c=P + 16) == ALIGN and f(s=P + 2) == ALIGN and f(oc=P + 16) == ALIGN and f(os_=P + 2) == ALIGN
    assert f(i=P + 2) == ALIGN and f(off=P + 4) == ALIGN
    assert f(M=0, R_=0, c=None, s=None, oc=None, os_=None) == OK and f(K=0, c=None) == OK


def test_dequantize(L):
    # (codes, scales, M, K, index, R, y, y_type, stream)
    def f(c=P, s=P, M=4, K=64, i=None, R_=4, y=P, yt=0):
        return L.mx_dequantize_b128_rows(c, s, M, K, i, R_, y, yt, None)
    assert f(M=-1) == SHAPE and f(K=40) == SHAPE and f(R_=5) == SHAPE and f(i=P, R_=-1) == SHAPE
    assert f(yt=2) == UNSUP
    assert f(c=None) == NULL and f(s=None) == NULL and f(y=None) == NULL
    assert f(c=P + 16) == ALIGN and f(s=P + 2) == ALIGN and f(y=P + 16) == ALIGN and f(i=P + 2) == ALIGN
    assert f(R_=0, M=0, c=None, s=None, y=None) == OK and f(K=0, c=None) == OK


def test_give_ups_want_a_launch(L):
    for limit, M, K in ((0, 4, 64), (100000001, 4, 64), (5, 0, 64), (5, 4, 0)):
        assert L.mx_selftest_layer_norm_give_up(P, M, K, P, limit, None) == SHAPE
        assert L.mx_selftest_layer_norm_backward_give_up(P, P, 0, None, P, P, M, K, P, limit, None) == SHAPE


# ---------------------------------------------------------------------------------------------
# the definitions themselves
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("center", [True, False])
def test_norm_backward_is_the_gradient_of_norm(center):
    rng = np.random.default_rng(3)
    x, w, dy = rng.standard_normal((4, 24)) + 2, 1 + 0.3 * rng.standard_normal(24), rng.standard_normal((4, 24))
    t = [torch.from_numpy(v).requires_grad_() for v in (x, w, np.zeros(24))]
    d = t[0] - t[0].mean(1, keepdim=True) if center else t[0]
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + float(np.float32(1e-5))) * t[1] + t[2]
    y.backward(torch.from_numpy(dy))
    got_y, mean, rstd, _ = T.norm(x, w, None, 1e-5, center)
    assert np.abs(got_y - y.detach().numpy()).max() < 1e-12
    dx, dw, db = T.norm_backward(dy, x, mean if center else None, rstd, w, center)[:3]
    for got, want in zip((dx, dw, db), t):
        assert np.abs(got - want.grad.numpy()).max() < 1e-12


def test_check_codes_notices_a_wrong_code_and_scale():
    rng = np.random.default_rng(4)
    v = rng.standard_normal((3, 256))
    codes, scales, _ = T.checkpoint(torch.from_numpy(v).float())
    v = v.astype(np.float32).astype(np.float64)
    none = np.zeros_like(v)
    c, s = torch.from_numpy(codes), torch.from_numpy(scales)
    T.check_codes(c, s, v, none)
    for at in ((0, 0), (2, 200)):
        bad = c.clone()
        bad[at] += 1
        with pytest.raises(AssertionError):
            T.check_codes(bad, s, v, none)
    bad = s.clone()
    bad[1, 2] *= 1 + 2.0 ** -20
    with pytest.raises(AssertionError):
        T.check_codes(c, bad, v, none)


# ---------------------------------------------------------------------------------------------
# memory of the stream it is used on
# ---------------------------------------------------------------------------------------------
def calls():
    bf16, u8 = torch.bfloat16, torch.uint8
    x, w, row = on_device(16, 256, dtype=bf16), on_device(256), on_device(16)
    kept = on_device(16, 256, dtype=u8), on_device(2, 16)
    dh = on_device(16, 128, dtype=bf16)
    return [
        # (a call with every output left to the binding, outputs, workspaces)
        (lambda **s: mxq.mx_layer_norm(x, w, w, stats=True, **s), 3, 0),
        (lambda **s: mxq.mx_layer_norm_b128(x, w, w, stats=True, checkpoint=True, **s), 6, 0),
        (lambda **s: mxq.mx_layer_norm_backward(x, x, row, row, w, **s), 3, 1),
        (lambda **s: mxq.mx_layer_norm_backward(x, kept[0], row, row, w, x_scales=kept[1], **s), 3, 1),
        (lambda **s: mxq.mx_activation_b128(x, checkpoint=True, **s), 4, 0),
        (lambda **s: mxq.mx_activation_backward(dh, x, operand=True, **s), 3, 0),
        (lambda **s: mxq.mx_requantize_b128_cols(*kept, **s), 2, 0),
        (lambda **s: mxq.mx_dequantize_b128_rows(*kept, **s), 1, 0),
        (lambda **s: mxq.mx_selftest_layer_norm_give_up(x, 1, **s), 1, 0),
        (lambda **s: mxq.mx_selftest_layer_norm_backward_give_up(x, x, row, row, 1, **s), 1, 0),
    ]


@pytest.mark.parametrize("i", range(10))
def test_memory_is_of_the_stream_it_is_used_on(noted, monkeypatch, i):  # noqa: F811
    monkeypatch.setattr(mxq, "mx_b128_padded_rows", lambda *a: 128)
    monkeypatch.setattr(mxq, "mx_layer_norm_backward_workspace", lambda *a: 4096)
    call, outputs, scratch = calls()[i]
    noted["taken"].clear()
    call(stream=SIDE)
    assert [stream for stream, _ in noted["taken"]] == [SIDE] * (outputs + scratch)
    assert noted["recorded"] == ["current"] * outputs  # a workspace is not the caller's
    noted["taken"].clear()
    call()
    assert [stream for stream, _ in noted["taken"]] == ["current"] * (outputs + scratch)


def test_quantise_of_the_reference_is_that_of_expert_layers():
    x = torch.from_numpy(np.random.default_rng(8).standard_normal((5, 300))).bfloat16()
    codes, scales, v = T.checkpoint(x)
    c, s = R.quantize(R.f32(x), 1, R.BLK)
    assert (codes == c).all() and (scales == s.T).all()
    assert np.abs(v - R.f32(x)).max() <= 2.0 ** -4 * np.abs(R.f32(x)).max()
