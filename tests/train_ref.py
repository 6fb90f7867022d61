"""Plain 64-bit definitions of what stands between the products of an 8-bit training step (layer norm,
activation, checkpoints), with bounds on how far fp32 arithmetic may be from them; nothing here uses the
library. U is the unit roundoff of fp32."""

from __future__ import annotations

import math

import numpy as np
import torch

import expert_ref as R

U = 2.0 ** -24
# Depth of any fp32 sum over a row of at most 16384 values: at most 32 in a lane's chain, 5 steps in a
# warp, 16 warps, and the roundings of the terms: below 64.
DEPTH = 64


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def checkpoint(x: torch.Tensor):
    """codes, scales and the fp32 values that they stand for."""
    codes, scales = R.quantize(R.f32(x), 1, R.BLK)
    return codes, np.ascontiguousarray(scales.T), values(codes, scales.T)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp32 values of rows' codes [M, K] under scales [K / 128, M]."""
    per = np.repeat(scales.T, R.BLK, 1)[:, :codes.shape[1]]
    with np.errstate(invalid="ignore"):
        return (R.decode(codes).astype(np.float32) * per).astype(np.float32)


# ---------------------------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------------------------
def norm(x, w, b, eps, center):
    """-> y, mean, rstd and the bound of y before it is rounded. x, w, b: float64."""
    K = x.shape[1]
    w = np.ones(K) if w is None else w
    b = np.zeros(K) if b is None else b
    mean = x.mean(1) if center else np.zeros(x.shape[0])
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + np.float64(np.float32(eps)))
    y = d * rstd[:, None] * w
    # mean: DEPTH roundings of sums of |x|. d carries that and its own; the variance (and rstd) the
    # roundings of its sum and, times d / rstd, the mean's error again.
    size = np.abs(x).mean(1)[:, None] if center else np.zeros((x.shape[0], 1))
    tol = DEPTH * U * (np.abs(w) * rstd[:, None] * (size + np.abs(d)) +
                       np.abs(y) * (1 + rstd[:, None] * size) + np.abs(b))
    return y + b, mean, rstd, tol


def norm_backward(dy, x, mean, rstd, w, center, checkpoint=False):
    """-> dx, dw, db and the bounds of each before rounding. mean, rstd: what the kernel was given.

    checkpoint: x is of products code * scale, rounded here, that the kernel may fold into xhat =
    fma(code, scale * rstd, -(mean * rstd)) and (code, scale * c, -mean c + ..) in dx, c = s2 rstd^2: beside the
    rounding of x (U |x|) those of scale * rstd, of mean * rstd and of their sum, each at most U (|x| + |mean|)
    rstd, so that xhat is off by at most 4 U (|x| + |mean|) rstd more."""
    M, K = x.shape
    w = np.ones(K) if w is None else w
    mean = np.zeros(M) if mean is None else mean
    r = rstd[:, None]
    xh = (x - mean[:, None]) * r
    g = dy * w
    s1 = g.mean(1, keepdims=True) if center else np.zeros((M, 1))
    s2 = (g * xh).mean(1, keepdims=True)
    dx = r * (g - s1 - xh * s2)
    a1 = np.abs(g).mean(1, keepdims=True) if center else 0.0
    a2 = np.abs(g * xh).mean(1, keepdims=True)
    tol = DEPTH * U * r * (np.abs(g) + a1 + np.abs(xh) * a2)
    rows = (M + DEPTH) * U
    tol_w = rows * np.abs(dy * xh).sum(0)
    if checkpoint:  # what xhat is off by more, in its own place, in s2 and in the weight's gradient
        off = 4 * U * (np.abs(x) + np.abs(mean)[:, None]) * r
        tol = tol + r * (off * np.abs(s2) + np.abs(xh) * (np.abs(g) * off).mean(1, keepdims=True))
        tol_w = tol_w + (np.abs(dy) * off).sum(0)
    return dx, (dy * xh).sum(0), dy.sum(0), tol, tol_w, rows * np.abs(dy).sum(0)


# ---------------------------------------------------------------------------------------------
# activation
# ---------------------------------------------------------------------------------------------
def act(kind: str, g: np.ndarray):
    """-> f(g), f'(g) and bounds of the two in fp32.

    The fast exponential is within 2 + 1.173 |x| ulp, the fast quotient within 2 ulp, erfc within 4 ulp
    (an ulp is at most 2^-23 relative); an argument off by d relative moves an exponential of z by |z| d,
    erfc(z) by 2 z^2 d. Beyond fp32's exponents the logistic function is 0 where it is below 2^-126."""
    from scipy.special import expit, ndtr

    e = 2.0 ** -23
    if kind == "silu":
        s, q = expit(g), expit(-g)
        h = g * s
        d = s + h * q
        rel = e * (16 + 4 * np.abs(g))
        return h, d, rel * np.abs(h) + np.abs(g) * 2.0 ** -125, rel * (s + np.abs(h) * q) + np.abs(g) * 2.0 ** -125
    if kind == "gelu":
        p = ndtr(g)
        phi = np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        rel = e * (16 + 4 * g * g)
        return g * p, p + g * phi, rel * np.abs(g * p) + np.abs(g) * 2.0 ** -125, \
            rel * (p + np.abs(g) * phi) + np.abs(g) * 2.0 ** -125
    c = math.sqrt(8 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    s, q = expit(z), expit(-z)
    k = c * (1 + 3 * 0.044715 * g * g)
    h = g * s
    rel = e * (24 + 8 * np.abs(z))
    # (below, q s is at most 1 / 4 and |z| e^-|z| bounded, but k grows with g^2)
    return h, s + h * q * k, rel * np.abs(h) + np.abs(g) * 2.0 ** -125, \
        rel * (s + np.abs(h) * q * k) + np.abs(g) * (1 + k) * 2.0 ** -125


# ---------------------------------------------------------------------------------------------
# comparisons
# ---------------------------------------------------------------------------------------------
def check_values(got, want, tol, dtype, what=""):
    """Within tol before a rounding to dtype, half a step after it (and below its least normal, half of
    its least subnormal step, which is under 2^-133 for bf16 and fp32)."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    err = np.abs(got - want)
    bound = tol + half_step(dtype) * (np.abs(want) + tol) + 2.0 ** -133
    assert (err <= bound).all(), (what, float((err / bound).max()), int((err > bound).sum()))


def step_of(t: np.ndarray) -> np.ndarray:
    """Distance of neighbouring E4M3 values at |t| (saturated at 448)."""
    _, e = np.frexp(np.minimum(np.abs(t), 448.0))
    return 2.0 ** (np.maximum(e, -5) - 4.0)


def check_codes(codes, scales, want, tol, what=""):
    """Codes [M, K] and scales [ceil(K / 128), M] of values that are within tol of want (float64) before
    the quantisation: the scale follows the largest value, a code is the nearest to value * 448 / a for
    some such value and a within its bound."""
    codes, scales = codes.cpu().numpy(), f64(scales)
    M, K = want.shape
    B = -(-K // R.BLK)
    def block(v):
        p = np.zeros((M, B * R.BLK))
        p[:, :K] = v
        return p.reshape(M, B, R.BLK)
    a = np.maximum(np.abs(block(want)).max(2), 2.0 ** -100)
    da = block(tol).max(2)
    assert scales.shape == (B, M), what
    err = np.abs(scales.T * 448 - a)
    bound = da + 3 * U * (a + da)
    assert (err <= bound).all(), (what, "scales", float((err / bound).max()))
    t = want * np.repeat(448 / a, R.BLK, 1)[:, :K]
    rel = np.repeat(bound / a + 4 * U, R.BLK, 1)[:, :K]
    dt = tol * np.repeat(448 / a, R.BLK, 1)[:, :K] + np.abs(t) * rel
    v = R.decode(codes)
    t = np.clip(t, -448, 448)
    err = np.abs(v - t)
    bound = step_of(np.abs(t) + dt) / 2 + dt
    assert (err <= bound).all(), (what, "codes", float((err / bound).max()), int((err > bound).sum()))
    # and none is off where the value is clear of every midpoint: the nearest grid value of t itself
    near = R.decode(R.encode(t.astype(np.float32)))
    clear = (step_of(t) / 2 - np.abs(t - near) > dt + 4 * U * np.abs(t)) & (step_of(t) == step_of(np.abs(t) + dt))
    assert (v[clear] == near[clear]).all(), what
