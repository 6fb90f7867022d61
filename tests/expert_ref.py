"""Plain 64-bit definitions of the expert-layer operators, on the CPU with numpy and torch; nothing
here uses the library. E4M3 codes are compared bit for bit (the definition fixes every fp32 step),
everything else within bounds that the tests derive from the arithmetic."""

from __future__ import annotations

import numpy as np
import torch

BLK = 128
FLOOR = np.float32(2.0 ** -100)
U = 2.0 ** -24  # unit roundoff of fp32


def up(n: int) -> int:
    return -(-n // BLK) * BLK


# ---------------------------------------------------------------------------------------------
# operands with a scale per block of 128
# ---------------------------------------------------------------------------------------------
def f32(x: torch.Tensor) -> np.ndarray:
    return x.detach().cpu().float().numpy()


def encode(t: np.ndarray) -> np.ndarray:
    """E4M3 bytes of fp32 values: nearest even, saturating, 0x7F for NaN."""
    v = torch.from_numpy(np.ascontiguousarray(np.clip(t, -448, 448)))
    b = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
    b[np.isnan(t)] = 0x7F
    return b


def decode(codes: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def factors(amax: np.ndarray):
    a = np.maximum(amax.astype(np.float32), FLOOR)
    with np.errstate(invalid="ignore", over="ignore"):
        r, s = np.float32(448) / a, a / np.float32(448)
    bad = ~np.isfinite(amax)
    r[bad] = s[bad] = np.nan
    return r, s


def blocks_of(v: np.ndarray, br: int, bc: int):
    """v [R, C] padded with zeros to whole br x bc blocks -> [R/br, br, C/bc, bc]."""
    R, C = -(-v.shape[0] // br) * br, -(-v.shape[1] // bc) * bc
    p = np.zeros((R, C), np.float32)
    p[:v.shape[0], :v.shape[1]] = v
    return p.reshape(R // br, br, C // bc, bc)


def quantize(v: np.ndarray, br: int, bc: int):
    """-> codes like v, scales [rows of blocks, columns of blocks]."""
    b = blocks_of(v, br, bc)
    with np.errstate(invalid="ignore", over="ignore"):
        # max propagates NaN in numpy
        r, s = factors(np.abs(b).max((1, 3)))
        codes = encode(b * r[:, None, :, None]).reshape(b.shape[0] * br, b.shape[2] * bc)
    return codes[:v.shape[0], :v.shape[1]], s


def rows(x: torch.Tensor, index=None):
    v = f32(x)
    if index is not None:
        ok = (index >= 0) & (index < v.shape[0])
        v = np.where(ok[:, None], v[np.clip(index, 0, max(v.shape[0] - 1, 0))], np.float32(0))
    codes, s = quantize(v, 1, BLK)
    return codes, np.ascontiguousarray(s.T)


def cols(x: torch.Tensor, index=None, offsets=None):
    """codes [K, P'], scales [P' / 128, K] up to the end P' of the last expert's blocks."""
    v = f32(x)
    if index is not None:
        ok = (index >= 0) & (index < v.shape[0])
        v = np.where(ok[:, None], v[np.clip(index, 0, max(v.shape[0] - 1, 0))], np.float32(0))
    offsets = [0, v.shape[0]] if offsets is None else list(offsets)
    parts = []
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        p = np.zeros((up(hi - lo), v.shape[1]), np.float32)
        p[:hi - lo] = v[lo:hi]
        parts.append(p)
    codes, s = quantize(np.concatenate(parts), BLK, 1)
    return np.ascontiguousarray(codes.T), s


def values(codes, scales, form: str):
    """64-bit values: scales [K / 128, rows] ("rows") or [rows / 128, K / 128] ("blocks")."""
    s = scales.astype(np.float64)
    if form == "rows":
        s = np.repeat(s.T, BLK, 1)
    else:
        s = np.repeat(np.repeat(s, BLK, 0), BLK, 1)
    v = decode(codes)
    return v * s[:v.shape[0], :v.shape[1]]


def product(a: np.ndarray, b: np.ndarray):
    """-> C = a b^T and the sum of the magnitudes that bounds its error."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def product_bound(C, S, K: int, bf16: bool):
    """|C' - C| of a kernel that sums each block of 128 in fp32 (each of its additions errs by at
    most 2^-23 of a partial sum, at most S), multiplies it by a product of two scales (three
    roundings) and adds it in fp32; then one rounding to bf16 (2^-8 of the value)."""
    steps = -(-K // BLK)
    acc = (BLK + steps + 4) * 2 * U * S
    out = 2.0 ** -8 if bf16 else 2 * U
    return out * np.abs(C) + (1 + out) * acc + 1e-38


# ---------------------------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------------------------
def scores(l: np.ndarray, score: str):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    with np.errstate(invalid="ignore"):
        m = l.max(1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        e = np.exp(l - m)
        total = e.sum(1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1, total))


def route(l: np.ndarray, k: int, score="softmax", bias=None, groups=1, top=1, renorm=True,
          scale=1.0):
    """Finite, -inf and tied logits (l in 64 bits) -> experts, weights."""
    T, E = l.shape
    s = scores(l, score)
    c = l if bias is None and score == "softmax" else s if bias is None else s + bias
    excluded = np.isneginf(l) | np.isneginf(c)
    c = np.where(excluded, -np.inf, c)
    if groups > 1:
        cs = np.where(excluded, -np.inf, s if bias is None else s + bias)
        two = -np.sort(-cs.reshape(T, groups, -1), 2)[:, :, :2]
        g = two[:, :, 0].copy()
        if two.shape[2] > 1:
            g += np.where(np.isneginf(two[:, :, 1]), 0.0, two[:, :, 1])
        kept = np.argsort(-g, 1, kind="stable")[:, :top]
        keep = np.zeros((T, groups), bool)
        np.put_along_axis(keep, kept, True, 1)
        c = np.where(np.repeat(keep, E // groups, 1), c, -np.inf)
    order = np.argsort(-c, 1, kind="stable")[:, :k]
    made = ~np.isneginf(np.take_along_axis(c, order, 1))
    w = np.where(made, np.take_along_axis(s, order, 1), 0.0)
    if renorm:
        P = w.sum(1, keepdims=True)
        w = np.where(P == 0, 0.0, w / np.where(P == 0, 1, P))
    return np.where(made, order, -1).astype(np.int32), w * scale


def chosen_weights(l, experts, score, renorm, scale):
    """Weights of given choices, differentiable in l (torch, 64 bits)."""
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    made = experts >= 0
    w = torch.where(made, s.gather(1, experts.clamp_min(0).long()), torch.zeros((), dtype=l.dtype))
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return w * scale


def plan(experts: np.ndarray, E: int):
    T, k = experts.shape
    flat = experts.reshape(-1).astype(np.int64)
    flat = np.where((flat < 0) | (flat >= E), E, flat)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])])
    order = np.argsort(flat, kind="stable")
    made = int(offsets[-1])
    tokens = np.full(T * k, -1, np.int32)
    tokens[:made] = order[:made] // k
    slots = np.full(T * k, -1, np.int32)
    slots[order[:made]] = np.arange(made)
    return offsets.astype(np.int64), tokens, slots.reshape(T, k)
