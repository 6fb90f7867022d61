"""Layer norm, activation and activation checkpoints on the GPU against their plain 64-bit definitions
(tests/train_ref.py). What the definition fixes step by step (checkpoints, the operands made of them) is
compared exactly, the rest within bounds derived from the arithmetic there."""

import numpy as np
import pytest
import torch

import __graft_entry__
import expert_ref as R
import mx_microscaling_quantize_gb300 as mxq
import train_ref as T

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
KINDS = {"silu": mxq.SILU, "gelu": mxq.GELU, "gelu_tanh": mxq.GELU_TANH}


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    yield
    assert mxq.mx_device_errors() == 0


def cpu(t):
    return t.cpu().numpy()


def rows(seed, M, K, dtype, offset=0.3):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) + offset
    x[:, rng.random(K) < 0.02] *= 30
    if M > 2:
        x[1] *= 2.0 ** 40   # a large row
        x[2] *= 2.0 ** -60  # a tiny one: eps decides
    return torch.from_numpy(x).to(dtype).cuda()


def params(seed, K, dtype):
    rng = np.random.default_rng(seed + 1)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(K)).to(dtype).cuda()
    b = torch.from_numpy(0.1 * rng.standard_normal(K)).to(dtype).cuda()
    return w, b


def either(t):
    return None if t is None else T.f64(t)


# ---------------------------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------------------------
NORMS = [(1, 1), (1, 33), (3, 7), (5, 32), (2, 512), (7, 520), (130, 1024), (17, 1032), (65, 2048),
         (33, 2056), (9, 8192), (300, 4096), (4, 8200), (3, 16384), (5, 16383), (1500, 96), (700, 1000)]


@pytest.mark.parametrize("M,K", NORMS)
@pytest.mark.parametrize("x_type,y_type", [(BF16, BF16), (FP32, BF16), (FP32, FP32), (BF16, FP32)])
@pytest.mark.parametrize("center", [True, False])
def test_layer_norm(M, K, x_type, y_type, center):
    x = rows(M * K, M, K, x_type)
    w, b = params(K, K, FP32 if M % 2 else BF16)
    for weight, bias in ((w, b), (w, None), (None, b), (None, None)):
        y, mean, rstd = mxq.mx_layer_norm(x, weight, bias, eps=1e-5, center=center, out_dtype=y_type, stats=True)
        want, m, r, tol = T.norm(T.f64(x), either(weight), either(bias), 1e-5, center)
        assert y.dtype == y_type
        T.check_values(y, want, tol, y_type)
        if center:
            T.check_values(mean, m, T.DEPTH * T.U * np.abs(T.f64(x)).mean(1), FP32, "mean")
        else:
            assert mean is None
        # rstd: the variance's sum, and the mean's error against the deviation
        rel = T.DEPTH * T.U * (1 + (np.abs(T.f64(x)).mean(1) * r if center else 0))
        T.check_values(rstd, r, rel * r, FP32, "rstd")
        if weight is None:  # without statistics: the same
            alone = mxq.mx_layer_norm(x, weight, bias, eps=1e-5, center=center, out_dtype=y_type)
            assert torch.equal(alone.view(torch.uint8), y.view(torch.uint8))


OPERANDS = [(1, 32), (3, 64), (5, 160), (2, 512), (130, 1024), (65, 1056), (300, 2048), (9, 8192), (4, 8224),
            (3, 16384), (1500, 96)]


@pytest.mark.parametrize("M,K", OPERANDS)
@pytest.mark.parametrize("x_type", [BF16, FP32])
@pytest.mark.parametrize("center", [True, False])
def test_layer_norm_operand(M, K, x_type, center):
    x = rows(M * K, M, K, x_type)
    w, b = params(K, K, BF16 if M % 2 else FP32)
    codes, scales, mean, rstd, kept, kept_scales = mxq.mx_layer_norm_b128(
        x, w, b, center=center, stats=True, checkpoint=True)
    want, _, _, tol = T.norm(T.f64(x), T.f64(w), T.f64(b), 1e-5, center)
    T.check_codes(codes, scales, want, tol)
    c, s, _ = T.checkpoint(x)
    assert (cpu(kept) == c).all() and (cpu(kept_scales) == s).all()
    # the same statistics as the plain call, the same operand without the extras
    _, mean2, rstd2 = mxq.mx_layer_norm(x, w, b, center=center, stats=True)
    assert torch.equal(rstd, rstd2) and (mean is None if not center else torch.equal(mean, mean2))
    alone = mxq.mx_layer_norm_b128(x, w, b, center=center)
    assert len(alone) == 2 and torch.equal(alone[0], codes) and torch.equal(alone[1], scales)
    assert len(mxq.mx_layer_norm_b128(x, None, None, center=center, checkpoint=True)) == 4


@pytest.mark.parametrize("M,K", NORMS)
@pytest.mark.parametrize("x_type,dy_type,dx_type", [(BF16, BF16, BF16), (FP32, BF16, FP32), (FP32, FP32, FP32),
                                                    (BF16, FP32, FP32)])
@pytest.mark.parametrize("center", [True, False])
def test_layer_norm_backward(M, K, x_type, dy_type, dx_type, center):
    x = rows(M * K, M, K, x_type)
    w, _ = params(K, K, BF16 if M % 2 else FP32)
    dy = rows(M * K + 7, M, K, dy_type, 0.0)
    _, mean, rstd = mxq.mx_layer_norm(x, w, None, center=center, stats=True)
    for weight in (w, None):
        dx, dw, db = mxq.mx_layer_norm_backward(dy, x, mean, rstd, weight, out_dtype=dx_type)
        want = T.norm_backward(T.f64(dy), T.f64(x), either(mean), T.f64(rstd), either(weight), center)
        assert dx.dtype == dx_type and dw.dtype == db.dtype == FP32
        T.check_values(dx, want[0], want[3], dx_type, "dx")
        T.check_values(dw, want[1], want[4], FP32, "dw")
        T.check_values(db, want[2], want[5], FP32, "db")
    only = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w, weight_grad=False, bias_grad=False, out_dtype=dx_type)
    assert only[1] is None and only[2] is None
    both = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w, out_dtype=dx_type)
    assert torch.equal(only[0].view(torch.uint8), both[0].view(torch.uint8))
    for kw, k in ((dict(weight_grad=False), 2), (dict(bias_grad=False), 1)):
        one = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w, out_dtype=dx_type, **kw)
        assert one[3 - k] is None and torch.equal(one[k], both[k])


@pytest.mark.parametrize("M,K", OPERANDS)
@pytest.mark.parametrize("dy_type,dx_type", [(BF16, BF16), (BF16, FP32), (FP32, FP32)])
@pytest.mark.parametrize("center", [True, False])
def test_layer_norm_backward_from_checkpoint(M, K, dy_type, dx_type, center):
    x = rows(M * K, M, K, FP32)
    w, _ = params(K, K, FP32)
    dy = rows(M * K + 7, M, K, dy_type, 0.0)
    _, _, mean, rstd, kept, kept_scales = mxq.mx_layer_norm_b128(x, w, None, center=center, stats=True,
                                                                 checkpoint=True)
    dx, dw, db = mxq.mx_layer_norm_backward(dy, kept, mean, rstd, w, x_scales=kept_scales, out_dtype=dx_type)
    v = T.values(cpu(kept), cpu(kept_scales)).astype(np.float64)
    want = T.norm_backward(T.f64(dy), v, either(mean), T.f64(rstd), T.f64(w), center, checkpoint=True)
    T.check_values(dx, want[0], want[3], dx_type, "dx")
    T.check_values(dw, want[1], want[4], FP32, "dw")
    T.check_values(db, want[2], want[5], FP32, "db")


@pytest.mark.parametrize("center", [True, False])
def test_layer_norm_gradients_against_differences(center):
    """Central differences of sum(dy * y) in fp32 in and out: y is off by some 2^-19 of its size, steps of
    2^-7 leave an error of the square, so a difference is good to about 2^-11 of the gradient's size."""
    M, K, h = 3, 40, 2.0 ** -7
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((M, K))).float().cuda()
    w, b = params(5, K, FP32)
    dy = torch.from_numpy(rng.standard_normal((M, K))).float().cuda()
    _, mean, rstd = mxq.mx_layer_norm(x, w, b, center=center, stats=True)
    dx, dw, db = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w)

    def loss(x, w, b):
        return float((mxq.mx_layer_norm(x, w, b, center=center).double() * dy.double()).sum())

    def differences(t, call):
        out = np.zeros(t.shape)
        for i in np.ndindex(*t.shape):
            up, down = t.clone(), t.clone()
            up[i] += h
            down[i] -= h
            out[i] = (call(up) - call(down)) / float(up[i] - down[i])
        return out
    for got, want in ((dx, differences(x, lambda t: loss(t, w, b))), (dw, differences(w, lambda t: loss(x, t, b))),
                      (db, differences(b, lambda t: loss(x, w, t)))):
        assert np.abs(T.f64(got) - want).max() <= 2.0 ** -9 * max(1.0, np.abs(want).max())


# ---------------------------------------------------------------------------------------------
# activation
# ---------------------------------------------------------------------------------------------
ACTS = [(1, 32), (1, 1024), (5, 96), (3, 128), (33, 640), (130, 256), (17, 2048), (700, 128), (2, 28672)]


def act_input(seed, R_, U_):
    rng = np.random.default_rng(seed)
    u = rng.standard_normal((R_, U_)) * 2
    u[:, rng.random(U_) < 0.03] *= 30  # saturated both ways
    if R_ > 1:
        u[1, : U_ // 2] *= 2.0 ** -20
    return torch.from_numpy(u).bfloat16().cuda()


@pytest.mark.parametrize("M,H", ACTS)
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("gated", [True, False])
def test_activation(M, H, kind, gated):
    u = act_input(M * H, M, H * (2 if gated else 1))
    codes, scales = mxq.mx_activation_b128(u, KINDS[kind], gated=gated)
    v = T.f64(u)
    h, _, tol, _ = T.act(kind, v[:, :H])
    if gated:
        tol = tol * np.abs(v[:, H:]) + T.U * np.abs(h * v[:, H:])
        h = h * v[:, H:]
    T.check_codes(codes, scales, h, tol)
    if gated and H % 128:
        with pytest.raises(mxq.MXError):
            mxq.mx_activation_b128(u, KINDS[kind], checkpoint=True)
        return
    c2, s2, kept, kept_scales = mxq.mx_activation_b128(u, KINDS[kind], gated=gated, checkpoint=True)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    c, s = mxq.mx_quantize_b128_rows(u)
    assert torch.equal(kept, c) and torch.equal(kept_scales, s)


@pytest.mark.parametrize("M,H", ACTS)
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("checkpoint", [True, False])
def test_activation_backward(M, H, kind, gated, checkpoint):
    u = act_input(M * H, M, H * (2 if gated else 1))
    dh = rows(M + H, M, H, BF16, 0.0)
    whole = not gated or H % 128 == 0
    kw = {}
    src, v = u, T.f64(u)
    if checkpoint:
        if not whole:
            pytest.skip("blocks of gate and up would share a scale")
        src, kw["u_scales"] = mxq.mx_quantize_b128_rows(u)
        v = T.values(cpu(src), cpu(kw["u_scales"])).astype(np.float64)
    h, d, tol_h, tol_d = T.act(kind, v[:, :H])
    g = T.f64(dh)
    if gated:
        up = v[:, H:]
        want = np.concatenate([g * up * d, g * h], 1)
        tol = np.concatenate([np.abs(g * up) * (tol_d + 3 * T.U * np.abs(d)), np.abs(g) * (tol_h + T.U * np.abs(h))], 1)
    else:
        want, tol = g * d, np.abs(g) * (tol_d + T.U * np.abs(d))
    du = mxq.mx_activation_backward(dh, src, KINDS[kind], gated=gated, **kw)
    T.check_values(du, want, tol, BF16)
    if not whole:
        with pytest.raises(mxq.MXError):
            mxq.mx_activation_backward(dh, src, KINDS[kind], gated=gated, operand=True, **kw)
        return
    du2, codes, scales = mxq.mx_activation_backward(dh, src, KINDS[kind], gated=gated, operand=True, **kw)
    assert torch.equal(du2.view(torch.int16), du.view(torch.int16))
    T.check_codes(codes, scales, want, tol)
    c3, s3 = mxq.mx_activation_backward(dh, src, KINDS[kind], gated=gated, operand=True, grad=False, **kw)
    assert torch.equal(c3, codes) and torch.equal(s3, scales)


@pytest.mark.parametrize("kind", list(KINDS))
def test_activation_gradient_is_that_of_the_definition(kind):
    """The formulas of T.act against its own central differences in 64 bits."""
    g, h = np.linspace(-9, 9, 721), 1e-5
    d = (T.act(kind, g + h)[0] - T.act(kind, g - h)[0]) / (2 * h)
    assert np.abs(d - T.act(kind, g)[1]).max() < 1e-8


# ---------------------------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------------------------
def stored(seed, M, K):
    """A checkpoint with a block of zeros, tiny and huge blocks."""
    x = rows(seed, M, K, BF16)
    if M > 4 and K >= 256:
        x[3, :128] = 0
        x[4, 128:256] *= 2.0 ** -120
    return mxq.mx_quantize_b128_rows(x)


SHAPES = [(1, 32), (5, 96), (128, 128), (130, 160), (300, 1056), (64, 4096), (1, 8192), (1000, 224)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_dequantize(M, K, dtype):
    codes, scales = stored(M * K, M, K)
    want = torch.from_numpy(T.values(cpu(codes), cpu(scales)))
    assert torch.equal(mxq.mx_dequantize_b128_rows(codes, scales, out_dtype=dtype).cpu(), want.to(dtype))
    index = torch.tensor([M - 1, 0, -1, M, M // 2, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    got = mxq.mx_dequantize_b128_rows(codes, scales, index, out_dtype=dtype).cpu()
    for i, r in enumerate(index.tolist()):
        assert torch.equal(got[i], want[r].to(dtype) if 0 <= r < M else torch.zeros(K, dtype=dtype)), i


def requantized(v, R_, offsets=None):
    """Reference columns of rows v (fp32), grouped by offsets: codes [K, P], scales [P / 128, K]."""
    K = v.shape[1]
    parts = [v] if offsets is None else [v[a:b] for a, b in zip(offsets[:-1], offsets[1:])]
    codes, scales = [], []
    for p in parts:
        if p.shape[0] == 0:
            continue
        full = np.zeros((R.up(p.shape[0]), K), np.float32)
        full[:p.shape[0]] = p
        c, s = R.quantize(full, R.BLK, 1)
        codes.append(c)
        scales.append(s)
    return (np.concatenate(codes).T, np.concatenate(scales)) if codes else (np.zeros((K, 0)), np.zeros((0, K)))


@pytest.mark.parametrize("M,K", SHAPES + [(2500, 4128)])
def test_requantize_cols(M, K):
    codes, scales = stored(M * K, M, K)
    got = mxq.mx_requantize_b128_cols(codes, scales)
    want = requantized(T.values(cpu(codes), cpu(scales)), M)
    assert (cpu(got[0]) == want[0]).all() and (cpu(got[1]) == want[1]).all()


@pytest.mark.parametrize("counts", [[0, 5, 0, 300, 128], [1], [0, 0], [129, 1, 127, 0, 64, 256], [40] * 60])
@pytest.mark.parametrize("K", [96, 1056])
@pytest.mark.parametrize("gather", [False, True])
def test_requantize_cols_by_expert(counts, K, gather):
    rng = np.random.default_rng(sum(counts) + K)
    off = np.concatenate([[0], np.cumsum(counts)])
    n = int(off[-1])
    M = 77 if gather else n
    codes, scales = stored(n + K, M, K) if M else (torch.empty(0, K, dtype=torch.uint8, device="cuda"),
                                                   torch.empty(-(-K // 128), 0, device="cuda"))
    v = T.values(cpu(codes), cpu(scales))
    index = None
    if gather:
        at = rng.integers(-2, M + 2, n)
        index = torch.from_numpy(at.astype(np.int32)).cuda()
        v = np.where(((at >= 0) & (at < M))[:, None], v[np.clip(at, 0, M - 1)], np.float32(0))
    offsets = torch.from_numpy(off).cuda()
    P = mxq.mx_b128_padded_rows(n, len(counts))
    out = torch.full((K, P), 0xA5, dtype=torch.uint8, device="cuda")
    out_s = torch.full((P // 128, K), -7.0, device="cuda")
    mxq.mx_requantize_b128_cols(codes, scales, index, offsets, out_codes=out, out_scales=out_s)
    want, want_s = requantized(v, n, off)
    c, s = cpu(out), cpu(out_s)
    p = want.shape[1]
    assert (c[:, :p] == want).all() and (s[:p // 128] == want_s).all()
    assert (c[:, p:] == 0xA5).all() and (s[p // 128:] == -7.0).all()  # the caller's
