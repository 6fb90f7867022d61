"""Where layer norm, activation and checkpoints can go wrong on the GPU: unaligned bases, NaN, infinities and
the ends of fp32, large means, rows that do not fill their groups, streams, graphs, chains of dependent calls,
give-ups, offsets that break their contract, refusals, and the far end of large tensors."""

import numpy as np
import pytest
import torch

import __graft_entry__
import expert_ref as R
import mx_microscaling_quantize_gb300 as mxq
import train_ref as T
from test_gpu_train import BF16, FP32, KINDS, act_input, cpu, either, params, rows, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    yield
    assert mxq.mx_device_errors() == 0


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return a is b is None or (a.dtype == b.dtype and torch.equal(bits(a), bits(b)))


def off_base(t, by=1):
    """A copy of t that starts `by` elements past an aligned base."""
    flat = torch.empty(t.numel() + by + 16, dtype=t.dtype, device=t.device)
    flat[by:by + t.numel()] = t.flatten()
    return flat[by:by + t.numel()].view(t.shape)


# ---------------------------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("M,K", [(5, 64), (33, 1024), (3, 8192)])
@pytest.mark.parametrize("which", ["x", "w", "b", "y", "all"])
@pytest.mark.parametrize("x_type", [BF16, FP32])
def test_norm_of_bases_that_allow_no_wide_loads(M, K, which, x_type):
    x = rows(M * K, M, K, x_type)
    w, b = params(K, K, FP32)
    want, _, _, tol = T.norm(T.f64(x), T.f64(w), T.f64(b), 1e-5, True)
    y = torch.empty(M, K, dtype=BF16, device="cuda")
    args = {"x": x, "w": w, "b": b, "y": y}
    for name in args:
        if which in (name, "all"):
            args[name] = off_base(args[name])
    got = mxq.mx_layer_norm(args["x"], args["w"], args["b"], y=args["y"])
    assert got.data_ptr() == args["y"].data_ptr()
    T.check_values(got, want, tol, BF16)


@pytest.mark.parametrize("M,K", [(5, 64), (33, 1024), (3, 8224)])
@pytest.mark.parametrize("which", ["x", "w", "dy", "dx", "all"])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_norm_backward_of_bases_that_allow_no_wide_loads(M, K, which, checkpoint):
    x = rows(M * K, M, K, FP32)
    w, _ = params(K, K, FP32)
    dy = rows(M + K, M, K, BF16, 0.0)
    _, mean, rstd = mxq.mx_layer_norm(x, w, None, stats=True)
    kw, v = {}, T.f64(x)
    if checkpoint:
        x, kw["x_scales"] = mxq.mx_layer_norm_b128(x, checkpoint=True)[2:]
        v = T.values(cpu(x), cpu(kw["x_scales"])).astype(np.float64)
    args = {"x": x, "w": w, "dy": dy, "dx": torch.empty(M, K, dtype=BF16, device="cuda")}
    for name in args:
        if which in (name, "all"):
            args[name] = off_base(args[name])
    dx, dw, db = mxq.mx_layer_norm_backward(args["dy"], args["x"], mean, rstd, args["w"], dx=args["dx"], **kw)
    want = T.norm_backward(T.f64(dy), v, T.f64(mean), T.f64(rstd), T.f64(w), True, checkpoint=checkpoint)
    T.check_values(dx, want[0], want[3], BF16, "dx")
    T.check_values(dw, want[1], want[4], FP32, "dw")
    T.check_values(db, want[2], want[5], FP32, "db")


@pytest.mark.parametrize("M", [1, 2, 152, 153, 160, 305])
@pytest.mark.parametrize("K", [40, 1024, 2080, 9000])
def test_norm_parameter_gradients_at_any_base(M, K):
    """Few rows leave their shares of dw and db as they are, more of them go through the groups' sums."""
    x, dy = rows(M + K, M, K, BF16), rows(M * 5 + K, M, K, BF16, 0.0)
    w, _ = params(K, K, FP32)
    _, mean, rstd = mxq.mx_layer_norm(x, w, None, stats=True)
    want = T.norm_backward(T.f64(dy), T.f64(x), T.f64(mean), T.f64(rstd), T.f64(w), True)
    need = mxq.mx_layer_norm_backward_workspace(M, K)
    guarded = [torch.full((n + 16,), -3.0, device="cuda") for n in (K, K, need // 4)]
    for at in (0, 1, 4, 8):
        dw, db, ws = (g[at:at + n] for g, n in zip(guarded, (K, K, need // 4)))
        mxq.mx_layer_norm_backward(dy, x, mean, rstd, w, dweight=dw, dbias=db, workspace=ws)
        T.check_values(dw, want[1], want[4], FP32, "dw")
        T.check_values(db, want[2], want[5], FP32, "db")
        for g, n in zip(guarded, (K, K, need // 4)):
            assert (g[:at] == -3).all() and (g[at + n:] == -3).all()
            g.fill_(-3.0)
        only = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w, weight_grad=False)
        assert only[1] is None and same(only[2], mxq.mx_layer_norm_backward(dy, x, mean, rstd, w)[2])


@pytest.mark.parametrize("K", [96, 1024, 1111, 8192])
@pytest.mark.parametrize("x_type", [BF16, FP32])
def test_norm_of_large_means(K, x_type):
    """A mean of 64 deviations: the variance is that of the differences, not of the squares."""
    x = rows(K, 37, K, FP32, 64.0).to(x_type)
    y, mean, rstd = mxq.mx_layer_norm(x, out_dtype=FP32, stats=True)
    want, m, r, tol = T.norm(T.f64(x), None, None, 1e-5, True)
    T.check_values(y, want, tol, FP32)
    rel = T.DEPTH * T.U * (1 + np.abs(T.f64(x)).mean(1) * r)
    T.check_values(rstd, r, rel * r, FP32, "rstd")


@pytest.mark.parametrize("K", [32, 512, 1024, 1056, 8192, 333])
@pytest.mark.parametrize("center", [True, False])
def test_norm_of_nan_and_infinite_rows(K, center):
    """A row with a NaN or an infinity (centred: whose mean is none) is NaN; its neighbours are not."""
    x = rows(K, 12, K, FP32)
    clean = x.clone()
    bad = {1: np.nan, 4: np.inf, 5: -np.inf, 8: np.nan, 11: np.nan}
    for r, v in bad.items():
        x[r, (7 * r) % K] = v
    w, b = params(K, K, FP32)
    y, mean, rstd = mxq.mx_layer_norm(x, w, b, center=center, stats=True)
    want = mxq.mx_layer_norm(clean, w, b, center=center)
    for r in range(12):
        if r not in bad:
            assert torch.equal(y[r], want[r])
        elif center or np.isnan(bad[r]):
            assert y[r].isnan().all() and rstd[r].isnan()
        else:  # not centred, infinite: 1 / deviation is 0
            at = (7 * r) % K
            assert rstd[r] == 0 and y[r, at].isnan()
            rest = torch.arange(K, device="cuda") != at
            assert torch.equal(y[r][rest], b[rest])
    if K % 32:
        return
    codes, scales, kept, kept_scales = mxq.mx_layer_norm_b128(x, w, b, center=center, checkpoint=True)
    want = mxq.mx_layer_norm_b128(clean, w, b, center=center, checkpoint=True)
    for r in range(12):
        if r not in bad:
            assert torch.equal(codes[r], want[0][r]) and torch.equal(scales[:, r], want[1][:, r])
            assert torch.equal(kept[r], want[2][r]) and torch.equal(kept_scales[:, r], want[3][:, r])
        else:
            if center or np.isnan(bad[r]):
                assert scales[:, r].isnan().all() and (codes[r] == 0x7F).all()
            kb = (7 * r) % K // 128
            assert kept_scales[kb, r].isnan() and (kept[r, kb * 128:(kb + 1) * 128] == 0x7F).all()
            assert kept_scales[:, r].isnan().sum() == 1


def test_norm_of_constant_and_zero_rows():
    x = torch.zeros(4, 512, device="cuda")
    x[1] = 3.0
    x[2] = 1e30
    w, b = params(1, 512, FP32)
    y, mean, rstd = mxq.mx_layer_norm(x, w, b, stats=True)
    assert torch.equal(y[0], b) and torch.equal(y[1], b) and torch.equal(y[3], b)
    r = 1 / np.sqrt(np.float64(np.float32(1e-5)))
    assert abs(float(rstd[0]) / r - 1) < 4 * T.U and abs(float(rstd[1]) / r - 1) < 4 * T.U
    codes, scales = mxq.mx_layer_norm_b128(x[:1].contiguous())  # all zeros: the floor's scale
    assert not codes.any() and (scales == float(np.float32(R.FLOOR) / np.float32(448))).all()


def test_norm_backward_of_a_nan_stays_in_its_row_and_column():
    x, dy = rows(1, 40, 1024, FP32), rows(2, 40, 1024, BF16, 0.0)
    w, _ = params(3, 1024, FP32)
    _, mean, rstd = mxq.mx_layer_norm(x, w, None, stats=True)
    want = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w)
    dy[17, 300] = float("nan")
    dx, dw, db = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w)
    keep = torch.arange(40, device="cuda") != 17
    assert dx[17].isnan().all() and torch.equal(dx[keep], want[0][keep])
    keep = torch.arange(1024, device="cuda") != 300
    for got, ref in ((dw, want[1]), (db, want[2])):
        assert got[300].isnan() and torch.equal(got[keep], ref[keep])


@pytest.mark.parametrize("M,K", [(1, 8192), (2, 8192), (305, 8192), (609, 2048), (4865, 1024), (7, 16384),
                                 (2433, 512), (9729, 256), (313, 5120), (1000, 24)])
def test_rows_do_not_depend_on_their_neighbours(M, K):
    """Row by row the bits of a call on that row alone: whatever group, stage or pair it falls into."""
    x, dy = rows(M + K, M, K, BF16), rows(M * 3 + K, M, K, BF16, 0.0)
    w, b = params(K, K, FP32)
    y, mean, rstd = mxq.mx_layer_norm(x, w, b, stats=True)
    dx, dw, db = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w)
    for r in sorted({0, 1, M // 2, M - 2, M - 1} & set(range(M))):
        one = slice(r, r + 1)
        y1, m1, r1 = mxq.mx_layer_norm(x[one], w, b, stats=True)
        assert same(y1, y[one]) and same(m1, mean[one]) and same(r1, rstd[one])
        assert same(mxq.mx_layer_norm_backward(dy[one], x[one], m1, r1, w)[0], dx[one])
        if K % 32 == 0:
            got = mxq.mx_layer_norm_b128(x[one], w, b, checkpoint=True)
            want = mxq.mx_layer_norm_b128(x, w, b, checkpoint=True)
            assert same(got[0], want[0][one]) and same(got[1], want[1][:, one])
            assert same(got[2], want[2][one]) and same(got[3], want[3][:, one])
    want = T.norm_backward(T.f64(dy), T.f64(x), T.f64(mean), T.f64(rstd), T.f64(w), True)
    T.check_values(dw, want[1], want[4], FP32, "dw")
    T.check_values(db, want[2], want[5], FP32, "db")


@pytest.mark.parametrize("M,K", [(4001, 2048), (1219, 1032), (2501, 520), (1217, 40), (701, 8200), (305, 16384),
                                 (465, 5120), (3001, 96), (331, 14400), (2435, 256), (1233, 512), (613, 4096)])
@pytest.mark.parametrize("x_type", [BF16, FP32])
@pytest.mark.parametrize("center", [True, False])
def test_norm_of_many_rows_is_that_of_few(M, K, x_type, center):
    """Few rows go by a kernel of their own (a CTA each), many by groups that walk pairs of them: the same bits."""
    x = rows(M + K, M, K, x_type)
    w, b = params(K, K, FP32 if M % 2 else BF16)
    kw = dict(center=center, stats=True)
    parts = [x[i:i + 100].contiguous() for i in range(0, M, 100)]

    def check(many, few, dims):
        for i, dim in enumerate(dims):
            got = many[i]
            assert got is None and few[0][i] is None or same(got, torch.cat([f[i] for f in few], dim))
    for y_type in (BF16, FP32):
        check(mxq.mx_layer_norm(x, w, b, out_dtype=y_type, **kw),
              [mxq.mx_layer_norm(p, w, b, out_dtype=y_type, **kw) for p in parts], (0, 0, 0))
    if K % 32 == 0:
        check(mxq.mx_layer_norm_b128(x, w, b, checkpoint=True, **kw),
              [mxq.mx_layer_norm_b128(p, w, b, checkpoint=True, **kw) for p in parts], (0, 1, 0, 0, 0, 1))
        check(mxq.mx_layer_norm_b128(x, w, None, **kw), [mxq.mx_layer_norm_b128(p, w, None, **kw) for p in parts],
              (0, 1, 0, 0))


def test_norm_of_no_rows_and_no_columns():
    empty = torch.empty(0, 64, dtype=BF16, device="cuda")
    w, b = params(1, 64, FP32)
    y, mean, rstd = mxq.mx_layer_norm(empty, w, b, stats=True)
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    assert [tuple(t.shape) for t in mxq.mx_layer_norm_b128(empty, w, b, checkpoint=True)] == \
        [(0, 64), (1, 0), (0, 64), (1, 0)]
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    dx, dw, db = mxq.mx_layer_norm_backward(empty, empty, mean, rstd, w, dweight=dw, dbias=db)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    none = torch.empty(3, 0, device="cuda")
    y, mean, rstd = mxq.mx_layer_norm(none, stats=True)
    assert y.shape == (3, 0)
    assert mxq.mx_layer_norm_backward(none, none, mean, rstd)[0].shape == (3, 0)


def test_norm_statistics_of_rows_without_columns_are_zeros():
    none = torch.empty(3, 0, device="cuda")
    for norm in (mxq.mx_layer_norm, mxq.mx_layer_norm_b128):
        mean, rstd = torch.full((3,), 7.0, device="cuda"), torch.full((3,), 7.0, device="cuda")
        norm(none, mean=mean, rstd=rstd)
        assert not mean.any() and not rstd.any()


def test_norm_backward_refuses_a_workspace_that_is_shorter_than_it_looks():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    mean, rstd = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
    need = mxq.mx_layer_norm_backward_workspace(4, 64)
    for bad in (torch.zeros(1, device="cuda").expand(need), torch.zeros(need // 4 - 1, device="cuda"),
                torch.zeros(need, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            mxq.mx_layer_norm_backward(x, x, mean, rstd, workspace=bad)
    with pytest.raises(mxq.MXError):
        mxq.mx_layer_norm_backward(x, x, mean, rstd,
                                   workspace=torch.zeros(need + 1, dtype=torch.uint8, device="cuda")[1:])


def test_norm_writes_nothing_beside_its_outputs():
    M, K = 7, 1000
    x = rows(1, M, K, BF16)
    for by in (0, 1, 16):
        flat = torch.full((M * K + 64,), 7.0, dtype=BF16, device="cuda")
        mxq.mx_layer_norm(x, y=flat[by:by + M * K].view(M, K))
        assert (flat[:by] == 7).all() and (flat[by + M * K:] == 7).all()
        _, mean, rstd = mxq.mx_layer_norm(x, stats=True)
        flat.fill_(7.0)
        mxq.mx_layer_norm_backward(x, x, mean, rstd, dx=flat[by:by + M * K].view(M, K))
        assert (flat[:by] == 7).all() and (flat[by + M * K:] == 7).all()


# ---------------------------------------------------------------------------------------------
# activation
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", list(KINDS))
def test_activation_at_the_ends(kind):
    """Values of every bf16 exponent, in blocks of their own, forward and backward."""
    mag = np.ldexp(1.0, np.arange(-126, 127))
    v = np.concatenate([mag, -mag, [0.0, -0.0]])
    u = torch.zeros(v.size, 128, dtype=BF16, device="cuda")
    u[:, 0] = torch.from_numpy(v).bfloat16().cuda()
    g = T.f64(u)
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        h, d, tol_h, tol_d = T.act(kind, np.clip(g, -1e6, 1e6))
        h, tol_h = np.where(g > 1e6, g, h), np.where(g > 1e6, np.abs(g) * 2.0 ** -22, tol_h)
    codes, scales = mxq.mx_activation_b128(u, KINDS[kind], gated=False)
    # values whose scaled block is a number in fp32 (the largest are the block's own abs-max)
    T.check_codes(codes, scales, h, tol_h)
    dh = torch.ones(v.size, 128, dtype=BF16, device="cuda")
    du = mxq.mx_activation_backward(dh, u, KINDS[kind], gated=False)
    # beyond 2^20 the derivative is 0 or 1 within the bound at the clipped place
    T.check_values(du, d, tol_d, BF16)
    assert du.isfinite().all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_activation_of_nan_and_infinity(kind):
    u = act_input(3, 6, 512)
    clean = u.clone()
    u[1, 3], u[2, 200], u[4, 300], u[5, 10] = float("nan"), float("inf"), float("nan"), float("-inf")
    codes, scales, kept, kept_scales = mxq.mx_activation_b128(u, KINDS[kind], checkpoint=True)
    want = mxq.mx_activation_b128(clean, KINDS[kind], checkpoint=True)
    dh = rows(1, 6, 256, BF16, 0.0)
    du = mxq.mx_activation_backward(dh, u, KINDS[kind])
    du_want = mxq.mx_activation_backward(dh, clean, KINDS[kind])
    hit = {(1, 0), (2, 1), (4, 0), (5, 0)}  # rows and blocks of h
    for r in range(6):
        for kb in range(2):
            cols = slice(kb * 128, kb * 128 + 128)
            if (r, kb) in hit:
                assert scales[kb, r].isnan() and (codes[r, cols] == 0x7F).all()
            else:
                assert torch.equal(codes[r, cols], want[0][r, cols]) and torch.equal(scales[kb, r], want[1][kb, r])
    assert kept_scales.isnan().sum() == 4
    ok = torch.ones(6, 256, dtype=torch.bool, device="cuda")
    ok[1, 3] = ok[2, 200] = ok[4, 44] = ok[5, 10] = False
    both = torch.cat([ok, ok], 1)
    assert torch.equal(du[both], du_want[both])
    assert du[1, 3].isnan() and du[1, 259].isnan() and du[4, 44].isnan()


@pytest.mark.parametrize("M,H", [(1, 32), (2, 4096 + 32), (1000, 544), (9, 128)])
def test_activation_writes_nothing_beside_its_outputs(M, H):
    u, dh = act_input(M + H, M, H), rows(H, M, H, BF16, 0.0)
    B = -(-H // 128)
    for call, want in ((lambda c, s: mxq.mx_activation_b128(u, gated=False, codes=c, scales=s), None),
                       (lambda c, s: mxq.mx_activation_backward(dh, u, gated=False, grad=False, codes=c, scales=s),
                        None)):
        c = torch.full((M * H + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((B * M + 8,), -7.0, device="cuda")
        got = call(c[32:32 + M * H].view(M, H), s[4:4 + B * M].view(B, M))
        assert len(got) == 2
        assert (c[:32] == 0xA5).all() and (c[32 + M * H:] == 0xA5).all()
        assert (s[:4] == -7).all() and (s[4 + B * M:] == -7).all() and (s[4:4 + B * M] > 0).all()


# ---------------------------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------------------------
def test_requantize_of_nan_blocks():
    x = rows(5, 300, 384, BF16)
    x[17, 130] = float("nan")
    x[200, 5] = float("inf")
    codes, scales = mxq.mx_quantize_b128_rows(x)
    got, got_s = mxq.mx_requantize_b128_cols(codes, scales)
    bad = torch.zeros(3, 384, dtype=torch.bool, device="cuda")  # blocks of rows, columns
    bad[0, 128:256] = bad[1, :128] = True
    assert torch.equal(got_s.isnan(), bad)
    for b in range(3):
        assert (got[:, b * 128:(b + 1) * 128][bad[b]] == 0x7F).all()
    clean = torch.where(x.isfinite(), x, 0)
    clean[17, 128:256] = clean[200, :128] = 0
    want, want_s = mxq.mx_requantize_b128_cols(*mxq.mx_quantize_b128_rows(clean))
    for b in range(3):
        ok = ~bad[b]
        assert torch.equal(got[:, b * 128:(b + 1) * 128][ok], want[:, b * 128:(b + 1) * 128][ok])
        assert torch.equal(got_s[b][ok], want_s[b][ok])
    v = mxq.mx_dequantize_b128_rows(codes, scales)
    assert v[17, 128:256].isnan().all() and v[200, :128].isnan().all()
    assert int(v.isnan().sum()) == 256


def test_requantize_contract_breaking_offsets_stay_inside():
    codes, scales = stored(1, 300, 160)
    for off in ([0, 500, 300], [-5, 10, 300], [0, 200, 100, 300], [300, 0, 300], [2 ** 40, -2 ** 40, 7, 300]):
        P = mxq.mx_b128_padded_rows(300, len(off) - 1)
        flat = torch.full((160 * P + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((P // 128 * 160 + 8,), -7.0, device="cuda")
        mxq.mx_requantize_b128_cols(codes, scales, None, torch.tensor(off, device="cuda"),
                                    out_codes=flat[32:32 + 160 * P].view(160, P),
                                    out_scales=s[4:4 + P // 128 * 160].view(P // 128, 160))
        assert (flat[:32] == 0xA5).all() and (flat[32 + 160 * P:] == 0xA5).all()
        assert (s[:4] == -7).all() and (s[4 + P // 128 * 160:] == -7).all()


def test_empty_checkpoints():
    codes, scales = torch.empty(0, 64, dtype=torch.uint8, device="cuda"), torch.empty(1, 0, device="cuda")
    assert mxq.mx_dequantize_b128_rows(codes, scales).shape == (0, 64)
    c, s = mxq.mx_requantize_b128_cols(codes, scales)
    assert c.shape == (64, 0) and s.shape == (0, 64)
    # rows of nothing are zeros, gathered or not
    index = torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda")
    assert not mxq.mx_dequantize_b128_rows(codes, scales, index).any()
    c, s = mxq.mx_requantize_b128_cols(codes, scales, index)
    assert c.shape == (64, 128) and not c.any() and (s == float(np.float32(R.FLOOR) / np.float32(448))).all()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    codes, scales = stored(2, 9, 64)
    assert mxq.mx_dequantize_b128_rows(codes, scales, none).shape == (0, 64)
    assert mxq.mx_requantize_b128_cols(codes, scales, none)[0].shape == (64, 0)


# ---------------------------------------------------------------------------------------------
# streams, graphs, chains, repeats, give-ups
# ---------------------------------------------------------------------------------------------
def layer_step(x, dy, w, b, up, down, kind, **at):
    """Norm, gated products and the way back, everything kept in 8 bits: every output of every call."""
    (wu, su, wut, sut), (wd, sd, wdt, sdt) = up, down
    xn, xns, mean, rstd, xk, xks = mxq.mx_layer_norm_b128(x, w, b, stats=True, checkpoint=True, **at)
    u = mxq.mx_gemm_b128(xn, xns, wu, su, **at)
    h, hs, uk, uks = mxq.mx_activation_b128(u, kind, checkpoint=True, **at)
    y = mxq.mx_gemm_b128(h, hs, wd, sd, **at)
    dh = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(dy, **at), wdt, sdt, **at)
    dwd = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_cols(dy, **at), *mxq.mx_requantize_b128_cols(h, hs, **at),
                           mxq.B128_ROWS, out_dtype=FP32, **at)
    du, duc, dus = mxq.mx_activation_backward(dh, uk, kind, u_scales=uks, operand=True, **at)
    dwu = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_cols(du, **at), *mxq.mx_requantize_b128_cols(xn, xns, **at),
                           mxq.B128_ROWS, out_dtype=FP32, **at)
    dxn = mxq.mx_gemm_b128(duc, dus, wut, sut, **at)
    dx, dw, db = mxq.mx_layer_norm_backward(dxn, xk, mean, rstd, w, x_scales=xks, **at)
    y2, m2, r2 = mxq.mx_layer_norm(x, w, b, stats=True, **at)
    plain = mxq.mx_layer_norm_backward(dxn, x, m2, r2, w, **at)
    return [xn, xns, mean, rstd, xk, xks, u, h, hs, uk, uks, y, dh, dwd, du, duc, dus, dwu, dxn, dx, dw, db, y2,
            *plain, mxq.mx_dequantize_b128_rows(xk, xks, **at)]


def layer_inputs(seed, M=700, D=512, H=384):
    rng = np.random.default_rng(seed)
    new = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().cuda()  # noqa: E731
    x, dy = new(M, D).bfloat16(), new(M, D).bfloat16()
    w, b = 1 + 0.1 * new(D), 0.1 * new(D)
    up = mxq.mx_quantize_b128_blocks((new(2 * H, D) / D ** 0.5).bfloat16(), transpose=True)
    down = mxq.mx_quantize_b128_blocks((new(D, H) / H ** 0.5).bfloat16(), transpose=True)
    return x, dy, w, b, up, down, mxq.SILU


@pytest.mark.parametrize("raw", [False, True])
def test_stream_argument(raw):
    args = layer_inputs(1)
    want = layer_step(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = layer_step(*args, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert all(same(g, w) for g, w in zip(got, want))


def test_in_a_graph_replayed_on_new_inputs_and_beside_another_graph():
    a, b = layer_inputs(2), layer_inputs(3, M=333)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer_step(*a), layer_step(*b)
    side.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga, stream=side):
        ra = layer_step(*a)
    with torch.cuda.graph(gb, stream=side):
        rb = layer_step(*b)
    a[0].copy_(torch.randn_like(a[0]))
    a[1].copy_(torch.randn_like(a[1]))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):  # both at once, each with workspaces of its own
        with torch.cuda.stream(side):
            ga.replay()
        with torch.cuda.stream(other):
            gb.replay()
    torch.cuda.synchronize()
    assert all(same(g, w) for g, w in zip(ra, layer_step(*a)))
    assert all(same(g, w) for g, w in zip(rb, layer_step(*b)))


def test_two_streams_at_once():
    a, b = layer_inputs(4, M=2000), layer_inputs(5, M=1500)
    want = layer_step(*a), layer_step(*b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        got = []
        for stream, args in zip(s, (a, b)):
            with torch.cuda.stream(stream):
                got.append(layer_step(*args))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(same(p, q) for p, q in zip(g, w))


def test_dependent_calls_keep_stream_order():
    """The step into the same buffers over and over, each call reading what the one before has just written:
    the bytes are those of a synchronization after every call."""
    x, dy, w, b, up, down, kind = layer_inputs(6, M=1111)
    M, D = x.shape
    H = down[0].shape[1]
    P = mxq.mx_b128_padded_rows(M)
    u8 = torch.uint8
    new = lambda *s, dtype=FP32: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
    sources = [torch.randn(M, D, device="cuda").bfloat16() for _ in range(3)]
    o = dict(x=new(M, D, dtype=BF16), c=new(M, D, dtype=u8), s=new(D // 128, M), mean=new(M), rstd=new(M),
             xc=new(M, D, dtype=u8), xs=new(D // 128, M), u=new(M, 2 * H, dtype=BF16), h=new(M, H, dtype=u8),
             hs=new(H // 128, M), uc=new(M, 2 * H, dtype=u8), us=new(2 * H // 128, M), dh=new(M, H, dtype=BF16),
             du=new(M, 2 * H, dtype=BF16), duc=new(M, 2 * H, dtype=u8), dus=new(2 * H // 128, M),
             cc=new(D, P, dtype=u8), cs=new(P // 128, D), dxn=new(M, D, dtype=BF16), dx=new(M, D, dtype=BF16),
             dw=new(D), db=new(D), back=new(M, D, dtype=BF16), y=new(M, D, dtype=BF16),
             ws=new(mxq.mx_layer_norm_backward_workspace(M, D), dtype=u8))

    def chain(sync=False):
        seen = []
        for i in range(3):
            for step in (
                lambda: o["x"].copy_(sources[i]),
                lambda: mxq.mx_layer_norm_b128(o["x"], w, b, codes=o["c"], scales=o["s"], mean=o["mean"],
                                               rstd=o["rstd"], x_codes=o["xc"], x_scales=o["xs"]),
                lambda: mxq.mx_gemm_b128(o["c"], o["s"], up[0], up[1], c=o["u"]),
                lambda: mxq.mx_activation_b128(o["u"], kind, codes=o["h"], scales=o["hs"], u_codes=o["uc"],
                                               u_scales=o["us"]),
                lambda: mxq.mx_dequantize_b128_rows(o["h"], o["hs"], y=o["dh"]),
                lambda: mxq.mx_activation_backward(o["dh"], o["uc"], kind, u_scales=o["us"], du=o["du"],
                                                   codes=o["duc"], scales=o["dus"]),
                lambda: mxq.mx_gemm_b128(o["duc"], o["dus"], up[2], up[3], c=o["dxn"]),
                lambda: mxq.mx_layer_norm_backward(o["dxn"], o["xc"], o["mean"], o["rstd"], w, x_scales=o["xs"],
                                                   dx=o["dx"], dweight=o["dw"], dbias=o["db"], workspace=o["ws"]),
                lambda: mxq.mx_requantize_b128_cols(o["xc"], o["xs"], out_codes=o["cc"], out_scales=o["cs"]),
                lambda: mxq.mx_dequantize_b128_rows(o["xc"], o["xs"], y=o["back"]),
                lambda: mxq.mx_layer_norm(o["dx"], w, b, mean=o["mean"], rstd=o["rstd"], y=o["y"]),
                lambda: mxq.mx_layer_norm_backward(o["dxn"], o["dx"], o["mean"], o["rstd"], w, dx=o["x"],
                                                   dweight=o["dw"], dbias=o["db"], workspace=o["ws"]),
            ):
                step()
                if sync:
                    torch.cuda.synchronize()
            seen.append({name: t.clone() for name, t in o.items() if name != "ws"})
            if sync:
                torch.cuda.synchronize()
        return seen

    def check(got):
        torch.cuda.synchronize()
        for g, h in zip(got, want):
            for name in g:
                assert same(g[name], h[name]), name

    want = chain(sync=True)
    for _ in range(5):
        check(chain())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = chain()
    for _ in range(3):
        graph.replay()
        check(captured)


def test_repeated_calls_give_the_same_bits():
    args = layer_inputs(7, M=5000)
    first = layer_step(*args)
    for _ in range(3):
        assert all(same(g, w) for g, w in zip(layer_step(*args), first))


@pytest.mark.parametrize("M,K", [(3000, 8192), (5000, 1024), (900, 16384), (4000, 200)])
@pytest.mark.parametrize("limit", [1, 1000, 20000])
def test_give_up_leaves_the_context_usable(M, K, limit):
    x, dy = rows(M, M, K, BF16), rows(M + 1, M, K, BF16, 0.0)
    want, mean, rstd = mxq.mx_layer_norm(x, stats=True)
    calls = [(lambda ns: mxq.mx_selftest_layer_norm_give_up(x, ns), lambda: mxq.mx_layer_norm(x), want),
             (lambda ns: mxq.mx_selftest_layer_norm_backward_give_up(dy, x, mean, rstd, ns),
              lambda: mxq.mx_layer_norm_backward(dy, x, mean, rstd)[0], None)]
    if K % 32 == 0:
        kept, kept_scales = mxq.mx_quantize_b128_rows(x)
        calls.append((lambda ns: mxq.mx_selftest_layer_norm_backward_give_up(dy, kept, mean, rstd, ns,
                                                                             x_scales=kept_scales),
                      lambda: mxq.mx_layer_norm_backward(dy, kept, mean, rstd, x_scales=kept_scales)[0], None))
    for give_up, call, ref in calls:
        ref = call() if ref is None else ref
        torch.cuda.synchronize()
        assert mxq.mx_device_errors() == 0
        give_up(limit)
        assert mxq.mx_device_errors() in (0, 1)
        assert same(call(), ref)
        assert mxq.mx_device_errors() == 0


# ---------------------------------------------------------------------------------------------
# the operators together: a gated layer whose step keeps 8 bits, against the layer in 64 bits
# ---------------------------------------------------------------------------------------------
def test_step_of_a_layer_kept_in_8_bits():
    """Every operand and checkpoint rounds its values by up to 2^-4 (some 0.026 of their size on average), seven
    of them one after another on the longest way (dx): norms agree to a tenth."""
    x, dy, w, b, up, down, kind = layer_inputs(8, M=640)
    out = dict(zip(("xn", "xns", "mean", "rstd", "xk", "xks", "u", "h", "hs", "uk", "uks", "y", "dh", "dwd", "du",
                    "duc", "dus", "dwu", "dxn", "dx", "dw", "db"), layer_step(x, dy, w, b, up, down, kind)))

    def weight(codes, scales):
        v = T.f64(codes.view(torch.float8_e4m3fn).float())
        return torch.from_numpy(v * np.repeat(np.repeat(T.f64(scales), 128, 0), 128, 1)).requires_grad_()
    wu, wd = weight(*up[:2]), weight(*down[:2])
    X, W, B = (t.detach().cpu().double().requires_grad_() for t in (x, w, b))
    d = X - X.mean(1, keepdim=True)
    xn = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * W + B
    gate, upper = (xn @ wu.t()).chunk(2, 1)
    y = (torch.nn.functional.silu(gate) * upper) @ wd.t()
    y.backward(dy.cpu().double())
    for name, want in (("y", y.detach()), ("dx", X.grad), ("dw", W.grad), ("db", B.grad), ("dwu", wu.grad),
                       ("dwd", wd.grad)):
        got = out[name].cpu().double()
        assert float((got - want).norm() / want.norm()) <= 0.1, name


# ---------------------------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------------------------
def test_refusals():
    x, w = torch.zeros(4, 256, device="cuda", dtype=BF16), torch.ones(256, device="cuda")
    row = torch.zeros(4, device="cuda")
    codes, scales = mxq.mx_quantize_b128_rows(x)
    for call, error in (
        (lambda: mxq.mx_layer_norm(x.half()), TypeError), (lambda: mxq.mx_layer_norm(x.cpu()), TypeError),
        (lambda: mxq.mx_layer_norm(x.t()), ValueError), (lambda: mxq.mx_layer_norm(x[None]), ValueError),
        (lambda: mxq.mx_layer_norm(x, w[:8].contiguous()), ValueError),
        (lambda: mxq.mx_layer_norm(x, w, w[:8].contiguous()), ValueError),
        (lambda: mxq.mx_layer_norm(x, w, w.bfloat16()), TypeError),
        (lambda: mxq.mx_layer_norm(x, w.half()), TypeError),
        (lambda: mxq.mx_layer_norm(x, out_dtype=torch.float16), TypeError),
        (lambda: mxq.mx_layer_norm(x, y=x[:2]), ValueError),
        (lambda: mxq.mx_layer_norm(x, center=False, mean=row), ValueError),
        (lambda: mxq.mx_layer_norm(torch.zeros(2, 16392, device="cuda")), mxq.MXError),
        (lambda: mxq.mx_layer_norm_b128(x[:, :40].contiguous()), mxq.MXError),
        (lambda: mxq.mx_layer_norm_b128(off_base(x)), mxq.MXError),
        (lambda: mxq.mx_layer_norm_b128(x, off_base(w)), mxq.MXError),
        (lambda: mxq.mx_layer_norm_b128(x, scales=torch.zeros(3, device="cuda")), ValueError),
        (lambda: mxq.mx_layer_norm_backward(x, x[:2], row, row), ValueError),
        (lambda: mxq.mx_layer_norm_backward(x, x, row[:2], row), ValueError),
        (lambda: mxq.mx_layer_norm_backward(x, x, row, None), TypeError),
        (lambda: mxq.mx_layer_norm_backward(x, codes, row, row), TypeError),
        (lambda: mxq.mx_layer_norm_backward(x, codes, row, row, x_scales=scales[:1]), ValueError),
        (lambda: mxq.mx_layer_norm_backward(x, x, row, row, w[:8].contiguous()), ValueError),
        (lambda: mxq.mx_layer_norm_backward(x, x, row, row, workspace=torch.zeros(8, device="cuda")), ValueError),
        (lambda: mxq.mx_activation_b128(x.float()), TypeError),
        (lambda: mxq.mx_activation_b128(x[:, :33].contiguous()), ValueError),
        (lambda: mxq.mx_activation_b128(x[:, :80].contiguous()), mxq.MXError),
        (lambda: mxq.mx_activation_b128(x[:, :192].contiguous(), checkpoint=True), mxq.MXError),
        (lambda: mxq.mx_activation_b128(x, 3), mxq.MXError), (lambda: mxq.mx_activation_b128(off_base(x)), mxq.MXError),
        (lambda: mxq.mx_activation_backward(x, x), ValueError),
        (lambda: mxq.mx_activation_backward(x, x, gated=False, grad=False), ValueError),
        (lambda: mxq.mx_activation_backward(x, codes, gated=False), TypeError),
        (lambda: mxq.mx_activation_backward(x, codes, gated=False, u_scales=scales.half()), TypeError),
        (lambda: mxq.mx_requantize_b128_cols(codes, scales.t()), ValueError),
        (lambda: mxq.mx_requantize_b128_cols(codes.float(), scales), TypeError),
        (lambda: mxq.mx_requantize_b128_cols(codes, scales, row), TypeError),
        (lambda: mxq.mx_requantize_b128_cols(codes, scales, None, row.long()[:1]), ValueError),
        (lambda: mxq.mx_dequantize_b128_rows(codes, scales, out_dtype=torch.float16), TypeError),
        (lambda: mxq.mx_dequantize_b128_rows(codes, scales[:1]), ValueError),
        (lambda: mxq.mx_dequantize_b128_rows(codes, scales, y=x[:2]), ValueError),
    ):
        with pytest.raises(error):
            call()


# ---------------------------------------------------------------------------------------------
# tensors of more than 2^31 elements: the far end against a small call on a copy of it
# ---------------------------------------------------------------------------------------------
FAR, WIDE, NEAR = 1_100_000, 2048, 301


def far_rows(seed):
    x = torch.zeros(FAR, WIDE, device="cuda", dtype=BF16)
    x[-NEAR:] = rows(seed, NEAR, WIDE, BF16)
    return x, x[-NEAR:].clone()


def test_far_end_of_norms():
    x, near = far_rows(1)
    w, b = params(2, WIDE, FP32)
    y, mean, rstd = mxq.mx_layer_norm(x, w, b, stats=True)
    want = mxq.mx_layer_norm(near, w, b, stats=True)
    assert same(y[-NEAR:], want[0]) and same(mean[-NEAR:], want[1]) and same(rstd[-NEAR:], want[2])
    dx, dw, _ = mxq.mx_layer_norm_backward(y, x, mean, rstd, w, dx=torch.empty_like(x))
    want = mxq.mx_layer_norm_backward(want[0], near, *want[1:], w)
    assert same(dx[-NEAR:], want[0])
    del y, dx
    codes, scales, kept, kept_scales = mxq.mx_layer_norm_b128(x, w, b, checkpoint=True)
    want = mxq.mx_layer_norm_b128(near, w, b, checkpoint=True)
    assert torch.equal(codes[-NEAR:], want[0]) and torch.equal(scales[:, -NEAR:], want[1])
    assert torch.equal(kept[-NEAR:], want[2]) and torch.equal(kept_scales[:, -NEAR:], want[3])
    dx = mxq.mx_layer_norm_backward(x, kept, mean, rstd, w, x_scales=kept_scales, weight_grad=False, bias_grad=False)[0]
    want = mxq.mx_layer_norm_backward(near, want[2], mean[-NEAR:].clone(), rstd[-NEAR:].clone(), w, x_scales=want[3],
                                      weight_grad=False, bias_grad=False)[0]
    assert same(dx[-NEAR:], want)


def test_far_end_of_norms_of_any_length():
    x = torch.zeros(1_950_000, 1103, device="cuda", dtype=BF16)
    x[-5:] = rows(3, 5, 1103, BF16)
    near = x[-5:].clone()
    y, mean, rstd = mxq.mx_layer_norm(x, stats=True)
    want = mxq.mx_layer_norm(near, stats=True)
    assert same(y[-5:], want[0]) and same(mean[-5:], want[1])
    dx = mxq.mx_layer_norm_backward(x, y, mean, rstd, weight_grad=False, bias_grad=False)[0]
    want = mxq.mx_layer_norm_backward(near, want[0], *want[1:], weight_grad=False, bias_grad=False)[0]
    assert same(dx[-5:], want)


@pytest.mark.parametrize("gated", [True, False])
def test_far_end_of_activations(gated):
    u, near = far_rows(4)
    codes, scales, kept, kept_scales = mxq.mx_activation_b128(u, gated=gated, checkpoint=True)
    want = mxq.mx_activation_b128(near, gated=gated, checkpoint=True)
    assert torch.equal(codes[-NEAR:], want[0]) and torch.equal(scales[:, -NEAR:], want[1])
    assert torch.equal(kept[-NEAR:], want[2]) and torch.equal(kept_scales[:, -NEAR:], want[3])
    dh = torch.ones(FAR, codes.shape[1], device="cuda", dtype=BF16)
    for src, kw, small, small_kw in ((u, {}, near, {}),
                                     (kept, dict(u_scales=kept_scales), want[2], dict(u_scales=want[3]))):
        du, dc, ds = mxq.mx_activation_backward(dh, src, gated=gated, operand=True, **kw)
        ref = mxq.mx_activation_backward(dh[-NEAR:].clone(), small, gated=gated, operand=True, **small_kw)
        assert same(du[-NEAR:], ref[0]) and torch.equal(dc[-NEAR:], ref[1]) and torch.equal(ds[:, -NEAR:], ref[2])
        del du, dc, ds


@pytest.mark.parametrize("H", [1 << 27, (1 << 27) - 32, 512 * 4 * 65535])
def test_activation_of_the_longest_rows(H):
    """More tiles of columns than one dimension of a grid may have."""
    u = torch.zeros(1, H, device="cuda", dtype=BF16)
    at = list(range(0, H // 128, H // 1280)) + [H // 128 - 1]  # blocks with values in them
    for i in at:
        u[0, i * 128:i * 128 + 128] = rows(i, 1, 128, BF16)[0]
    dh = torch.ones_like(u)
    codes, scales = mxq.mx_activation_b128(u, mxq.GELU, gated=False)
    du, dc, ds = mxq.mx_activation_backward(dh, u, mxq.GELU, gated=False, operand=True)
    for i in at:
        one = slice(i * 128, i * 128 + 128)
        want = mxq.mx_activation_b128(u[:, one].contiguous(), mxq.GELU, gated=False)
        assert torch.equal(codes[:, one], want[0]) and torch.equal(scales[i], want[1][0])
        ref = mxq.mx_activation_backward(dh[:, one].contiguous(), u[:, one].contiguous(), mxq.GELU, gated=False,
                                         operand=True)
        assert same(du[:, one], ref[0]) and torch.equal(dc[:, one], ref[1]) and torch.equal(ds[i], ref[2][0])
    assert not codes.count_nonzero() - sum(codes[:, i * 128:i * 128 + 128].count_nonzero() for i in at)


def test_far_end_of_checkpoints():
    x, near = far_rows(5)
    codes, scales = mxq.mx_quantize_b128_rows(x)
    del x
    small = mxq.mx_quantize_b128_rows(near)
    want = mxq.mx_dequantize_b128_rows(*small)
    assert same(mxq.mx_dequantize_b128_rows(codes, scales)[-NEAR:], want)
    index = torch.arange(FAR - NEAR, FAR, device="cuda", dtype=torch.int32)
    assert same(mxq.mx_dequantize_b128_rows(codes, scales, index), want)
    want_c, want_s = mxq.mx_requantize_b128_cols(*small)
    got_c, got_s = mxq.mx_requantize_b128_cols(codes, scales, index)
    assert torch.equal(got_c, want_c) and torch.equal(got_s, want_s)
    offsets = torch.tensor([0, FAR - NEAR, FAR], device="cuda")
    got_c, got_s = mxq.mx_requantize_b128_cols(codes, scales, None, offsets)
    at = -(-(FAR - NEAR) // 128)
    assert torch.equal(got_c[:, at * 128:at * 128 + 384], want_c) and torch.equal(got_s[at:at + 3], want_s)
