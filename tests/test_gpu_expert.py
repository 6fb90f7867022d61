"""The expert-layer operators on the GPU against their plain 64-bit definitions (tests/expert_ref.py):
routing with its plan and gradient, E4M3 operands with a scale per block of 128, their products and
the combination of the experts' outputs. Codes, scales, choices and plans are compared exactly; the
bounds of everything else are derived from the arithmetic beside each test."""

import numpy as np
import pytest
import torch

import __graft_entry__
import expert_ref as R
import mx_microscaling_quantize_gb300 as mxq

pytestmark = pytest.mark.gpu
NEG = -np.inf
SCORES = {"softmax": mxq.SOFTMAX, "sigmoid": mxq.SIGMOID}


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    yield
    assert mxq.mx_device_errors() == 0


def cpu(t):
    return t.cpu().numpy()


def bf16_inputs(rng, M, K, special=True):
    """Activations with loud columns, a block of zeros, tiny and huge blocks where there is room."""
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.random(K) < 0.02] *= 50
    if special and M >= 4 and K >= 256:
        x[1, :128] = 0
        x[2, 128:256] *= 2.0 ** -110
        x[3, :] *= 2.0 ** 100
    return torch.from_numpy(x).bfloat16().cuda()


# ---------------------------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------------------------
def spaced_logits(rng, T, E, dtype):
    """Distinct logits per token, spaced so that no rounding reorders scores: a shuffled grid of
    step 1/16 (exact in both types for E <= 256; wider grids use fp32)."""
    grid = (np.arange(E) - E / 2) / 16.0
    l = np.stack([rng.permutation(grid) for _ in range(T)])
    return torch.from_numpy(l).to(dtype).cuda()


ROUTES = [
    # T, E, k, score, bias, groups, top, renorm, scale
    (1, 8, 1, "softmax", False, 1, 1, True, 1.0),
    (1, 128, 8, "softmax", False, 1, 1, True, 1.0),
    (3, 1, 1, "sigmoid", False, 1, 1, False, 1.0),
    (5, 2, 2, "softmax", False, 1, 1, False, 0.5),
    (33, 31, 7, "sigmoid", True, 1, 1, True, 2.5),
    (130, 32, 32, "softmax", False, 1, 1, True, 1.0),
    (257, 60, 6, "softmax", False, 1, 1, False, 16.0),
    (64, 64, 6, "sigmoid", True, 8, 3, True, 1.0),
    (100, 160, 6, "softmax", False, 8, 3, False, 1.0),
    (513, 256, 8, "sigmoid", True, 8, 4, True, 2.5),
    (65, 96, 4, "sigmoid", False, 32, 5, True, 1.0),
    (17, 32, 3, "sigmoid", True, 32, 3, True, 1.0),
    (9, 250, 5, "softmax", False, 5, 1, True, 1.0),
    (31, 1024, 32, "sigmoid", True, 16, 3, True, 1.0),
    (12, 777, 8, "softmax", True, 1, 1, True, 1.0),
]


def bias_for(rng, E, on):
    # multiples of 1/64, so that choices stay as far apart as the scores let them be
    return (rng.integers(-8, 9, E) / 64.0).astype(np.float32) if on else None


def well_separated(l, k, score, bias, groups, top):
    """Tokens whose choice no rounding to fp32 can change: the best choices, and the groups', lie
    apart by far more than the error of a score."""
    s = R.scores(l, score)
    c = s if bias is None else s + bias
    if bias is None and score == "softmax" and groups == 1:
        c = l  # ordered by the logits themselves, which differ by 1/16
    ok = np.ones(l.shape[0], bool)
    if groups > 1:
        two = -np.sort(-c.reshape(l.shape[0], groups, -1), 2)[:, :, :2].sum(2)
        g = -np.sort(-two, 1)
        if top < groups:
            ok &= g[:, top - 1] - g[:, top] > 1e-5
            bar = g[:, top - 1:top]
            c = np.where(np.repeat(two >= bar, l.shape[1] // groups, 1), c, -10.0)
    best = -np.sort(-c, 1)[:, :k + 1]
    return ok & (np.diff(-best, axis=1).min(1) > 1e-5) if best.shape[1] > 1 else ok


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,score,bias,groups,top,renorm,scale", ROUTES)
def test_route(T, E, k, score, bias, groups, top, renorm, scale, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    if dtype == torch.bfloat16 and E > 256:
        pytest.skip("the spaced grid needs more bits")
    logits = spaced_logits(rng, T, E, dtype)
    b = bias_for(rng, E, bias)
    experts, weights = mxq.mx_route(logits, k, SCORES[score],
                                    None if b is None else torch.from_numpy(b).cuda(),
                                    groups=groups, top_groups=top, renormalize=renorm, scale=scale)
    l = logits.cpu().double().numpy()
    want_e, want_w = R.route(l, k, score, None if b is None else b.astype(np.float64), groups, top,
                             renorm, scale)
    got_e, got_w = cpu(experts), cpu(weights).astype(np.float64)
    sure = well_separated(l, k, score, None if b is None else b.astype(np.float64), groups, top)
    if b is None and groups == 1:
        sure[:] = True  # scores keep the order of distinct logits
    assert (got_e[sure] == want_e[sure]).all()
    assert sure.mean() > 0.2 or T < 8 or E > 256
    # exp errs by 2 ulp plus |l - max| <= 64 units of its argument, the sums by at most 40 units,
    # each division by one: under 256 units in all, twice that where renormalised
    assert (np.abs(got_w - want_w)[sure] <= 512 * R.U * np.abs(want_w)[sure] + 1e-37).all()
    # the other tokens: distinct experts
    for row in got_e[~sure][:50]:
        assert len(set(row.tolist())) == k and (row >= 0).all() and (row < E).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest_index(score):
    rng = np.random.default_rng(5)
    for E, k in ((40, 6), (7, 7), (512, 9)):
        l = rng.integers(0, 3, (200, E)).astype(np.float32)
        experts, _ = mxq.mx_route(torch.from_numpy(l).cuda(), k, SCORES[score])
        want, _ = R.route(l.astype(np.float64), k, score)
        assert (cpu(experts) == want).all()


def test_route_equal_groups_go_to_the_lowest_index():
    l = torch.zeros(5, 64, device="cuda")
    l[:, 37] = -1.0
    experts, _ = mxq.mx_route(l, 4, mxq.SIGMOID, groups=8, top_groups=2)
    assert (cpu(experts) == np.array([0, 1, 2, 3])).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_route_masked_experts_are_never_chosen(score, groups, top):
    rng = np.random.default_rng(8)
    T, E, k = 64, 32, 8
    l = np.stack([rng.permutation(np.arange(E) / 16.0) for _ in range(T)])
    l[rng.random((T, E)) < 0.6] = NEG
    l[0] = NEG            # nothing to choose
    l[1] = NEG
    l[1, 17] = 3.0        # one expert left
    l[2, :] = -3.0e38     # the type's lowest values are numbers, not masks
    l[3] = NEG
    l[3, 30:] = 1.0       # the last group only
    experts, weights = mxq.mx_route(torch.from_numpy(l).float().cuda(), k, SCORES[score],
                                    groups=groups, top_groups=top)
    l32 = l.astype(np.float32).astype(np.float64)
    want_e, want_w = R.route(l32, k, score, None, groups, top)
    got = cpu(experts)
    rows = [t for t in range(T) if t != 2]
    assert (got[rows] == want_e[rows]).all()
    assert (got[0] == -1).all() and (cpu(weights)[0] == 0).all()
    assert (got[2] >= 0).all()
    assert np.abs(cpu(weights)[rows] - want_w[rows]).max() < 512 * R.U
    assert np.isfinite(cpu(weights)).all()


def test_route_bias_of_minus_infinity_and_nan_logits():
    rng = np.random.default_rng(9)
    l = torch.from_numpy(np.stack([rng.permutation(np.arange(16) / 4.0) for _ in range(4)])).float()
    bias = torch.zeros(16)
    bias[[3, 5]] = NEG
    experts, _ = mxq.mx_route(l.cuda(), 14, mxq.SIGMOID, bias.cuda())
    assert not (set(cpu(experts).ravel().tolist()) & {3, 5})
    l[1, 2] = float("nan")
    experts, weights = mxq.mx_route(l.cuda(), 15, mxq.SIGMOID, renormalize=False)
    e, w = cpu(experts), cpu(weights)
    assert 2 not in e[1] and np.isfinite(w).all()  # a NaN ranks below every number
    experts, weights = mxq.mx_route(l.cuda(), 3)
    assert np.isnan(cpu(weights)[1]).all() and np.isfinite(cpu(weights)[[0, 2, 3]]).all()
    assert ((cpu(experts) >= 0) & (cpu(experts) < 16)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (7, 1, 1), (65, 33, 5), (130, 256, 8), (3, 1024, 32)])
def test_route_backward(T, E, k, score, renorm, dtype):
    rng = np.random.default_rng(T + E)
    logits = (torch.from_numpy(rng.standard_normal((T, E))) * 2).to(dtype).cuda()
    experts, _ = mxq.mx_route(logits, k, SCORES[score], renormalize=renorm, scale=1.5)
    g = torch.from_numpy(rng.standard_normal((T, k))).float().cuda()
    got = mxq.mx_route_backward(g, logits, experts, SCORES[score], renormalize=renorm, scale=1.5)
    l = logits.cpu().double().requires_grad_(True)
    w = R.chosen_weights(l, experts.cpu(), score, renorm, 1.5)
    (want,) = torch.autograd.grad(w, l, g.cpu().double())
    # magnitudes that cancel: g and <g, w> against the smallest denominator of the token
    p = R.chosen_weights(l.detach(), experts.cpu(), score, False, 1.0)
    P = p.sum(1, keepdim=True) if renorm else torch.ones(T, 1, dtype=torch.float64)
    big = 1.5 * g.cpu().double().abs().sum(1, keepdim=True) / P
    s = torch.from_numpy(R.scores(l.detach().numpy(), score))
    bound = 512 * R.U * big * (s + 1e-30)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
    assert ((got.cpu().double() - want).abs() <= bound + 1e-37).all()


def test_route_backward_against_differences():
    rng = np.random.default_rng(3)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            l = rng.standard_normal((6, 12))
            logits = torch.from_numpy(l).float().cuda()
            experts, _ = mxq.mx_route(logits, 4, SCORES[score], renormalize=renorm)
            g = rng.standard_normal((6, 4)).astype(np.float32)
            got = cpu(mxq.mx_route_backward(torch.from_numpy(g).cuda(), logits, experts,
                                            SCORES[score], renormalize=renorm))
            l = cpu(logits).astype(np.float64)
            h = 1e-5
            for t in range(6):
                for e in range(12):
                    d = []
                    for sign in (1, -1):
                        m = l.copy()
                        m[t, e] += sign * h
                        w = R.chosen_weights(torch.from_numpy(m), experts.cpu(), score, renorm, 1.0)
                        d.append(float((w.numpy()[t] * g[t]).sum()))
                    # central differences err by h^2 times a third derivative below 10
                    assert abs(got[t, e] - (d[0] - d[1]) / (2 * h)) < 1e-5


def test_route_backward_of_no_choice_is_nothing():
    l = torch.full((2, 8), NEG, device="cuda")
    l[1, 3] = 0.5
    experts, _ = mxq.mx_route(l, 2, mxq.SOFTMAX)
    for score in (mxq.SOFTMAX, mxq.SIGMOID):
        for renorm in (True, False):
            d = cpu(mxq.mx_route_backward(torch.ones(2, 2, device="cuda"), l, experts, score,
                                          renormalize=renorm))
            assert (d[0] == 0).all() and np.isfinite(d).all()


@pytest.mark.parametrize("score", [mxq.SOFTMAX, mxq.SIGMOID])
@pytest.mark.parametrize("E", [6, 40, 600])
def test_route_backward_of_choices_named_twice(score, E):
    """No call of the router names an expert twice; the gradient of such weights is the sum."""
    rng = np.random.default_rng(E)
    experts = np.array([[2, 2, 5], [1, 1, 1], [-1, 0, 0], [3, -1, 4]], dtype=np.int32)
    l = rng.standard_normal((4, E)).astype(np.float32)
    g = rng.standard_normal((4, 3)).astype(np.float32)
    got = cpu(mxq.mx_route_backward(torch.from_numpy(g).cuda(), torch.from_numpy(l).cuda(),
                                    torch.from_numpy(experts).cuda(), score, renormalize=False))
    x = l.astype(np.float64)
    if score == mxq.SOFTMAX:
        s = np.exp(x - x.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    else:
        s = 1 / (1 + np.exp(-x))
    for t in range(4):
        d, size = np.zeros(E), np.zeros(E)
        for j, e in enumerate(experts[t]):
            if e >= 0:
                d[e] += g[t, j]
                size[e] += abs(float(g[t, j]))
        if score == mxq.SOFTMAX:
            want, size = s[t] * (d - d @ s[t]), s[t] * (size + size @ s[t])
        else:
            want, size = d * s[t] * (1 - s[t]), size * s[t]
        # exponentials, sums of E and of the choices, divisions and products: under 256 units in all
        assert (np.abs(got[t] - want) <= 256 * R.U * size + 1e-38).all()


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 128), (5, 3, 7), (300, 8, 64),
                                   (128, 4, 9), (128, 8, 40), (205, 5, 40), (511, 8, 1024), (513, 8, 256),
                                   (4096, 1, 3), (9001, 7, 130),
                                   (70000, 4, 17)])
def test_plan(T, k, E):
    rng = np.random.default_rng(T + E)
    experts = rng.integers(0, E, (T, k)).astype(np.int32)
    if T > 3:
        experts[rng.random((T, k)) < 0.1] = -1
        experts[T // 2] = E - 1
        experts[0, 0] = E + 5  # outside: counts as none
    got = mxq.mx_route_plan(torch.from_numpy(experts).cuda(), E)
    for g, w in zip(got, R.plan(experts, E)):
        assert (cpu(g) == w).all()


# ---------------------------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------------------------
SHAPES = [(1, 32), (1, 128), (3, 160), (128, 4096), (129, 256), (257, 1056), (1000, 512), (40, 4160)]


@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize_rows(M, K):
    x = bf16_inputs(np.random.default_rng(M + K), M, K)
    codes, scales = mxq.mx_quantize_b128_rows(x)
    want_c, want_s = R.rows(x)
    assert (cpu(codes) == want_c).all() and (cpu(scales) == want_s).all()


@pytest.mark.parametrize("M,K,rows", [(1, 32, 5), (50, 256, 300), (300, 672, 2000), (7, 128, 1)])
def test_quantize_gathered_rows(M, K, rows):
    rng = np.random.default_rng(M + K)
    x = bf16_inputs(rng, M, K)
    index = rng.integers(0, M, rows).astype(np.int32)
    index[rng.random(rows) < 0.2] = -1
    if rows > 3:
        index[2] = M  # outside: a row of zeros too
    codes, scales = mxq.mx_quantize_b128_rows(x, torch.from_numpy(index).cuda())
    want_c, want_s = R.rows(x, index)
    assert (cpu(codes) == want_c).all() and (cpu(scales) == want_s).all()


@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize_cols(M, K):
    x = bf16_inputs(np.random.default_rng(M * 3 + K), M, K)
    codes, scales = mxq.mx_quantize_b128_cols(x)
    assert codes.shape == (K, R.up(M)) and scales.shape == (R.up(M) // 128, K)
    want_c, want_s = R.cols(x)
    assert (cpu(codes) == want_c).all() and (cpu(scales) == want_s).all()


@pytest.mark.parametrize("M,K,E", [(2500, 4128, 0), (9000, 1056, 40)])
def test_quantize_cols_many_tiles(M, K, E):
    """More tiles than resident CTAs: every one walks several, over ends of blocks and of experts."""
    rng = np.random.default_rng(M)
    x = bf16_inputs(rng, M, K)
    offsets = None
    if E:
        offsets = np.concatenate([[0], np.sort(rng.integers(0, M, E - 1)), [M]]).astype(np.int64)
        offsets[5] = offsets[4]  # an expert without rows
    codes, scales = mxq.mx_quantize_b128_cols(
        x, None, None if offsets is None else torch.from_numpy(offsets).cuda())
    want_c, want_s = R.cols(x, None, offsets)
    n = want_s.shape[0]  # blocks that belong to experts
    assert (cpu(codes)[:, :n * 128] == want_c[:, :n * 128]).all() and (cpu(scales)[:n] == want_s).all()


def test_quantize_cols_contract_breaking_offsets_stay_inside():
    x = bf16_inputs(np.random.default_rng(1), 100, 128)
    P = mxq.mx_b128_padded_rows(100, 3)
    codes = torch.full((130, P), 5, device="cuda", dtype=torch.uint8)
    scales = torch.full((P // 128 + 2, 128), 5.0, device="cuda")
    for off in ([0, 90, 40, 1000], [-5, 10, 2 ** 40, 7], [50, 20, 10, 0], [0, 100, 0, 100]):
        mxq.mx_quantize_b128_cols(x, None, torch.tensor(off, device="cuda"), codes=codes[1:129],
                                  scales=scales[1:-1])
    torch.cuda.synchronize()
    assert (codes[0] == 5).all() and (codes[129] == 5).all()
    assert (scales[0] == 5).all() and (scales[-1] == 5).all()


@pytest.mark.parametrize("counts", [[0, 5, 0, 300, 128], [1], [0, 0], [129, 1, 127, 0, 64, 256]])
@pytest.mark.parametrize("gather", [False, True])
def test_quantize_cols_by_expert(counts, gather):
    rng = np.random.default_rng(len(counts))
    rows, K = sum(counts), 288
    x = bf16_inputs(rng, 200 if gather else rows, K)
    index = rng.integers(-1, 200, rows + 3).astype(np.int32) if gather else None
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    codes, scales = mxq.mx_quantize_b128_cols(
        x, None if index is None else torch.from_numpy(index).cuda(), torch.from_numpy(offsets).cuda())
    want_c, want_s = R.cols(x, index, offsets)
    n = want_c.shape[1]
    assert (cpu(codes)[:, :n] == want_c).all() and (cpu(scales)[:n // 128] == want_s).all()


@pytest.mark.parametrize("shape", [(1, 32), (128, 128), (130, 160), (300, 1056), (64, 4096),
                                   (3, 200, 288), (2, 128, 256)])
def test_quantize_blocks(shape):
    rng = np.random.default_rng(sum(shape))
    B = shape[0] if len(shape) == 3 else 1
    x = torch.stack([bf16_inputs(rng, *shape[-2:]) for _ in range(B)]).view(shape)
    codes, scales, codes_t, scales_t = mxq.mx_quantize_b128_blocks(x, transpose=True)
    alone = mxq.mx_quantize_b128_blocks(x)
    for i in range(B):
        want_c, want_s = R.quantize(R.f32(x.view(B, *shape[-2:])[i]), 128, 128)
        at = (lambda t: cpu(t.view(B, *t.shape[-2:])[i]))
        assert (at(codes) == want_c).all() and (at(scales) == want_s).all()
        assert (at(codes_t) == want_c.T).all() and (at(scales_t) == want_s.T).all()
        assert (at(alone[0]) == want_c).all() and (at(alone[1]) == want_s).all()


def test_quantize_nan_and_infinity():
    x = torch.ones(4, 256, device="cuda", dtype=torch.bfloat16)
    x[0, 5] = float("nan")
    x[1, 130] = float("-inf")
    codes, scales = (cpu(t) for t in mxq.mx_quantize_b128_rows(x))
    assert (codes[0, :128] == 0x7F).all() and (codes[1, 128:] == 0x7F).all()
    assert np.isnan(scales[0, 0]) and np.isnan(scales[1, 1])
    assert np.isfinite(scales[1, 0]) and (codes[2:] == 0x7E).all()
    codes, scales = (cpu(t) for t in mxq.mx_quantize_b128_cols(x))
    assert (codes[5, :128] == 0x7F).all() and np.isnan(scales[0, 130]) and np.isfinite(scales[0, 6])
    codes, scales = (cpu(t) for t in mxq.mx_quantize_b128_blocks(x))
    assert (codes == 0x7F).all() and np.isnan(scales).all()
    # a NaN row reaches its row of the product and no other
    b = mxq.mx_quantize_b128_blocks(torch.ones(64, 256, device="cuda", dtype=torch.bfloat16))
    c = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(x), *b).float().cpu()
    assert c[:2].isnan().all() and (c[2:] == 256).all()


# ---------------------------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------------------------
def operand(rng, M, K, form, loud=True):
    """Random codes of every finite value, scales over a few binades -> device tensors, values."""
    codes = rng.integers(0, 256, (M, K), dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] ^= 1
    kb = -(-K // 128)
    shape = (kb, M) if form == "rows" else (-(-M // 128), kb)
    scales = np.exp2(rng.uniform(-12, 3, shape)).astype(np.float32)
    return (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()), \
        R.values(codes, scales, form)


def check_product(C, a, b, K, what=""):
    want, S = R.product(a, b)
    bound = R.product_bound(want, S, K, C.dtype == torch.bfloat16)
    err = np.abs(C.double().cpu().numpy() - want)
    assert (err <= bound).all(), (what, (err / bound).max(), np.argwhere(~(err <= bound))[:3])


DENSE = [(1, 8, 32), (1, 128, 128), (2, 136, 160), (7, 264, 4096), (16, 256, 1024), (17, 512, 96),
         (33, 1024, 640), (64, 128, 2048), (65, 384, 256), (100, 1000, 512), (128, 256, 128),
         (129, 264, 384), (200, 2048, 1056), (257, 520, 2080), (300, 776, 1024), (513, 1280, 768),
         (1, 4096, 8192), (1024, 4104, 512)]


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("form", ["blocks", "rows"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm(M, N, K, form, dtype):
    rng = np.random.default_rng(M + N + K)
    (ac, asc), a = operand(rng, M, K, "rows")
    (bc, bsc), b = operand(rng, N, K, form)
    C = mxq.mx_gemm_b128(ac, asc, bc, bsc, mxq.B128_ROWS if form == "rows" else mxq.B128_BLOCKS,
                         out_dtype=dtype)
    assert C.dtype == dtype and C.shape == (M, N)
    check_product(C, a, b, K)


def test_gemm_of_quantized_operands_and_identity():
    rng = np.random.default_rng(1)
    x = bf16_inputs(rng, 300, 512, special=False)
    xq = mxq.mx_quantize_b128_rows(x)
    eye = torch.zeros(512, 512, dtype=torch.uint8, device="cuda")
    eye[range(512), range(512)] = 0x38  # 1.0
    C = mxq.mx_gemm_b128(*xq, eye, torch.ones(4, 4, device="cuda"), out_dtype=torch.float32)
    # one product per entry: the operand's own values, each one fp32 rounding
    want = R.values(cpu(xq[0]), cpu(xq[1]), "rows")
    assert (cpu(C) == want.astype(np.float32)).all()


def test_gemm_writes_nothing_beside_its_output():
    rng = np.random.default_rng(2)
    for M, N, K in ((5, 136, 256), (130, 264, 128), (70, 8, 64)):
        (ac, asc), a = operand(rng, M, K, "rows")
        (bc, bsc), b = operand(rng, N, K, "blocks")
        buf = torch.full(((M + 2) * N + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
        c = buf[N:N + M * N].view(M, N) if (N * 2) % 16 == 0 else None
        mxq.mx_gemm_b128(ac, asc, bc, bsc, c=c)
        check_product(c, a, b, K)
        assert (buf[:N] == 7).all() and (buf[N + M * N:] == 7).all()


GROUPS = [[5], [0, 3, 0], [128, 1, 127, 0, 300], [1] * 40, [0] * 7 + [260], [16, 17, 15, 33, 64, 65],
          [700, 2, 0, 90]]


@pytest.mark.parametrize("counts", GROUPS)
@pytest.mark.parametrize("N,K", [(128, 128), (264, 416), (1024, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_grouped(counts, N, K, dtype):
    rng = np.random.default_rng(len(counts) + N)
    E, rows = len(counts), sum(counts) + 3  # three rows past the last expert's
    (ac, asc), a = operand(rng, rows, K, "rows")
    bs = [operand(rng, N, K, "blocks") for _ in range(E)]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    c = torch.full((rows, N), 3.0, device="cuda", dtype=dtype)
    mxq.mx_gemm_b128_grouped(ac, asc, torch.stack([b[0][0] for b in bs]),
                             torch.stack([b[0][1] for b in bs]), torch.from_numpy(offsets).cuda(), c=c)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            check_product(c[lo:hi], a[lo:hi], bs[e][1], K, e)
    assert (c[offsets[-1]:] == 3).all()


@pytest.mark.parametrize("counts", GROUPS)
@pytest.mark.parametrize("M,N", [(32, 64), (160, 264), (512, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_grouped_wgrad(counts, M, N, dtype):
    rng = np.random.default_rng(len(counts) + M)
    rows = sum(counts)
    dy, x = bf16_inputs(rng, rows, M, False), bf16_inputs(rng, rows, N, False) if N % 32 == 0 else None
    if x is None:
        N = 256
        x = bf16_inputs(rng, rows, N, False)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    off = torch.from_numpy(offsets).cuda()
    C = mxq.mx_gemm_b128_grouped_wgrad(*mxq.mx_quantize_b128_cols(dy, None, off),
                                       *mxq.mx_quantize_b128_cols(x, None, off), off, out_dtype=dtype)
    assert C.shape == (len(counts), M, N)
    for e, n in enumerate(counts):
        if n == 0:
            assert (C[e] == 0).all()
            continue
        part = slice(offsets[e], offsets[e + 1])
        u = R.values(*R.cols(dy[part]), "rows")
        v = R.values(*R.cols(x[part]), "rows")
        check_product(C[e], u, v, R.up(n), e)


@pytest.mark.parametrize("E,most,N,K", [(96, 40, 520, 2016), (40, 300, 264, 1568), (1024, 3, 128, 160)])
def test_gemm_grouped_many_tiles_and_steps(E, most, N, K):
    """More tiles than CTAs and more steps than stages, in both sizes of tiles."""
    rng = np.random.default_rng(E)
    counts = rng.integers(0, most + 1, E)
    (ac, asc), a = operand(rng, int(counts.sum()), K, "rows")
    bs = [operand(rng, N, K, "blocks") for _ in range(E)]
    bc, bsc = torch.stack([b[0][0] for b in bs]), torch.stack([b[0][1] for b in bs])
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    c = mxq.mx_gemm_b128_grouped(ac, asc, bc, bsc, torch.from_numpy(offsets).cuda())
    for e in range(E):
        part = slice(offsets[e], offsets[e + 1])
        if counts[e]:
            check_product(c[part], a[part], bs[e][1], K, e)


def test_gemm_grouped_contract_breaking_offsets_stay_inside():
    rng = np.random.default_rng(4)
    (ac, asc), _ = operand(rng, 100, 128, "rows")
    bs = [operand(rng, 128, 128, "blocks")[0] for _ in range(3)]
    b = torch.stack([q[0] for q in bs]), torch.stack([q[1] for q in bs])
    buf = torch.full((102 * 128,), 5.0, device="cuda", dtype=torch.bfloat16)
    c = buf[128:128 + 100 * 128].view(100, 128)
    for off in ([0, 90, 40, 1000], [-5, 10, 2 ** 40, 7], [50, 20, 10, 0]):
        mxq.mx_gemm_b128_grouped(ac, asc, *b, torch.tensor(off, device="cuda"), c=c)
    torch.cuda.synchronize()
    assert (buf[:128] == 5).all() and (buf[128 + 100 * 128:] == 5).all()


def test_training_step_of_a_layer():
    """y, dx and dw from the three forms of quantised operands, against 64-bit products."""
    rng = np.random.default_rng(6)
    M, N, K = 200, 160, 288
    x, w = bf16_inputs(rng, M, K, False), bf16_inputs(rng, N, K, False)
    dy = bf16_inputs(rng, M, N, False)
    wq, ws, wtq, wts = mxq.mx_quantize_b128_blocks(w, transpose=True)
    y = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(x), wq, ws)
    dx = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(dy), wtq, wts)
    dw = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_cols(dy), *mxq.mx_quantize_b128_cols(x),
                          mxq.B128_ROWS, out_dtype=torch.float32)
    wv = R.values(*R.quantize(R.f32(w), 128, 128), "blocks")
    check_product(y, R.values(*R.rows(x), "rows"), wv, K)
    check_product(dx, R.values(*R.rows(dy), "rows"), wv.T, N)
    check_product(dw, R.values(*R.cols(dy), "rows"), R.values(*R.cols(x), "rows"), M)
    # and near the unquantised products: E4M3 errs by at most 2^-4 of an element
    exact = R.f32(x).astype(np.float64) @ R.f32(w).astype(np.float64).T
    assert np.linalg.norm(y.float().cpu().numpy() - exact) < 0.1 * np.linalg.norm(exact)


# ---------------------------------------------------------------------------------------------
# combination
# ---------------------------------------------------------------------------------------------
COMBINES = [(1, 1, 8), (1, 8, 2048), (16, 8, 2048), (3, 2, 136), (50, 3, 1000), (200, 5, 264),
            (33, 9, 4096), (5, 64, 64), (1000, 4, 128)]


def combine_case(T, k, N, seed):
    rng = np.random.default_rng(seed)
    rows = T * k
    y = bf16_inputs(rng, rows, N, False)
    slots = rng.permutation(rows).reshape(T, k).astype(np.int32)
    if T > 2:
        slots[rng.random((T, k)) < 0.15] = -1
        slots[1] = -1
        slots[0, 0] = rows + 4  # outside: none
    w = rng.standard_normal((T, k)).astype(np.float32)
    return y, slots, w


@pytest.mark.parametrize("T,k,N", COMBINES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, N, weighted):
    y, slots, w = combine_case(T, k, N, T + N)
    out = mxq.mx_combine(y, torch.from_numpy(slots).cuda(),
                         torch.from_numpy(w).cuda() if weighted else None)
    v = R.f32(y).astype(np.float64)
    ok = (slots >= 0) & (slots < T * k)
    rows = v[np.where(ok, slots, 0)] * ((w if weighted else np.ones_like(w)) * ok)[:, :, None]
    want, S = rows.sum(1), np.abs(rows).sum(1)
    bound = 2.0 ** -8 * np.abs(want) + 2 * k * R.U * S + 1e-38
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("T,k,N", COMBINES)
def test_combine_backward(T, k, N):
    y, slots, w = combine_case(T, k, N, T + N)
    rng = np.random.default_rng(T)
    dout = bf16_inputs(rng, T, N, False)
    dy = torch.full((T * k, N), 9.0, device="cuda", dtype=torch.bfloat16)
    _, dw = mxq.mx_combine_backward(dout, y, torch.from_numpy(slots).cuda(),
                                    torch.from_numpy(w).cuda(), dy=dy)
    v, d = R.f32(y).astype(np.float64), R.f32(dout).astype(np.float64)
    got_dy, got_dw = dy.double().cpu().numpy(), cpu(dw)
    named = np.zeros(T * k, bool)
    for t in range(T):
        for j in range(k):
            r = slots[t, j]
            if r < 0 or r >= T * k:
                assert got_dw[t, j] == 0
                continue
            named[r] = True
            want = w[t, j] * d[t]
            assert (np.abs(got_dy[r] - want) <= 2.0 ** -8 * np.abs(want) + 1e-38).all()
            S = np.abs(d[t] * v[r]).sum()
            assert abs(got_dw[t, j] - d[t] @ v[r]) <= N * R.U * S + 1e-38
    assert (got_dy[~named] == 9).all()


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------
def test_on_a_side_stream_and_in_a_graph():
    """The whole chain on a stream of its own, then captured and replayed on new inputs."""
    rng = np.random.default_rng(11)
    T, E, k, N, K = 40, 6, 2, 256, 256
    x = bf16_inputs(rng, T, K, False)
    logits = spaced_logits(rng, T, E, torch.float32)
    w = mxq.mx_quantize_b128_blocks(
        torch.stack([bf16_inputs(rng, N, K, False) for _ in range(E)]))

    def layer():
        experts, weights = mxq.mx_route(logits, k)
        offsets, tokens, slots = mxq.mx_route_plan(experts, E)
        y = mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(x, tokens), *w, offsets)
        return mxq.mx_combine(y, slots, weights)

    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = layer()
    side.synchronize()
    assert torch.equal(on_side, want)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, want)
    logits.copy_(spaced_logits(rng, T, E, torch.float32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, layer())


@pytest.mark.parametrize("raw", [False, True])
def test_stream_argument(raw):
    """Every call on a stream passed as an object or as a handle."""
    rng = np.random.default_rng(14)
    T, E, k, N, K = 700, 6, 2, 128, 256
    x, dout = bf16_inputs(rng, T, K, False), bf16_inputs(rng, T, N, False)
    logits = spaced_logits(rng, T, E, torch.float32)
    weight = torch.stack([bf16_inputs(rng, N, K, False) for _ in range(E)])

    def layer(**at):
        experts, weights = mxq.mx_route(logits, k, **at)
        offsets, tokens, slots = mxq.mx_route_plan(experts, E, **at)
        wc, ws, wct, wst = mxq.mx_quantize_b128_blocks(weight, transpose=True, **at)
        y = mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(x, tokens, **at), wc, ws, offsets, **at)
        out = mxq.mx_combine(y, slots, weights, **at)
        dy, dweights = mxq.mx_combine_backward(dout, y, slots, weights, **at)
        dw = mxq.mx_gemm_b128_grouped_wgrad(*mxq.mx_quantize_b128_cols(dy, None, offsets, **at),
                                            *mxq.mx_quantize_b128_cols(x, tokens, offsets, **at),
                                            offsets, **at)
        one = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(x, **at), wc[0], ws[0], **at)
        return out, dy, dw, one, mxq.mx_route_backward(dweights, logits, experts, **at)

    want = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = layer(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(12)
    (ac, asc), _ = operand(rng, 70, 2048, "rows")
    (bc, bsc), _ = operand(rng, 512, 2048, "blocks")
    first = mxq.mx_gemm_b128(ac, asc, bc, bsc, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(first, mxq.mx_gemm_b128(ac, asc, bc, bsc, out_dtype=torch.float32))


@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("limit", [1, 1000, 20000])
def test_give_up_leaves_the_context_usable(M, limit):
    rng = np.random.default_rng(13)
    (ac, asc), a = operand(rng, M, 2048, "rows")
    (bc, bsc), b = operand(rng, 1024, 2048, "blocks")
    mxq.mx_selftest_gemm_b128_give_up(ac, asc, bc, bsc, limit)
    assert mxq.mx_device_errors() in (0, 1)
    if limit == 1:
        mxq.mx_selftest_gemm_b128_give_up(ac, asc, bc, bsc, limit)
        assert mxq.mx_device_errors() == 1
    check_product(mxq.mx_gemm_b128(ac, asc, bc, bsc), a, b, 2048)
    assert mxq.mx_device_errors() == 0


# ---------------------------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------------------------
def test_refusals():
    x = torch.zeros(4, 256, device="cuda", dtype=torch.bfloat16)
    l = torch.zeros(4, 8, device="cuda")
    i32 = dict(device="cuda", dtype=torch.int32)
    with pytest.raises(TypeError):
        mxq.mx_route(l.double(), 2)
    with pytest.raises(TypeError):
        mxq.mx_route(l.cpu(), 2)
    with pytest.raises(ValueError):
        mxq.mx_route(l.t(), 2)
    with pytest.raises(ValueError):
        mxq.mx_route(l, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(mxq.MXError):
        mxq.mx_route(l, 9)
    with pytest.raises(mxq.MXError):
        mxq.mx_route(l, 2, groups=3)
    with pytest.raises(mxq.MXError):
        mxq.mx_route(l, 5, groups=4, top_groups=2)
    with pytest.raises(ValueError):
        mxq.mx_route_backward(torch.zeros(4, 3, device="cuda"), l, torch.zeros(4, 2, **i32))
    with pytest.raises(TypeError):
        mxq.mx_route_plan(torch.zeros(4, 2, device="cuda", dtype=torch.int64), 8)
    with pytest.raises(TypeError):
        mxq.mx_quantize_b128_rows(x.float())
    with pytest.raises(mxq.MXError):
        mxq.mx_quantize_b128_rows(torch.zeros(2, 40, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        mxq.mx_quantize_b128_rows(x, torch.zeros(4, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError):
        mxq.mx_quantize_b128_rows(x, scales=torch.zeros(3, device="cuda"))
    a, b = mxq.mx_quantize_b128_rows(x), mxq.mx_quantize_b128_blocks(x)
    with pytest.raises(ValueError):
        mxq.mx_gemm_b128(*a, *a)  # rows-form scales of B given as blocks
    with pytest.raises(TypeError):
        mxq.mx_gemm_b128(*a, *b, out_dtype=torch.float16)
    with pytest.raises(mxq.MXError):
        mxq.mx_gemm_b128(*a, *b)  # N = 4
    with pytest.raises(ValueError):
        mxq.mx_gemm_b128_grouped(*a, *b, torch.zeros(2, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError):
        mxq.mx_combine(x, torch.zeros(2, 2, **i32), torch.zeros(2, 3, device="cuda"))
    with pytest.raises(ValueError):
        mxq.mx_combine_backward(x, x, torch.zeros(2, 2, **i32), torch.zeros(2, 2, device="cuda"))


# ---------------------------------------------------------------------------------------------
# tensors of more than 2^31 elements: the far end against a small call on a copy of it
# ---------------------------------------------------------------------------------------------
FAR, WIDE = 1_100_000, 2048


def far_rows(n):
    x = torch.zeros(FAR, WIDE, device="cuda", dtype=torch.bfloat16)
    x[-n:] = bf16_inputs(np.random.default_rng(n), n, WIDE, False)
    return x


def test_far_end_of_quantised_rows_and_columns():
    x = far_rows(300)
    near = x[-300:].clone()
    want_c, want_s = mxq.mx_quantize_b128_rows(near)
    codes, scales = mxq.mx_quantize_b128_rows(x)
    assert torch.equal(codes[-300:], want_c) and torch.equal(scales[:, -300:], want_s)
    del codes, scales
    index = torch.arange(FAR - 300, FAR, device="cuda", dtype=torch.int32)
    codes, scales = mxq.mx_quantize_b128_rows(x, index)
    assert torch.equal(codes, want_c) and torch.equal(scales, want_s)
    del codes, scales
    offsets = torch.tensor([0, FAR - 300, FAR], device="cuda")
    codes, scales = mxq.mx_quantize_b128_cols(x, None, offsets)
    want_c, want_s = mxq.mx_quantize_b128_cols(near)
    at = -(-(FAR - 300) // 128)
    assert torch.equal(codes[:, at * 128:at * 128 + 384], want_c)
    assert torch.equal(scales[at:at + 3], want_s)


def test_far_end_of_squares():
    x = far_rows(256).view(FAR // 16, 16 * WIDE)
    codes, scales, codes_t, scales_t = mxq.mx_quantize_b128_blocks(x, transpose=True)
    start = (x.shape[0] - 1) // 128 * 128
    want = mxq.mx_quantize_b128_blocks(x[start:].clone(), transpose=True)
    assert torch.equal(codes[start:], want[0]) and torch.equal(scales[-1:], want[1])
    assert torch.equal(codes_t[:, start:], want[2]) and torch.equal(scales_t[:, -1:], want[3])


def test_far_end_of_products():
    rng = np.random.default_rng(5)
    (bc, bsc), b = operand(rng, WIDE, 128, "blocks")
    (ac, asc), a = operand(rng, 300, 128, "rows")
    codes = torch.zeros(FAR, 128, device="cuda", dtype=torch.uint8)
    scales = torch.ones(1, FAR, device="cuda")
    codes[-300:], scales[:, -300:] = ac, asc
    check_product(mxq.mx_gemm_b128(codes, scales, bc, bsc)[-300:], a, b, 128)
    for offsets in ([0, FAR], [0, FAR - 300, FAR - 100, FAR]):
        E = len(offsets) - 1
        c = mxq.mx_gemm_b128_grouped(codes, scales, bc.expand(E, -1, -1).contiguous(),
                                     bsc.expand(E, -1, -1).contiguous(),
                                     torch.tensor(offsets, device="cuda"))
        check_product(c[-300:], a, b, 128)
        del c


def test_far_end_of_combined_rows():
    y, dout = far_rows(6), bf16_inputs(np.random.default_rng(1), 3, WIDE, False)
    near = y[-6:].clone()
    small = torch.tensor([[5, 0], [1, -1], [3, 4]], device="cuda", dtype=torch.int32)
    slots = torch.where(small >= 0, small + (FAR - 6), small)
    weights = torch.rand(3, 2, device="cuda")
    assert torch.equal(mxq.mx_combine(y, slots, weights), mxq.mx_combine(near, small, weights))
    dy = torch.zeros_like(y)
    dy, dw = mxq.mx_combine_backward(dout, y, slots, weights, dy=dy)
    want_y, want_w = mxq.mx_combine_backward(dout, near, small, weights, dy=torch.zeros_like(near))
    assert torch.equal(dy[-6:], want_y) and torch.equal(dw, want_w) and not dy[:-6].any()


def test_far_end_of_routed_tokens():
    T, E = 2_200_000, 1024
    logits = torch.zeros(T, E, device="cuda", dtype=torch.bfloat16)
    logits[-5:] = bf16_inputs(np.random.default_rng(2), 5, E, False)
    near = logits[-5:].clone()
    experts, weights = mxq.mx_route(logits, 4)
    want_e, want_w = mxq.mx_route(near, 4)
    assert torch.equal(experts[-5:], want_e) and torch.equal(weights[-5:], want_w)
    g = torch.rand(T, 4, device="cuda")
    assert torch.equal(mxq.mx_route_backward(g, logits, experts)[-5:],
                       mxq.mx_route_backward(g[-5:].clone(), near, want_e))


def test_far_end_of_experts():
    rng = np.random.default_rng(9)
    E, N, K = 1024, 1056, 2048
    (bc, bsc), b = operand(rng, N, K, "blocks")
    (ac, asc), a = operand(rng, 140, K, "rows")
    codes = torch.zeros(E, N, K, device="cuda", dtype=torch.uint8)
    scales = torch.ones(E, *bsc.shape, device="cuda")
    codes[-1], scales[-1] = bc, bsc
    for counts in ([0] * (E - 1) + [140], [0] * (E - 2) + [130, 10]):
        offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), device="cuda")
        c = mxq.mx_gemm_b128_grouped(ac, asc, codes, scales, offsets)
        n = counts[-1]
        check_product(c[-n:], a[-n:], b, K)
    del codes
    dy, x = bf16_inputs(rng, 140, N, False), bf16_inputs(rng, 140, K, False)
    offsets = torch.tensor([0] * E + [140], device="cuda")
    dw = mxq.mx_gemm_b128_grouped_wgrad(*mxq.mx_quantize_b128_cols(dy, None, offsets),
                                        *mxq.mx_quantize_b128_cols(x, None, offsets), offsets)
    one = mxq.mx_gemm_b128_grouped_wgrad(*mxq.mx_quantize_b128_cols(dy), *mxq.mx_quantize_b128_cols(x),
                                         torch.tensor([0, 140], device="cuda"))
    assert torch.equal(dw[-1], one[0]) and not dw[:-1].any()
