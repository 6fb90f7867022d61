"""The expert-layer operators where their kernels' own edges are: parts of a contraction joined by many
CTAs, CTAs that walk several tiles, rows that no choice names, confident routers, scales at the ends of
their range, streams that are not ordered after one another. Definitions and bounds as in
test_gpu_expert.py."""

import numpy as np
import pytest
import torch

import __graft_entry__
import expert_ref as R
import mx_microscaling_quantize_gb300 as mxq
from test_gpu_expert import bf16_inputs, check_product, cpu, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    yield
    assert mxq.mx_device_errors() == 0


# ---------------------------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------------------------
def dense(M, N, K, form, dtype):
    rng = np.random.default_rng(M + N + K)
    (ac, asc), a = operand(rng, M, K, "rows")
    (bc, bsc), b = operand(rng, N, K, form)
    C = mxq.mx_gemm_b128(ac, asc, bc, bsc, mxq.B128_ROWS if form == "rows" else mxq.B128_BLOCKS,
                         out_dtype=dtype)
    check_product(C, a, b, K)
    return C, (ac, asc, bc, bsc)


@pytest.mark.parametrize("M,N,K", [(128, 4096, 4096), (113, 4096, 4096), (300, 776, 1024)])
@pytest.mark.parametrize("form", ["blocks", "rows"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_parts_of_wide_tiles(M, N, K, form, dtype):
    """More than 64 tokens a tile and the contraction over four CTAs: each writes two groups of columns
    of every warp, through the same staging."""
    C, operands = dense(M, N, K, form, dtype)
    for _ in range(20):
        again = mxq.mx_gemm_b128(*operands, mxq.B128_ROWS if form == "rows" else mxq.B128_BLOCKS,
                                 out_dtype=dtype)
        assert torch.equal(again, C)


@pytest.mark.parametrize("K", [32, 416])
def test_pairs_of_few_steps_one_after_another(K):
    """Pairs whose contraction is over before their stages are used twice (or just after), launch upon
    launch: each leaves only after everything that the other CTA sends it has arrived."""
    rng = np.random.default_rng(K)
    counts = [300, 0, 129, 700]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    off = torch.from_numpy(offsets).cuda()
    (ac, asc), a = operand(rng, sum(counts), K, "rows")
    bs = [operand(rng, 520, K, "blocks") for _ in counts]
    bc, bsc = torch.stack([b[0][0] for b in bs]), torch.stack([b[0][1] for b in bs])
    few = torch.tensor([0, 100, 100, 228, 229], device="cuda")  # rows of the weight gradients
    u, v = (mxq.mx_quantize_b128_cols(bf16_inputs(rng, 229, n, False), None, few) for n in (288, 512))
    c = mxq.mx_gemm_b128_grouped(ac, asc, bc, bsc, off)
    w = mxq.mx_gemm_b128_grouped_wgrad(*u, *v, few)
    for e in range(len(counts)):
        part = slice(offsets[e], offsets[e + 1])
        if counts[e]:
            check_product(c[part], a[part], bs[e][1], K, e)
    outs = [(mxq.mx_gemm_b128_grouped(ac, asc, bc, bsc, off), mxq.mx_gemm_b128_grouped_wgrad(*u, *v, few))
            for _ in range(100)]
    for c2, w2 in outs:
        assert torch.equal(c2, c) and torch.equal(w2, w)


# By the rule of the dense products' shapes: more 128-row tiles of weights than CTAs, one walk of the
# contraction each, and still fewer waves than 256 x 256 tiles on pairs take.
@pytest.mark.parametrize("M,N,K", [(3, 40000, 416), (64, 32768, 1056), (100, 24000, 544), (17, 20488, 96)])
@pytest.mark.parametrize("form", ["blocks", "rows"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_of_few_tokens_and_several_tiles_per_cta(M, N, K, form, dtype):
    """A CTA's barriers, scales and staging go on from one tile to the next, whole batches or not."""
    dense(M, N, K, form, dtype)


def check_give_up(call, check, limit):
    call(limit)
    assert mxq.mx_device_errors() in (0, 1)
    if limit == 1:
        call(limit)
        assert mxq.mx_device_errors() == 1
    check()
    assert mxq.mx_device_errors() == 0


@pytest.mark.parametrize("form", ["blocks", "rows"])
@pytest.mark.parametrize("limit", [1, 1000, 20000])
def test_give_up_of_pairs(form, limit):
    """2048 x 2048 x 2048: 64 tiles on pairs in one wave, against 256 tiles of the other shape in two."""
    rng = np.random.default_rng(17)
    (ac, asc), a = operand(rng, 2048, 2048, "rows")
    (bc, bsc), b = operand(rng, 2048, 2048, form)
    f = mxq.B128_ROWS if form == "rows" else mxq.B128_BLOCKS
    check_give_up(lambda ns: mxq.mx_selftest_gemm_b128_give_up(ac, asc, bc, bsc, ns, f),
                  lambda: check_product(mxq.mx_gemm_b128(ac, asc, bc, bsc, f), a, b, 2048), limit)


@pytest.mark.parametrize("counts", [[300, 0, 129, 1000], [5, 128, 0, 77] * 20])  # pairs; single CTAs
@pytest.mark.parametrize("limit", [1, 1000, 20000])
def test_give_up_by_expert(counts, limit):
    rng = np.random.default_rng(18)
    N, K = 1024, 2048
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    off = torch.from_numpy(offsets).cuda()
    (ac, asc), a = operand(rng, sum(counts), K, "rows")
    (bc, bsc), b = operand(rng, N, K, "blocks")
    bc, bsc = (t.expand(len(counts), -1, -1).contiguous() for t in (bc, bsc))
    check_give_up(lambda ns: mxq.mx_selftest_gemm_b128_grouped_give_up(ac, asc, bc, bsc, off, ns),
                  lambda: check_product(mxq.mx_gemm_b128_grouped(ac, asc, bc, bsc, off), a, b, K), limit)


# ---------------------------------------------------------------------------------------------
# streams that nothing orders after one another
# ---------------------------------------------------------------------------------------------
def test_plans_on_two_streams_at_once():
    """Each stream's workspaces are its own, whatever the other has queued."""
    rng = np.random.default_rng(3)
    cases = []
    for T in (700, 9001):
        experts = rng.integers(-1, 64, (T, 4)).astype(np.int32)
        cases.append((torch.from_numpy(experts).cuda(), R.plan(experts, 64)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        if i % 10 == 0:
            torch.cuda._sleep(200_000)  # the current stream falls behind
        for j, (experts, _) in enumerate(cases):
            got.append((j, mxq.mx_route_plan(experts, 64)))
            got.append((j, mxq.mx_route_plan(experts, 64, stream=side if i % 2 else side.cuda_stream)))
    torch.cuda.synchronize()
    for j, plan in got:
        for g, w in zip(plan, cases[j][1]):
            assert (cpu(g) == w).all()


def test_outputs_of_another_stream_are_not_memory_still_in_use():
    """The current stream has writes queued into blocks that were given back: outputs of a call on
    another stream, which runs at once, are not among them. Nor does the other stream take an output
    back while the current stream still reads it."""
    rng = np.random.default_rng(4)
    x = bf16_inputs(rng, 640, 512, False)
    logits = torch.from_numpy(rng.standard_normal((640, 16))).float().cuda()

    def work(**at):
        experts, weights = mxq.mx_route(logits, 2, **at)
        offsets, tokens, slots = mxq.mx_route_plan(experts, 16, **at)
        codes, scales = mxq.mx_quantize_b128_rows(x, tokens, **at)
        return [experts, weights, offsets, tokens, slots, codes, scales,
                *mxq.mx_quantize(x, mxq.E4M3, **at), mxq.mx_combine(x, slots, weights, **at)]

    side = torch.cuda.Stream()
    want = [t.clone() for t in work()]
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)  # the current stream is busy for some milliseconds
        junk = [torch.empty_like(t) for t in want]
        for t in junk:
            t.view(torch.uint8).fill_(0x33)
        del junk, t
        got = work(stream=side)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
        torch.cuda._sleep(20_000_000)
        kept = [g.clone() for g in got]  # queued behind the pause
        del got, g
        work(stream=side)                # would take the blocks that the copies are yet to read
        side.synchronize()
        with torch.cuda.stream(side):
            for t in [torch.empty_like(t) for t in want]:
                t.view(torch.uint8).fill_(0x44)
        torch.cuda.synchronize()
        for g, w in zip(kept, want):
            assert torch.equal(g, w)


# ---------------------------------------------------------------------------------------------
# gradients of rows that no choice names
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,rows,N", [(0, 2, 40, 64), (1, 1, 1, 8), (3, 2, 6, 136), (50, 3, 333, 1000),
                                        (33, 9, 500, 264), (700, 4, 2800, 128), (1000, 2, 9000, 40)])
@pytest.mark.parametrize("missing", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward_zeroes_rows_that_no_slot_names(T, k, rows, N, missing, weighted):
    """The gradient as the call allocates it: more rows than choices, choices of none, over memory that
    held NaN; the workspace is over memory that held choices' numbers."""
    rng = np.random.default_rng(T + N)
    slots = rng.permutation(rows)[:T * k].reshape(T, k).astype(np.int32)
    slots[rng.random((T, k)) < missing] = -1
    if T > 2 and missing < 1:
        slots[0, 0] = rows + 2  # outside: none
    y, dout = bf16_inputs(rng, rows, N, False), bf16_inputs(rng, T, N, False)
    w = torch.from_numpy(rng.standard_normal((T, k))).float().cuda()
    s = torch.from_numpy(slots).cuda()
    given = torch.zeros(rows, N, device="cuda", dtype=torch.bfloat16)
    want, want_w = mxq.mx_combine_backward(dout, y, s, w if weighted else None, dy=given)
    for stale in (float("nan"), 1.0):
        a = torch.full((rows, N), stale, device="cuda", dtype=torch.bfloat16)
        b = torch.arange(rows, device="cuda", dtype=torch.int32) % max(T * k, 1)
        del a, b  # the next tensors of their sizes lie where they lay
        dy, dw = mxq.mx_combine_backward(dout, y, s, w if weighted else None)
        assert torch.equal(dy, want) and torch.equal(dw, want_w)
    named = slots[(slots >= 0) & (slots < rows)]
    assert not want[np.setdiff1d(np.arange(rows), named)].any()


# ---------------------------------------------------------------------------------------------
# gradients of confident routers
# ---------------------------------------------------------------------------------------------
def test_route_backward_of_confident_sigmoids():
    """s (1 - s) where s is next to 1: the second factor is as small as the other expert's s. Each of
    s and 1 - s errs by an exponential (2 ulp: 4 units), a sum and a division (1 each), their product with
    the gradient and the scale by three roundings: 15 units, twice that allowed."""
    rng = np.random.default_rng(21)
    for k, E in ((1, 40), (8, 300)):
        l = rng.uniform(8, 60, (64, E)) * rng.choice([-1, 1], (64, E))
        l[:, :k] = np.abs(l[:, :k])
        logits = torch.from_numpy(l).float().cuda()
        experts, _ = mxq.mx_route(logits, k, mxq.SIGMOID, renormalize=False)
        g = rng.standard_normal((64, k)).astype(np.float32)
        got = cpu(mxq.mx_route_backward(torch.from_numpy(g).cuda(), logits, experts, mxq.SIGMOID,
                                        renormalize=False, scale=1.5)).astype(np.float64)
        l = cpu(logits).astype(np.float64)
        want = np.zeros_like(l)
        chosen = np.take_along_axis(l, cpu(experts).astype(np.int64), 1)
        np.put_along_axis(want, cpu(experts).astype(np.int64),
                          1.5 * g / (1 + np.exp(-chosen)) / (1 + np.exp(chosen)), 1)
        assert (np.abs(got - want) <= 30 * R.U * np.abs(want) + 1e-37).all()


def pairwise_gradient(l, experts, g, scale, score, renorm):
    """The gradient as sums of differences, in 64 bits, with the sums of their magnitudes: with p the
    scores and D the gradient of every score (scale g at the chosen ones, 0 elsewhere),
    softmax dl_i = p_i sum_j p_j (D_i - D_j); renormalised D_i = scale sum_j p_j (g_i - g_j) / P^2 first."""
    T, E = l.shape
    p = R.scores(l, score)
    at = experts.astype(np.int64)
    c = np.take_along_axis(p, at, 1)
    d, size = scale * g, scale * np.abs(g)
    if renorm:
        P = c.sum(1, keepdims=True)
        between = (g[:, :, None] - g[:, None, :]) * c[:, None, :]
        d = scale * between.sum(2) / P / P
        size = scale * np.abs(between).sum(2) / P / P
    D, S = np.zeros_like(l), np.zeros_like(l)
    np.put_along_axis(D, at, d, 1)
    np.put_along_axis(S, at, size, 1)
    if score == "sigmoid":
        q = 1 / (1 + np.exp(l))  # 1 - p
        return D * p * q, S * p * q
    if renorm:  # sum_j p_j D_j is 0
        return p * D, p * (S + (p * S).sum(1, keepdims=True))
    between = D[:, :, None] - D[:, None, :]
    return p * (p[:, None, :] * between).sum(2), p * (p[:, None, :] * np.abs(between)).sum(2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(3, 1), (40, 2), (64, 6), (257, 8), (1024, 32)])
@pytest.mark.parametrize("equal", [False, True])
def test_route_backward_of_confident_routers(E, k, score, renorm, equal):
    """Nearly all of the score at one expert (or at the chosen ones together): what is left of the
    gradient is far below the terms that it is usually written with, and as accurate as they are."""
    rng = np.random.default_rng(E + k)
    T = 48
    l = rng.standard_normal((T, E))
    l[np.arange(T), rng.integers(0, E, T)] += rng.uniform(0, 30, T)
    if k > 1:
        top = np.argsort(-l, 1)[:, :k]
        late = T // 2  # half of the tokens: all chosen experts far above the others
        np.put_along_axis(l[late:], top[late:], np.take_along_axis(l[late:], top[late:], 1) + 15, 1)
    l = l.astype(np.float32)
    logits = torch.from_numpy(l).cuda()
    experts, _ = mxq.mx_route(logits, k, mxq.SOFTMAX if score == "softmax" else mxq.SIGMOID)
    g = np.ones((T, k), np.float32) if equal else rng.standard_normal((T, k)).astype(np.float32)
    got = cpu(mxq.mx_route_backward(torch.from_numpy(g).cuda(), logits, experts,
                                    mxq.SOFTMAX if score == "softmax" else mxq.SIGMOID,
                                    renormalize=renorm, scale=2.5)).astype(np.float64)
    want, size = pairwise_gradient(l.astype(np.float64), cpu(experts), g.astype(np.float64), 2.5, score,
                                   renorm)
    # a score errs by under 128 units (exponential of a rounded argument up to 40, sum of E, division);
    # a term of the sums is a difference (1 unit) times one score, or two where renormalised, times p_i
    assert (np.abs(got - want) <= 512 * R.U * size + 1e-37).all(), (np.abs(got - want) / (size + 1e-37)).max()


# ---------------------------------------------------------------------------------------------
# scales at the ends of fp32
# ---------------------------------------------------------------------------------------------
def far_operand(rng, rows, K, form, exponent):
    """operand() with every third row (or 128-row block) of scale 1.25 * 2^exponent; -> also which rows."""
    (codes, scales), _ = operand(rng, rows, K, form)
    scales = cpu(scales)
    hot = (np.arange(rows) // (1 if form == "rows" else 128)) % 3 == 0
    if form == "rows":
        scales[:, hot] = 2.0 ** exponent * 1.25
    else:
        scales[::3] = 2.0 ** exponent * 1.25
    return (codes, torch.from_numpy(scales).cuda()), R.values(cpu(codes), scales, form), hot


def check_far_product(C, a, b, K, hot_a, hot_b, beyond, what=""):
    """Against the 64-bit product. Where the factor of two scales is beyond fp32 every block's sum times it
    is infinite, or NaN of a sum of nothing: those entries are not finite, and no others are touched."""
    C = C.double().cpu().numpy()
    want, S = R.product(a, b)
    bound = R.product_bound(want, S, K, True)
    far = hot_a[:, None] & hot_b[None, :] & beyond
    assert not np.isfinite(C[far]).any(), what
    assert (np.abs(C - want)[~far] <= bound[~far]).all(), what


FAR = [
    # exponents of the operands' scales; whether their product is beyond fp32
    (60, 40, False), (-40, 95, False), (100, -100, False),
    (-30, -64, False),            # results of 2^-80, their factors near the least normal number
    (100, 40, True), (40, 100, True),
]


@pytest.mark.parametrize("M,N,K", [(5, 392, 416), (100, 4096, 4096), (40, 1000, 2048), (2048, 2048, 640)])
@pytest.mark.parametrize("form", ["blocks", "rows"])
@pytest.mark.parametrize("ea,eb,beyond", FAR)
def test_gemm_scales_at_the_ends_of_fp32(M, N, K, form, ea, eb, beyond):
    rng = np.random.default_rng(M + N)
    (ac, asc), a, hot_a = far_operand(rng, M, K, "rows", ea)
    (bc, bsc), b, hot_b = far_operand(rng, N, K, form, eb)
    for dtype in (torch.bfloat16, torch.float32):
        C = mxq.mx_gemm_b128(ac, asc, bc, bsc, mxq.B128_ROWS if form == "rows" else mxq.B128_BLOCKS,
                             out_dtype=dtype)
        check_far_product(C, a, b, K, hot_a, hot_b, beyond)


@pytest.mark.parametrize("ea,eb,beyond", FAR)
def test_gemm_by_expert_scales_at_the_ends_of_fp32(ea, eb, beyond):
    rng = np.random.default_rng(7)
    counts, N, K = [5, 0, 300, 128, 17, 129], 520, 416
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    off = torch.from_numpy(offsets).cuda()
    (ac, asc), a, hot_a = far_operand(rng, sum(counts), K, "rows", ea)
    bs = [far_operand(rng, N, K, "blocks", eb) for _ in counts]
    C = mxq.mx_gemm_b128_grouped(ac, asc, torch.stack([b[0][0] for b in bs]),
                                 torch.stack([b[0][1] for b in bs]), off)
    P = mxq.mx_b128_padded_rows(sum(counts), len(counts))
    (uc, usc), u, hot_u = far_operand(rng, 288, P, "rows", ea)
    (vc, vsc), v, hot_v = far_operand(rng, 392, P, "rows", eb)
    W = mxq.mx_gemm_b128_grouped_wgrad(uc, usc, vc, vsc, off)
    at = 0
    for e, n in enumerate(counts):
        part = slice(offsets[e], offsets[e + 1])
        if n:
            check_far_product(C[part], a[part], bs[e][1], K, hot_a[part], bs[e][2], beyond, e)
            check_far_product(W[e], u[:, at:at + R.up(n)], v[:, at:at + R.up(n)], R.up(n), hot_u, hot_v,
                              beyond, e)
        at += R.up(n)


def test_gemm_of_quantised_huge_tiny_and_empty_rows():
    """What the quantisers make of blocks of zeros, of 2^-110 and of 2^100, multiplied with ordinary ones."""
    rng = np.random.default_rng(31)
    x, w = bf16_inputs(rng, 300, 512), bf16_inputs(rng, 264, 512, False)
    for rows in (x[:5].contiguous(), x):
        q = mxq.mx_quantize_b128_rows(rows)
        a = R.values(cpu(q[0]), cpu(q[1]), "rows")
        for (bc, bs), form, name in ((mxq.mx_quantize_b128_blocks(w), mxq.B128_BLOCKS, "blocks"),
                                     (mxq.mx_quantize_b128_rows(w), mxq.B128_ROWS, "rows")):
            check_product(mxq.mx_gemm_b128(*q, bc, bs, form), a, R.values(cpu(bc), cpu(bs), name), 512)


# ---------------------------------------------------------------------------------------------
# routing: bases, NaN in groups, close scores
# ---------------------------------------------------------------------------------------------
def off_base(t, by=1):
    """A copy of t whose first element lies `by` elements after an allocation's start."""
    buf = torch.empty(t.numel() + by, device="cuda", dtype=t.dtype)
    view = buf[by:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [mxq.SOFTMAX, mxq.SIGMOID])
@pytest.mark.parametrize("E,k,groups,top", [(128, 8, 1, 1), (256, 8, 8, 4), (512, 6, 1, 1), (1024, 8, 16, 3)])
@pytest.mark.parametrize("by", [1, 2, 3])
def test_route_of_bases_that_allow_no_wide_loads(dtype, score, E, k, groups, top, by):
    rng = np.random.default_rng(E + by)
    logits = torch.from_numpy(rng.standard_normal((37, E))).to(dtype).cuda()
    bias = torch.from_numpy(rng.standard_normal(E) * 0.1).float().cuda()
    at = dict(groups=groups, top_groups=top)
    want = mxq.mx_route(logits, k, score, bias, **at)
    grad = torch.from_numpy(rng.standard_normal((37, k))).float().cuda()
    want_d = mxq.mx_route_backward(grad, logits, want[0], score)
    l, b = off_base(logits, by), off_base(bias, by)
    assert l.data_ptr() % 16 and b.data_ptr() % 16
    for li, bi in ((l, bias), (logits, b), (l, b)):
        got = mxq.mx_route(li, k, score, bi, experts=off_base(want[0]), weights=off_base(want[1]), **at)
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    for li, out in ((l, torch.zeros_like(logits)), (logits, off_base(logits, by)), (l, off_base(logits, by))):
        got = mxq.mx_route_backward(off_base(grad), li, off_base(want[0]), score, grad_logits=out)
        assert torch.equal(got, want_d)


def order(c):
    """What a choice is ordered by: excluded ones last, NaN before them, then numbers."""
    return (0, 0.0) if c == -np.inf else (1, 0.0) if np.isnan(c) else (2, float(c))


def plain_route(c, k, groups, top):
    """One token's experts from its choices c, with NaN and -inf among them; and the least distance
    between two numbers that were compared and decided something."""
    size, near = len(c) // groups, np.inf
    allowed = range(len(c))
    if 1 < groups and top < groups:
        keys = []
        for g in range(groups):
            best = sorted((order(x) for x in c[g * size:(g + 1) * size]), reverse=True)[:2]
            if best[0][0] < 2 or len(best) == 1 or best[1][0] == 0:
                keys.append(best[0])
            else:
                keys.append(best[0] if best[1][0] == 0 else
                            (1, 0.0) if best[1][0] == 1 else (2, best[0][1] + best[1][1]))
        ranked = sorted(range(groups), key=lambda g: (keys[g], -g), reverse=True)
        if keys[ranked[top - 1]][0] == 2 and keys[ranked[top]][0] == 2:
            near = keys[ranked[top - 1]][1] - keys[ranked[top]][1]
        allowed = [e for g in sorted(ranked[:top]) for e in range(g * size, (g + 1) * size)]
    ranked = sorted(allowed, key=lambda e: (order(c[e]), -e), reverse=True)
    for a, b in zip(ranked[:k], ranked[1:k + 1]):
        if order(c[a])[0] == 2 and order(c[b])[0] == 2:
            near = min(near, c[a] - c[b])
    chosen = [e if order(c[e])[0] else -1 for e in ranked[:k]]
    return chosen + [-1] * (k - len(chosen)), near


@pytest.mark.parametrize("E,k,groups,top", [(32, 6, 8, 3), (60, 7, 5, 2), (64, 6, 16, 5), (256, 8, 8, 4),
                                            (32, 3, 32, 4), (24, 8, 1, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_of_nan_and_masked_choices_in_groups(E, k, groups, top, biased):
    rng = np.random.default_rng(E + k)
    T = 200
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[rng.random((T, E)) < 0.25] = np.nan
    l[rng.random((T, E)) < 0.25] = -np.inf
    size = E // groups
    for t in range(0, T, 4):  # groups of nothing but NaN, of nothing, of one number
        g = rng.integers(0, groups, 3)
        l[t, g[0] * size:(g[0] + 1) * size] = np.nan
        l[t, g[1] * size:(g[1] + 1) * size] = -np.inf
        l[t, g[2] * size:(g[2] + 1) * size] = -np.inf
        l[t, g[2] * size] = 2.0
    l[1], l[2] = np.nan, -np.inf
    bias = (rng.standard_normal(E) * 0.2).astype(np.float32) if biased else None
    experts, weights = mxq.mx_route(torch.from_numpy(l).cuda(), k, mxq.SIGMOID,
                                    torch.from_numpy(bias).cuda() if biased else None, groups=groups,
                                    top_groups=top, renormalize=False)
    experts, weights = cpu(experts), cpu(weights)
    sure = 0
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-l.astype(np.float64)))
    c = np.where(np.isneginf(l), -np.inf, s + (0 if bias is None else bias.astype(np.float64)))
    for t in range(T):
        want, near = plain_route(c[t], k, groups, top)
        if near < 1e-6:
            continue
        sure += 1
        assert experts[t].tolist() == want
        w = np.where(np.array(want) >= 0, s[t][np.maximum(want, 0)], 0.0)
        assert (np.abs(weights[t] - w) <= 8 * R.U * w)[~np.isnan(w)].all()
        assert (np.isnan(weights[t]) == np.isnan(w)).all()
    assert sure > 0.9 * T


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", [(64, 6, 1, 1), (256, 8, 8, 4), (777, 8, 1, 1), (1024, 32, 16, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_of_close_scores(score, E, k, groups, top, dtype):
    """Every token of scores as they come, near ties and (in bf16) exact ones among them: no expert left
    out is better than one chosen, nor a group, by more than the error of the scores."""
    rng = np.random.default_rng(E)
    T = 300
    logits = torch.from_numpy(rng.standard_normal((T, E))).to(dtype).cuda()
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    experts, weights = mxq.mx_route(logits, k, mxq.SOFTMAX if score == "softmax" else mxq.SIGMOID,
                                    torch.from_numpy(bias).cuda(), groups=groups, top_groups=top)
    e, w = cpu(experts).astype(np.int64), cpu(weights).astype(np.float64)
    s = R.scores(logits.cpu().double().numpy(), score)
    c = s + bias
    eps = 1e-6  # scores and sums below 2, each a few units of 2^-24 off
    assert (e >= 0).all() and all(len(set(row)) == k for row in e.tolist())
    if groups > 1:
        size = E // groups
        two = -np.sort(-c.reshape(T, groups, size), 2)[:, :, :2].sum(2)
        used = np.zeros((T, groups), bool)
        np.put_along_axis(used, e // size, True, 1)
        assert (used.sum(1) <= top).all()
        # any group used is within eps of the best `top`, any clearly among them is open to choice
        bar = -np.sort(-two, 1)[:, top - 1:top]
        assert (two[used] >= np.broadcast_to(bar, two.shape)[used] - eps).all()
        c = np.where(np.repeat(used | (two > bar + eps), size, 1), c, -10.0)
    got = np.take_along_axis(c, e, 1)
    assert (np.diff(got, axis=1) <= eps).all()
    rest = c.copy()
    np.put_along_axis(rest, e, -10.0, 1)
    assert (rest.max(1) <= got.min(1) + eps).all()
    p = np.take_along_axis(s, e, 1)
    p = p / p.sum(1, keepdims=True)
    assert (np.abs(w - p) <= 512 * R.U * p).all()


# ---------------------------------------------------------------------------------------------
# the example's autograd functions
# ---------------------------------------------------------------------------------------------
def example_layer():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer_edges", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("frozen", [("up",), ("up", "down", "shared"), ("router",)])
def test_example_computes_the_gradients_that_are_asked_for(monkeypatch, frozen):
    example = example_layer()
    torch.manual_seed(1)
    layer = example.ExpertLayer(256, 128, 8, 2).cuda()
    x = torch.randn(50, 256, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(50, 256, device="cuda").bfloat16()
    layer(x).backward(dy)
    want = {n: p.grad.clone() for n, p in layer.named_parameters()}
    layer.zero_grad()
    for name in frozen:
        getattr(layer, name).requires_grad_(False)
    calls = []
    real = mxq.mx_gemm_b128_grouped_wgrad
    monkeypatch.setattr(mxq, "mx_gemm_b128_grouped_wgrad", lambda *a, **k: calls.append(1) or real(*a, **k))
    layer(x).backward(dy)
    assert len(calls) == 2 - len({"up", "down"} & set(frozen))
    for name, p in layer.named_parameters():
        assert p.grad is None if name in frozen else torch.equal(p.grad, want[name])


def test_example_refuses_second_derivatives():
    example = example_layer()
    layer = example.ExpertLayer(128, 64, 4, 2).cuda()
    x = torch.randn(9, 128, device="cuda").bfloat16().requires_grad_()
    (dx,) = torch.autograd.grad(layer(x).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.float().square().sum().backward()


def test_example_keeps_no_tensor_outside_autograds_own_list():
    example = example_layer()
    torch.manual_seed(2)
    w = torch.randn(4, 64, 128, device="cuda", requires_grad=True)
    x = torch.randn(9, 128, device="cuda").bfloat16().requires_grad_()
    experts, _ = mxq.mx_route(torch.randn(9, 4, device="cuda"), 2)
    row_offsets, tokens, slots = mxq.mx_route_plan(experts, 4)
    y = example.ExpertLinear.apply(x, w, row_offsets, tokens, slots)
    tokens.add_(0)  # a change between forward and backward is noticed
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_an_empty_index_gathers_no_rows():
    x = torch.ones(40, 256, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, device="cuda", dtype=torch.int32)
    codes, scales = mxq.mx_quantize_b128_rows(x, none)
    assert codes.shape == (0, 256) and scales.shape == (2, 0)
    codes, scales = mxq.mx_quantize_b128_cols(x, none)
    assert codes.shape == (256, 0) and scales.shape == (0, 256)
    offsets = torch.zeros(4, device="cuda", dtype=torch.int64)
    u = mxq.mx_quantize_b128_cols(x, none, offsets)
    assert not mxq.mx_gemm_b128_grouped_wgrad(*u, *u, offsets).any()
    b = mxq.mx_quantize_b128_blocks(torch.ones(3, 64, 256, device="cuda", dtype=torch.bfloat16))
    assert mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(x, none), *b, offsets).shape == (0, 64)


# ---------------------------------------------------------------------------------------------
# stream order under programmatic dependent launch
# ---------------------------------------------------------------------------------------------
def test_dependent_expert_calls_keep_stream_order():
    """A chain in which every kernel of an expert layer reads what the launch before it has just written,
    index lists, slots, weights and workspaces among it, into buffers that the steps before read: back to
    back, and in a graph, the bytes are those of a synchronization after every call."""
    rng = np.random.default_rng(41)
    T, E, k, N, K = 3000, 24, 4, 512, 1024
    sources = [bf16_inputs(rng, T, K, False) for _ in range(3)]
    logit_sources = [torch.from_numpy(rng.standard_normal((T, E))).float().cuda() for _ in range(3)]
    w = mxq.mx_quantize_b128_blocks(torch.stack([bf16_inputs(rng, N, K, False) for _ in range(E)]))
    shared = mxq.mx_quantize_b128_blocks(bf16_inputs(rng, N, K, False))
    rows, P = T * k, mxq.mx_b128_padded_rows(T * k, E)
    new = lambda *s, dtype=torch.float32: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    b = dict(x=new(T, K, dtype=bf), logits=new(T, E), experts=new(T, k, dtype=i32), weights=new(T, k),
             offsets=new(E + 1, dtype=torch.int64), tokens=new(rows, dtype=i32), slots=new(T, k, dtype=i32),
             work=new(mxq.mx_route_plan_workspace(T, k, E), dtype=u8),
             rc=new(rows, K, dtype=u8), rs=new(K // 128, rows), y=new(rows, N, dtype=bf),
             out=new(T, N, dtype=bf), dy=new(rows, N, dtype=bf), dw=new(T, k), dl=new(T, E),
             uc=new(N, P, dtype=u8), us=new(P // 128, N), vc=new(K, P, dtype=u8), vs=new(P // 128, K),
             grad=new(E, N, K), dc=new(T, K, dtype=u8), ds=new(K // 128, T), one=new(T, N, dtype=bf),
             few=new(7, N, dtype=bf), fc=new(7, K, dtype=u8), fs=new(K // 128, 7), wc=new(N, N, dtype=u8),
             ws=new(N // 128, N // 128), wt=new(N, N, dtype=u8), wst=new(N // 128, N // 128))

    def chain(sync=False):
        seen = []
        for i in range(3):
            for step in (
                lambda: b["x"].copy_(sources[i]), lambda: b["logits"].copy_(logit_sources[i]),
                lambda: mxq.mx_route(b["logits"], k, experts=b["experts"], weights=b["weights"]),
                lambda: mxq.mx_route_plan(b["experts"], E, row_offsets=b["offsets"], tokens=b["tokens"],
                                          slots=b["slots"], workspace=b["work"]),
                lambda: mxq.mx_quantize_b128_rows(b["x"], b["tokens"], codes=b["rc"], scales=b["rs"]),
                lambda: mxq.mx_gemm_b128_grouped(b["rc"], b["rs"], *w, b["offsets"], c=b["y"]),
                lambda: mxq.mx_combine(b["y"], b["slots"], b["weights"], out=b["out"]),
                lambda: mxq.mx_combine_backward(b["out"], b["y"], b["slots"], b["weights"], dy=b["dy"],
                                                dweights=b["dw"]),
                lambda: mxq.mx_route_backward(b["dw"], b["logits"], b["experts"], grad_logits=b["dl"]),
                lambda: mxq.mx_quantize_b128_cols(b["dy"], None, b["offsets"], codes=b["uc"], scales=b["us"]),
                lambda: mxq.mx_quantize_b128_cols(b["x"], b["tokens"], b["offsets"], codes=b["vc"],
                                                  scales=b["vs"]),
                lambda: mxq.mx_gemm_b128_grouped_wgrad(b["uc"], b["us"], b["vc"], b["vs"], b["offsets"],
                                                       c=b["grad"]),
                lambda: mxq.mx_quantize_b128_rows(b["x"], codes=b["dc"], scales=b["ds"]),
                lambda: mxq.mx_gemm_b128(b["dc"], b["ds"], *shared, c=b["one"]),
                lambda: mxq.mx_quantize_b128_blocks(b["one"][:N], transpose=True, codes=b["wc"],
                                                    scales=b["ws"], codes_t=b["wt"], scales_t=b["wst"]),
                lambda: mxq.mx_quantize_b128_rows(b["x"][:7], codes=b["fc"], scales=b["fs"]),
                lambda: mxq.mx_gemm_b128(b["fc"], b["fs"], *shared, c=b["few"]),
            ):
                step()
                if sync:
                    torch.cuda.synchronize()
            seen.append({name: t.clone() for name, t in b.items() if name != "work"})
            if sync:
                torch.cuda.synchronize()
        return seen

    def same(got):
        torch.cuda.synchronize()
        for g, h in zip(got, want):
            for name in g:
                used = slice(None)
                if name in ("uc", "vc", "us", "vs"):  # past the last expert's blocks nothing is written
                    n = int(((h["offsets"].diff() + 127) // 128).sum())
                    used = (slice(None), slice(n * 128)) if name in ("uc", "vc") else slice(n)
                assert torch.equal(g[name][used], h[name][used]), name

    want = chain(sync=True)
    for _ in range(5):
        same(chain())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = chain()
    for _ in range(3):
        graph.replay()
        same(captured)


@pytest.mark.parametrize("handle", [0, 1, 2])  # the default stream by both its handles, the thread's own
def test_streams_by_their_special_handles(handle):
    rng = np.random.default_rng(5)
    x = bf16_inputs(rng, 640, 512, False)
    logits = torch.from_numpy(rng.standard_normal((640, 16))).float().cuda()

    def work(**at):
        experts, weights = mxq.mx_route(logits, 2, **at)
        offsets, tokens, slots = mxq.mx_route_plan(experts, 16, **at)
        return [experts, weights, offsets, tokens, slots, *mxq.mx_quantize_b128_rows(x, tokens, **at),
                *mxq.mx_quantize(x, mxq.E4M3, **at), mxq.mx_combine(x, slots, weights, **at)]

    want = work()
    torch.cuda.synchronize()
    for current in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(current):
            got = work(stream=handle)
            torch.cuda.synchronize()
            assert all(torch.equal(g, w) for g, w in zip(got, want))
            del got


def test_stream_argument_inside_a_capture():
    rng = np.random.default_rng(6)
    logits = torch.from_numpy(rng.standard_normal((700, 16))).float().cuda()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def work(**at):
        experts, weights = mxq.mx_route(logits, 2, **at)
        return [experts, weights, *mxq.mx_route_plan(experts, 16, **at)]

    want = work()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = work(stream=side.cuda_stream)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
