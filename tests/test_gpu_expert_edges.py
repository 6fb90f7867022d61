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
