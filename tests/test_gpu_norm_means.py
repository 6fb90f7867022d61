"""Layer norm of rows of equal values, whose mean takes all of their digits."""

import numpy as np
import pytest
import torch

import __graft_entry__
import mx_microscaling_quantize_gb300 as mxq
import train_ref as T
from test_gpu_train import BF16, FP32, params
from test_gpu_train_edges import off_base, same

pytestmark = pytest.mark.gpu
VALUES = [100.0, -1000.0, 1016.0, 16256.0, 65280.0, 1000.1, -3.0e-3, 1 / 3, 2.0 ** 60 * 1.2345, -1e30]


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    yield
    assert mxq.mx_device_errors() == 0


LENGTHS = [8, 24, 104, 448, 776, 832, 896, 1000, 1032, 1792, 2056, 3584, 7168, 14336, 16376, 1, 7, 333, 1001, 5555,
           8193, 16383]


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("M", [11, 1331])  # a CTA each, and groups that walk pairs of rows
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_of_equal_values_are_the_bias(K, M, dtype):
    """The sums of at most 2^14 values c of bf16's 8 digits are exact in fp32's 24, at any length, base and kernel, so
    the mean is c, x - mean 0 and y the bias."""
    x = torch.tensor(VALUES, device="cuda").bfloat16().to(dtype).repeat(-(-M // len(VALUES)))[:M, None].repeat(1, K)
    w, b = params(K, K, FP32)
    kw = dict(stats=True)
    for src in (x, off_base(x)):
        y, mean, rstd = mxq.mx_layer_norm(src, w, b, out_dtype=FP32, **kw)
        assert torch.equal(mean, x[:, 0].float())
        assert torch.equal(y, b.expand(M, K))
        # the deviation is 0, so rstd = 1 / sqrt(eps): a rounding of eps and at most two of rstd's own
        want = 1 / np.sqrt(np.float64(np.float32(1e-5)))
        assert np.abs(T.f64(rstd) / want - 1).max() <= 4 * T.U
    if K % 32 == 0:
        codes, scales = mxq.mx_layer_norm_b128(x, w, b)
        want = mxq.mx_layer_norm_b128(torch.zeros_like(x), w, b)
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


def test_few_rows_and_many_have_the_same_bits():
    for K in (776, 1000, 7168, 14336):
        x = (1000 + torch.randn(1400, K, device="cuda")).contiguous()
        for center in (True, False):
            many = mxq.mx_layer_norm(x, center=center, stats=True)
            few = mxq.mx_layer_norm(x[7:18].contiguous(), center=center, stats=True)
            assert all(same(m[7:18] if m is not None else None, f) for m, f in zip(many, few))
