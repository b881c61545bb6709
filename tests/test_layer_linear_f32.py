"""The fp32 matrix product in bf16 parts against float64, at fp32's accuracy.

Bound of a sum, from the arithmetic (products of parts are exact in fp32):
  * parts cut off after 8, 16 and 24 bits: |m| < 2^-7 |x|, |l| < 2^-14 |x|, so the products
    left out, m l, l m and l l, are below 2 * 2^-21 + 2^-28 < 2^-20 of |x w|;
  * one accumulator takes 32 columns in two steps of the leading products: a step aligns 16
    products and the sum to the largest and cuts two bits below its last one (17 * 2^-25),
    and the result once more (2^-23): 2 * 5.25 * 2^-23, and the ten steps of the smaller
    products add 2^-7 of that each, together 11 * 2^-23 of the accumulator's sum |x w|;
  * K / 32 additions to nearest, and those of the K slices: (K / 32 + 8) * 2^-24.
"""
import numpy as np
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import f64, gen

pytestmark = pytest.mark.gpu


def product(x, w):
    B, M, K = x.shape
    y = torch.empty(B, M, w.shape[0], device="cuda")
    mcs.mcs_linear(mcs.linear_desc(B, M, K, w.shape[0], torch.float32), x, w, None, None, None, y)
    mcs.mcs_check_status()
    return y


@pytest.mark.parametrize("kind", ["normal", "positive", "wide", "cancelling"])
@pytest.mark.parametrize("M,K,O", [(9, 32, 5), (40, 36, 130), (129, 520, 128), (300, 1536, 260), (33, 5120, 100)])
def test_accuracy(M, K, O, kind):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    g = gen(40)
    x, w = torch.randn(1, M, K, generator=g), torch.randn(O, K, generator=g)
    if kind == "positive":
        x, w = x.abs(), w.abs()
    elif kind == "wide":
        x, w = x * torch.exp(4 * torch.randn(1, M, K, generator=g)), w * torch.exp(4 * torch.randn(O, K, generator=g))
    elif kind == "cancelling":                       # pairs of columns that cancel to the last bits
        x[..., 1::2] = x[..., ::2]
        w[:, 1::2] = -w[:, ::2] * (1 + 2.0 ** -20 * torch.randn(O, K // 2, generator=g))
    x, w = x.cuda(), w.cuda()
    y = f64(product(x, w))
    want = f64(x) @ f64(w).T
    size = np.abs(f64(x)) @ np.abs(f64(w)).T
    bound = (2.0 ** -20 + 11 * 2.0 ** -23 + (K / 32 + 8) * 2.0 ** -24) * size + 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(y - want) <= bound), float((np.abs(y - want) / bound).max())


def test_rows_agree_with_the_few_rows_kernel():
    """The same rows through both paths (eight rows and more) agree within the sums' bounds."""
    g = gen(41)
    x, w = torch.randn(1, 40, 1024, generator=g).cuda(), torch.randn(200, 1024, generator=g).cuda()
    a, b = product(x, w), product(x[:, :8].contiguous(), w)
    size = np.abs(f64(x[:, :8])) @ np.abs(f64(w)).T
    assert np.all(np.abs(f64(a)[:, :8] - f64(b)) <= (19 * 2.0 ** -23 + 40 * 2.0 ** -24 + 64 * 2.0 ** -24) * size)


def test_infinities_and_nan_stay_in_their_rows():
    g = gen(42)
    x, w = torch.randn(1, 200, 96, generator=g).cuda(), torch.randn(72, 96, generator=g).cuda()
    clean = product(x, w)
    x[0, 3, 5], x[0, 130, 95] = float("nan"), float("inf")
    y = product(x, w)
    keep = [m for m in range(200) if m not in (3, 130)]
    assert torch.equal(y[0, keep], clean[0, keep])
    assert bool(y[0, 3].isnan().all()) and not bool(y[0, 130].isfinite().any())


def test_large_and_small_magnitudes():
    """Numbers up to fp32's largest and down to its normal range."""
    x = torch.zeros(1, 12, 32)
    x[0, :, 0] = torch.tensor([3.4e38, -3.4e38, 1e38, 1e-38, -1.2e-38, 1.0, 1 + 2.0 ** -23, -(2 - 2.0 ** -23), 0.0, 2e-30,
                               65504.0, 1 / 3])
    w = torch.zeros(3, 32)
    w[:, 0] = torch.tensor([1.0, -0.5, 2.0 ** -20])
    y = f64(product(x.cuda(), w.cuda()))
    want = f64(x) @ f64(w).T
    # powers of two: every part's product is exact, what leaves the normal range may be lost
    assert np.all(np.abs(y - want) <= 2.0 ** -126 * 2)
