"""The fp32 matrix product at the edges of its number parts and of fp32's range, by both of its
paths (up to eight rows, and more).

Single products (one column of x and w is not zero), from the arithmetic: parts rounded to
nearest leave |m| <= 2^-8 |x| (1 + 2^-8), |l| <= 2^-17 |x|, so the products left out are below
1.01 * 2^-24 |x w|; the leading product's step cuts its two terms two bits below the last one
(2 * 2^-25) and the result once (2^-23), the steps before it add 2^-6 of five such errors:
1.62 * 2^-23. Together below 2.25 * 2^-23 |x w|. Sums keep the bound of the accumulators (11 *
2^-23), and that of the products left out goes from 2^-20 to 2^-23: 12 * 2^-23.
"""
import numpy as np
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import f64, gen

pytestmark = pytest.mark.gpu


def product(x, w):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    B, M, K = x.shape
    y = torch.empty(B, M, w.shape[0], device="cuda")
    mcs.mcs_linear(mcs.linear_desc(B, M, K, w.shape[0], torch.float32), x, w, None, None, None, y)
    mcs.mcs_check_status()
    return y


# significands whose bits below the eighth and the sixteenth are all ones, all zeros, halves, or mixed
SIGNIFICANDS = [1 + 2.0 ** -7 - 2.0 ** -23, 2 - 2.0 ** -23, 1 + 2.0 ** -23, 1.5 + 2.0 ** -8 + 2.0 ** -16, 1 / 3 * 4,
                1 + 2.0 ** -8 - 2.0 ** -23, 1 + 2.0 ** -8 + 2.0 ** -17 - 2.0 ** -23, 1.0, 1 + 2.0 ** -15 - 2.0 ** -23,
                1.2345678]


@pytest.mark.parametrize("K,column", [(4, 0), (8, 3), (64, 37)])
@pytest.mark.parametrize("M", [6, 40])
def test_single_products(M, K, column):
    s = torch.tensor(SIGNIFICANDS, dtype=torch.float64)
    e = torch.randint(-30, 30, (M,), generator=gen(90)).double()
    x, w = torch.zeros(1, M, K), torch.zeros(130, K)
    x[0, :, column] = (s.repeat(-(-M // len(s)))[:M] * 2 ** e).float()
    w[:, column] = (s.repeat(13) * torch.where(torch.arange(130) % 2 == 0, 1.0, -0.25)).float()
    y = f64(product(x.cuda(), w.cuda()))
    want = f64(x) @ f64(w).T
    off = np.abs(y - want) / np.abs(want)
    assert off.max() <= 2.25 * 2.0 ** -23, float(off.max() * 2 ** 23)


@pytest.mark.parametrize("M", [7, 200])
def test_small_numbers_times_large_ones(M):
    """A number is held to 2^-133, bf16's last bit, whatever its size."""
    g = gen(91)
    K = 96
    x = torch.exp2(-119 + 16 * torch.rand(1, M, K, generator=g)) * torch.where(torch.rand(1, M, K, generator=g) < 0.5, 1, -1)
    w = torch.exp2(92 + 16 * torch.rand(70, K, generator=g))
    y, z = product(x.cuda(), w.cuda()), product(w[None].repeat(1, 3, 1).cuda(), x[0].contiguous().cuda())
    want = f64(x) @ f64(w).T
    size = np.abs(f64(x)) @ np.abs(f64(w)).T
    bound = (12 * 2.0 ** -23 + (K / 32 + 9) * 2.0 ** -24) * size + 2.0 ** -134 * np.abs(f64(w)).sum(1)
    assert np.all(np.abs(f64(y) - want) <= bound), float((np.abs(f64(y) - want) / bound).max())
    assert np.all(np.abs(f64(z)[0, :70].T - want[0]) <= bound[0])


@pytest.mark.parametrize("M", [5, 33])
def test_numbers_up_to_the_largest(M):
    """Finite numbers above bf16's largest are numbers, not infinities."""
    top = torch.finfo(torch.float32).max
    x, w = torch.zeros(1, M, 8), torch.zeros(3, 8)
    x[0, :, 0], x[0, :, 1] = top, -top / 2
    w[:, 0] = torch.tensor([1.0, -0.5, 2.0 ** -20])
    w[:, 1] = torch.tensor([1.0, 0.0, 2.0 ** -20])
    y = f64(product(x.cuda(), w.cuda()))
    want = f64(x) @ f64(w).T
    size = np.abs(f64(x)) @ np.abs(f64(w)).T
    assert np.all(np.abs(y - want) <= 2.25 * 2.0 ** -23 * size), y / want


@pytest.mark.parametrize("M,K,O", [(9, 8, 40), (40, 64, 130), (200, 1536, 260), (33, 5120, 100)])
def test_sums_within_the_documented_bound(M, K, O):
    """Numbers of one sign whose parts are all cut the same way, and numbers of all sizes."""
    g = gen(94)
    for kind in range(3):
        x, w = torch.rand(1, M, K, generator=g) + 0.5, torch.rand(O, K, generator=g) + 0.5
        if kind == 1:
            x, w = torch.full((1, M, K), SIGNIFICANDS[0]), torch.full((O, K), SIGNIFICANDS[0])
        if kind == 2:
            x, w = x * torch.exp(6 * torch.randn(1, M, K, generator=g)), w * torch.exp(6 * torch.randn(O, K, generator=g))
        y = f64(product(x.cuda(), w.cuda()))
        want = f64(x) @ f64(w).T
        assert np.all(np.abs(y - want) <= (12 * 2.0 ** -23 + (K / 32 + 9) * 2.0 ** -24) * want), kind
