"""Attention over packed sequences where weights underflow: the parts of a sequence that are joined (pieces of its keys,
quarters of a tile) may lie so far apart that one part's weight is 0 in fp32."""
import math

import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_packed_attn_gpu import DT, call

pytestmark = pytest.mark.gpu


def far_apart(dtype, d, heads, nq, far, value):
    """Keys of two kinds: scores of 256 and values of 2^-20, and, where `far`, scores of -256 and values of `value`."""
    H, Hk = heads
    nk = far.numel()
    q, k = (torch.zeros((h, n, d), dtype=DT[dtype], device="cuda") for h, n in ((H, nq), (Hk, nk)))
    v = torch.full((Hk, nk, d), 2.0 ** -20, dtype=DT[dtype], device="cuda")
    q[:, :, 0] = 16.0
    k[:, :, 0] = torch.where(far, -16.0, 16.0).to(k.dtype)
    v[:, far] = value
    return q, k, v


# the keys far below: the last quarter of every 128, the first or the second half of all
KINDS = {"quarter": lambda j, n: j % 128 >= 96, "first": lambda j, n: j < n // 2, "second": lambda j, n: j >= n // 2}


@pytest.mark.parametrize("dtype,d,nq", [("bf16", 64, 1), ("bf16", 64, 40), ("bf16", 128, 1), ("bf16", 128, 100), ("f32", 64, 1), ("f32", 128, 40)])
@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("nk", [256, 2048])
def test_finite_values_of_no_weight_add_nothing(dtype, d, nq, kind, nk):
    """Weights of e^-512 = 2^-739 beside 1: values of 2^110, of which 2,048 are still far from fp32's largest number, are
    below 2^-600 in the result. What is left is the mean of equal powers of two. fp32: weights of 1, exact sums, a reciprocal and
    a product. bf16: the maximum is rounded to 2^-16 of log2 units, so weights are off by 2^-16, far inside bf16's half step."""
    j = torch.arange(nk, device="cuda")
    far = KINDS[kind](j, nk)
    q, k, v = far_apart(dtype, d, (2, 1), nq, far, 2.0 ** 110)
    o, lse = call(q, k, v, [0, nq], [0, nk], False, nq, 1.0)
    mcs.mcs_check_status()
    assert (o.float() * 2.0 ** 20 - 1.0).abs().max() <= 2.0 ** -22
    assert (lse - (256.0 + math.log(int((~far).sum())))).abs().max() <= 256 * 2.0 ** -21


@pytest.mark.parametrize("dtype,d,nq", [("bf16", 64, 1), ("bf16", 128, 1), ("bf16", 128, 100), ("f32", 128, 1)])
@pytest.mark.parametrize("nk", [2048, 20480])
@pytest.mark.parametrize("kind", ["first", "second"])
def test_infinities_of_no_weight_stay(dtype, d, nq, nk, kind):
    """Pieces whose weight beside the others is 0 in fp32, though not in the formula, keep their infinities and NaN. (Within a
    piece such weights are 0, and 0 times an infinity is NaN: here a piece's keys are alike.)"""
    far = KINDS[kind](torch.arange(nk, device="cuda"), nk)
    at = int(far.nonzero()[-3])
    q, k, v = far_apart(dtype, d, (2, 1), nq, far, 1.0)
    v[0, at, 5], v[0, at + 1, 7], v[0, at + 1, 9] = float("inf"), float("-inf"), float("nan")
    desc = mcs.packed_desc(1, nq, nk, 2, 1, d, q.dtype, False, nq, 1.0)
    assert mcs.packed_attn_workspace(desc).numel() > 16  # the plan cuts
    o, _ = call(q, k, v, [0, nq], [0, nk], False, nq, 1.0)
    mcs.mcs_check_status()
    o = o.float()
    assert (o[:, :, 5] == float("inf")).all() and (o[:, :, 7] == float("-inf")).all() and torch.isnan(o[:, :, 9]).all()
    rest = [c for c in range(d) if c not in (5, 7, 9)]
    assert (o[:, :, rest] * 2.0 ** 20 - 1.0).abs().max() <= 2.0 ** -22
