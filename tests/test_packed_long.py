"""A prompt over so many keys that one pair of query tiles works on them for longer than the second that most waits of the
kernels may take."""

import pytest
import torch

from tests.test_packed_attn_gpu import call
from sparse_attention_diffusion_gb300 import mcs

pytestmark = pytest.mark.gpu


def test_items_of_more_than_a_second():
    """16,385 tokens over 2^27 kept keys of one head, d = 64: 65 pairs of tiles, which are not cut, of 1,048,577 tiles of keys
    each, 1.6 us a tile; the last pair has one row only, whose second tile waits all the while. All keys are zero but
    four, whose scores are 40: the others have e^-40 of their weight, 6e-10 in all, and values of zero."""
    nq, nk, d = 16385, 2 ** 27 + 77, 64
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    q = torch.zeros((1, nq, d), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((1, nk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[:, :, 0] = 8.0
    at = [5, 2 ** 26 + 3, nk - nq, nk - 100]
    g = torch.Generator(device="cuda").manual_seed(30)
    k[0, at, 0] = 40.0
    v[0, at] = (1.0 + torch.rand((4, d), generator=g, device="cuda")).bfloat16()
    o, lse = call(q, k, v, [0, nq], [0, nk], True, nq)
    mcs.mcs_check_status()
    rows = torch.arange(nq, device="cuda")
    sees = torch.tensor(at, device="cuda")[None, :] <= rows[:, None] + (nk - nq)
    n = sees.sum(1, keepdim=True).double()
    want = (sees.double() @ v[0, at].double()) / n
    # equal scores have equal weights: rounded to bf16 against a sum that is not (2^-8), and the output's rounding
    assert ((o[0].double() - want).abs() <= 2.0 ** -7 * want).all()
    # scores of 40: four sums of 16 products, each off by 5.25 * 2^-23 of them at most, and the scale
    assert ((lse[0].double() - 40.0 - torch.log(n[:, 0])).abs() <= 40 * (4 * 5.25 * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -16).all()
