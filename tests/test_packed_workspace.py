"""The workspace of mcs_packed_attn has room for the rows that can be there (CPU only)."""
import ctypes

import pytest

from sparse_attention_diffusion_gb300 import mcs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_q", [1, 3])
@pytest.mark.parametrize("S,Tk", [(64, 438_000), (1, 4000), (8, 240_000)])
def test_partial_sums_of_few_tokens(dtype, max_q, S, Tk):
    """Pieces of at least two tiles of 64 keys (one more a sequence), each with the sums, maximum and sum of weights of max_q tokens of
    a group for every key head, not of whole tiles of rows."""
    H, Hk, d = 32, 8, 128
    desc = mcs.packed_desc(S, S * max_q, Tk, H, Hk, d, dtype, True, max_q)
    n = mcs.load(build_if_missing=True).mcs_packed_attn_workspace_size(ctypes.byref(desc))
    assert 16 < n <= (Tk // 128 + S) * H * max_q * (d * 4 + 8)
