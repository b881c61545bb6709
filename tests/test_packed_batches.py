"""Batches of unlike sequences in one call: prompts beside single tokens over kept keys, more sequences than a warp has lanes
with cut sequences of several tiles, one long cache among many short ones."""
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_packed_attn_gpu import DT, call, check, starts, view

pytestmark = pytest.mark.gpu


def tensors(seed, dtype, H, Hk, d, Tq, Tk, layout="tokens"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return view(g, H, Tq, d, DT[dtype], layout, 2.0), view(g, Hk, Tk, d, DT[dtype], "tokens"), view(g, Hk, Tk, d, DT[dtype], layout)


def chunks(S, at, nq, nk):
    """S sequences, of which number `at` has several tiles and the others a few tokens, no tokens or no keys."""
    q = [(3 * i) % 4 if i % 6 else 0 for i in range(S)]
    k = [(97 * i * i) % 1500 if i % 9 else 0 for i in range(S)]
    q[at], k[at] = nq, nk
    return q, k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,at,nq,nk,heads", [(40, 17, 300, 2500, (4, 1)), (40, 17, 220, 2500, (4, 1)), (33, 0, 200, 200, (3, 1)), (40, 39, 150, 3000, (4, 2)), (71, 33, 90, 1700, (5, 1))])
def test_cut_sequences_of_several_tiles_among_many(dtype, causal, d, S, at, nq, nk, heads):
    """More than 32 sequences, whose pieces and tiles are found by a search over the offsets."""
    H, Hk = heads
    lq, lk = chunks(S, at, nq, nk)
    qs, ks = starts(lq, 2), starts(lk, 1)
    q, k, v = tensors(S, dtype, H, Hk, d, qs[-1] + 1, ks[-1] + 2)
    desc = mcs.packed_desc(S, qs[-1] + 1, ks[-1] + 2, H, Hk, d, DT[dtype], causal, max(lq))
    if dtype == "bf16" or nq * H // Hk <= 64 * 16:  # fp32 takes 16 rows a tile here, and does not cut more than 64 tiles
        assert mcs.packed_attn_workspace(desc).numel() > 16  # the plan cuts
    check(q, k, v, qs, ks, causal, max_q=max(lq))
    check(q, k, v, qs, ks, causal, max_q=qs[-1])  # a bound that nobody reaches: more tiles are numbered than there are


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [7, 38])
@pytest.mark.parametrize("longest", [900, 3000])
def test_prompts_beside_single_tokens(dtype, d, tokens, longest):
    """Two prompts and a chunk of one among single tokens over kept keys, cut or not, on both sides of 32 sequences; with the
    bound on the queries and without."""
    lq, lk = [1] * tokens, [1 + (i * 379) % longest for i in range(tokens)]
    lq[2:2], lk[2:2] = [300, 0], [300, 0]
    lq += [129, 40]
    lk += [129, longest]
    qs, ks = starts(lq), starts(lk)
    q, k, v = tensors(tokens, dtype, 8, 2, d, qs[-1], ks[-1])
    check(q, k, v, qs, ks, True, max_q=300)
    a, b = call(q, k, v, qs, ks, True, 0), call(q, k, v, qs, ks, True, 0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 31, 63])
def test_one_long_cache_among_short_ones(dtype, d, at):
    """64 single tokens, 63 of them over 64 keys and less: the sequences are not cut."""
    lk = [(13 * i) % 65 for i in range(64)]
    lk[at] = 9000
    qs, ks = starts([1] * 64), starts(lk)
    q, k, v = tensors(at, dtype, 8, 4, d, 64, ks[-1], "heads")
    check(q, k, v, qs, ks, True, max_q=1)
