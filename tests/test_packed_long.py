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


# Sums of P V: the tensor core adds 16 products at a time by truncation, 5.25 * 2^-23 of the running sum at most, over no more
# than 2^18 keys. bf16: the weights' rounding (where they are not powers of two) and the output's, 2^-8 each.
SUMS = 2 ** 18 / 16 * 5.25 * 2.0 ** -23
SPAN = 2 ** 17 / 16 * 5.25 * 2.0 ** -23 + 2.0 ** -12  # in spans of 2^17 keys, added in fp32


def values(Hk, nk, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.empty((Hk, nk, d), dtype=torch.bfloat16, device="cuda")
    for h in range(Hk):
        for at in range(0, nk, 1 << 22):
            part = v[h, at:at + (1 << 22)]
            part.copy_(1.0 + torch.rand(part.shape, generator=g, device="cuda"))
    return v


def room(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


@pytest.mark.parametrize("d,nq", [(64, 16385), (128, 16500)])
@pytest.mark.parametrize("nk", [2 ** 22 + 5, 2 ** 18 + 1])
def test_mean_of_many_values(d, nq, nk):
    """Equal weights over more keys than one sum of the tensor core bears: prompts of more than 64 pairs of tiles, which are not cut. 2^22
    truncated additions left the mean 2.6 % too small."""
    room(16)
    q, k, v = torch.zeros((1, nq, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, nk, d), dtype=torch.bfloat16, device="cuda"), values(1, nk, d, 31)
    o, lse = call(q, k, v, [0, nq], [0, nk], False, nq)
    mcs.mcs_check_status()
    want = v[0].sum(0, dtype=torch.float64) / nk
    assert ((o[0].double() - want).abs() <= (2.0 ** -8 + SPAN) * want).all()
    assert ((lse.double() - torch.log(torch.tensor(float(nk), dtype=torch.float64))).abs() <= 2.0 ** -14).all()


@pytest.mark.parametrize("d,heads", [(64, (1, 1)), (128, (2, 1))])
@pytest.mark.parametrize("up", [True, False])
def test_scores_that_rise_or_fall_along_many_keys(d, heads, up):
    """The maximum moves between the spans of keys: two sequences, one of them short, causal; infinities that only the last rows see."""
    room(16)
    H, Hk = heads
    nq, nk = [16400, 300], [2 ** 20 - 77, 300]
    Tq, Tk, n = sum(nq), sum(nk), nk[0]
    q, k = torch.zeros((H, Tq, d), dtype=torch.bfloat16, device="cuda"), torch.zeros((Hk, Tk, d), dtype=torch.bfloat16, device="cuda")
    v = values(Hk, Tk, d, 32)
    q[:, :, 0] = 8.0
    ramp = torch.linspace(-60, 60, n, device="cuda") * (1.0 if up else -1.0)
    k[0, :n, 0] = ramp.bfloat16()
    v[0, n - 3, 5] = float("inf")
    o, lse = call(q, k, v, [0, nq[0], Tq], [0, n, Tk], True, nq[0], 0.125)
    mcs.mcs_check_status()
    score = k[0, :n, 0].double()
    last = n - nq[0] + 1  # keys that the first query sees; each further one sees one more
    w = torch.exp(score - score.max())
    vd = v[0, :n].double()
    vd[n - 3, 5] = 0.0
    sums = torch.cat([(w[:last] @ vd[:last])[None], w[last:, None] * vd[last:]]).cumsum(0)
    total = torch.cat([w[:last].sum()[None], w[last:]]).cumsum(0)
    want = sums / total[:, None]
    for h in range(H):
        got = o[h, :nq[0]].double()
        assert (got[-3:, 5] == float("inf")).all() and torch.isfinite(got[:-3]).all()
        got[-3:, 5] = want[-3:, 5]
        # scores up to 60: 4 or 8 sums of 16 products and the scale, twice (weights and their sum)
        ds = 60 * (d / 16 * 5.25 * 2.0 ** -23 + 2.0 ** -22)
        assert ((got - want).abs() <= (2.0 ** -7 + SPAN + 2 * ds) * want).all()
        assert ((lse[h, :nq[0]].double() - score.max() - torch.log(total)).abs() <= ds + 2.0 ** -12).all()
        short = v[0, n:, :].double().cumsum(0) / torch.arange(1, 301, device="cuda")[:, None]
        assert ((o[h, nq[0]:].double() - short).abs() <= (2.0 ** -7 + SUMS) * short).all()


@pytest.mark.parametrize("d,heads,S,nq,nk", [(64, (8, 8), 153, 1, 2 ** 22 + 9), (128, (32, 8), 153, 3, 2 ** 21 + 9), (64, (1, 1), 1, 16384, 2 ** 24)])
def test_pieces_of_many_keys(d, heads, S, nq, nk):
    """Single tokens and chunks of so many requests that they would not be cut for the SMs' sake, one of them over a long cache; and
    a chunk whose pieces would be too long if they only filled the SMs."""
    room(60)
    H, Hk = heads
    lk = [(17 * i) % 50 for i in range(S)]
    lk[S // 2] = nk
    ks = [0]
    for x in lk:
        ks.append(ks[-1] + x)
    q = torch.zeros((H, S * nq, d), dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros((Hk, ks[-1], d), dtype=torch.bfloat16, device="cuda"), values(Hk, ks[-1], d, 33)
    o, lse = call(q, k, v, [nq * i for i in range(S + 1)], ks, False, nq)
    mcs.mcs_check_status()
    for i in range(S):
        got, n = o[:, nq * i:nq * (i + 1)].double(), lk[i]
        if n == 0:
            assert (got == 0).all()
            continue
        want = (v[:, ks[i]:ks[i + 1]].sum(1, dtype=torch.float64) / n).repeat_interleave(H // Hk, 0)[:, None]
        assert ((got - want).abs() <= (2.0 ** -8 + SPAN) * want).all()
        assert ((lse[:, nq * i:nq * (i + 1)].double() - torch.log(torch.tensor(float(n), dtype=torch.float64))).abs() <= 2.0 ** -14).all()


def test_own_keys_need_no_cut():
    """Many short prompts over their own tokens, more than 2^18 in all: queries and keys have the same bounds, so nothing is long."""
    S, n, d = 9000, 30, 64
    g = torch.Generator(device="cuda").manual_seed(34)
    q, k, v = (torch.randn((2, S * n, d), generator=g, device="cuda").bfloat16() for _ in range(3))
    bounds = torch.arange(0, S * n + 1, n, dtype=torch.int32, device="cuda")
    desc = mcs.packed_desc(S, S * n, S * n, 2, 2, d, q.dtype, True, n)
    ws = mcs.packed_attn_workspace(desc)
    got = []
    for ks in (bounds, bounds.clone()):
        o, lse = torch.empty_like(q), torch.empty((2, S * n), device="cuda")
        mcs.mcs_packed_attn(desc, q, k, v, bounds, ks, o, lse, ws)
        got.append((o, lse))
    mcs.mcs_check_status()
    # cut or not: sums in another order
    assert torch.allclose(got[0][0].float(), got[1][0].float(), rtol=2.0 ** -7, atol=2.0 ** -10) and torch.allclose(got[0][1], got[1][1], atol=2.0 ** -16)
    i = 4321
    z = (q[1, i * n:i * n + n].double() @ k[1, i * n:i * n + n].double().T) / 8.0
    z.masked_fill_(torch.ones(n, n, device="cuda").triu(1).bool(), -torch.inf)
    want = torch.softmax(z, -1) @ v[1, i * n:i * n + n].double()
    size = torch.softmax(z, -1) @ v[1, i * n:i * n + n].double().abs()
    assert ((got[0][0][1, i * n:i * n + n].double() - want).abs() <= 2.0 ** -8 * (want.abs() + size) + 2.0 ** -14 * size).all()


def reference(q, k, v, qs, ks, causal):
    """float64 on the GPU, a head of a sequence at a time: o, lse, weight and spread as the oracle's."""
    H, Tq, d = q.shape
    g = H // k.shape[0]
    o, w = (torch.zeros((H, Tq, d), dtype=torch.float64, device="cuda") for _ in range(2))
    lse, spread = torch.full((H, Tq), -torch.inf, dtype=torch.float64, device="cuda"), torch.zeros((H, Tq), dtype=torch.float64, device="cuda")
    for a, b, ka, kb in zip(qs, qs[1:], ks, ks[1:]):
        nq, nk = b - a, kb - ka
        if nq == 0 or nk == 0:
            continue
        hide = torch.arange(nk, device="cuda")[None, :] > torch.arange(nq, device="cuda")[:, None] + nk - nq
        for h in range(H):
            qh, kh, vh = q[h, a:b].double(), k[h // g, ka:kb].double(), v[h // g, ka:kb].double()
            z = qh @ kh.T / d ** 0.5
            if causal:
                z.masked_fill_(hide, -torch.inf)
            lse[h, a:b] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            seen = torch.isfinite(lse[h, a:b])[:, None]
            o[h, a:b], w[h, a:b] = torch.where(seen, p @ vh, 0.0), torch.where(seen, p @ vh.abs(), 0.0)
            spread[h, a:b] = (qh.abs() @ kh.abs().T).amax(-1) / d ** 0.5
    return o, lse, w, spread


@pytest.mark.parametrize("d,H,Hk", [(64, 8, 8), (128, 12, 6)])
@pytest.mark.parametrize("S,at", [(40, 7), (9, 8)])
def test_chunks_of_many_requests(d, H, Hk, S, at):
    """Prompts that go on over 2^18 and more kept keys in all, one of them over more than one span; on both sides of 32 sequences,
    back to back over one workspace whatever it holds, and captured with lengths that change."""
    g = torch.Generator(device="cuda").manual_seed(35)

    def lengths(long):
        nq = [(137 * i) % 600 if i % 5 else 0 for i in range(S)]
        nk = [(5501 * i) % 9000 if i % 7 else 0 for i in range(S)]
        nq[at], nk[at] = 650, long
        return nq, nk

    def bounds(n):
        out = [0]
        for x in n:
            out.append(out[-1] + x)
        return out

    kinds = [tuple(map(bounds, lengths(n))) for n in (280_000, 131_073, 600)]
    Tq, Tk = kinds[0][0][-1], kinds[0][1][-1]
    q = (1.5 * torch.randn((H, Tq, d), generator=g, device="cuda")).bfloat16()
    k, v = (torch.randn((Hk, Tk, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    desc = mcs.packed_desc(S, Tq, Tk, H, Hk, d, q.dtype, True, 650)
    ws = mcs.packed_attn_workspace(desc)
    assert ws.numel() >= 100 * 256 * d * 4  # a bank for each of many blocks
    at_ = lambda s: torch.tensor(s, dtype=torch.int32, device="cuda")
    qd, kd = at_(kinds[0][0]), at_(kinds[0][1])
    new = lambda: (torch.full_like(q, 7.0), torch.full((H, Tq), 7.0, device="cuda"))
    run = lambda o, lse: mcs.mcs_packed_attn(desc, q, k, v, qd, kd, o, lse, ws)
    got = []
    for _ in range(3):
        ws.fill_(255)
        got.append(new())
        run(*got[-1])
        got.append(new())
        run(*got[-1])
    mcs.mcs_check_status()
    for o, lse in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1])
    go = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*go)
    for qs, ks in kinds:
        qd.copy_(at_(qs)), kd.copy_(at_(ks))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        ro, rl, w, spread = reference(q, k, v, qs, ks, True)
        seen = torch.isfinite(rl)
        ds = spread * (d / 16 * 5.25 * 2.0 ** -23 + 2.0 ** -22)
        sums = SPAN + 2.0 ** -14
        bo = 2.0 ** -8 * (w + ro.abs()) + w * (2 * ds[..., None] + 2 * sums) + 1e-30
        assert ((go[0].double() - ro).abs() <= bo)[seen].all()
        assert ((go[1].double() - rl).abs() <= ds + 2.0 ** -13 + rl.abs() * 2.0 ** -22)[seen].all()
        assert (go[0][~seen] == 0).all() and torch.isneginf(go[1][~seen]).all()
    mcs.mcs_check_status()
