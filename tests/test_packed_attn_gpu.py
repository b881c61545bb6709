"""Attention over packed sequences against the float64 oracle: lengths from nothing to several tiles, masks that leave
rows empty, grouped heads, views, sequences cut along their keys, what lies behind them."""
import numpy as np
import pytest
import torch

from oracle import packed_oracle as orc
from sparse_attention_diffusion_gb300 import mcs

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def starts(lengths, first=0):
    return np.concatenate([[first], first + np.cumsum(lengths)]).astype(int).tolist()


def view(g, heads, tokens, d, dt, layout, gain=1.0):
    """A [heads, tokens, d] view: head by head in memory, or token by token in rows with a gap."""
    if layout == "heads":
        return (gain * torch.randn((heads, tokens, d), generator=g, device="cuda")).to(dt)
    x = (gain * torch.randn((tokens, heads + 3, d), generator=g, device="cuda")).to(dt)
    return x.transpose(0, 1)[1:heads + 1]


def bound(dtype, d, nk, o, lse, w, spread):
    """Largest errors of o and lse. bf16: the tensor core adds by truncation, up to 5.25 * 2^-23 of the running sum for
    16 products; weights are rounded to bf16 (2^-8), and so is the output. Scores are off by ds, which moves each weight
    by a factor 1 +- 2 ds at most after the division by the sum. fp32: every addition and product is off by 2^-24."""
    if dtype == "bf16":
        ds = spread * (d / 16 * 5.25 * 2.0 ** -23 + 2.0 ** -22)
        sums = nk / 16 * 5.25 * 2.0 ** -23 + nk * 2.0 ** -24 + 2.0 ** -20  # P V, the sum of weights, exponentials
        return 2.0 ** -8 * (w + np.abs(o)) + w * (2 * ds[..., None] + 2 * sums) + 1e-30, ds + sums + 2.0 ** -20 + np.abs(lse) * 2.0 ** -22
    ds = spread * (d + 4) * 2.0 ** -24 + spread * 2.0 ** -22
    sums = (2 * nk + 16) * 2.0 ** -24
    return w * (2 * ds[..., None] + 2 * sums) + np.abs(o) * 2.0 ** -23 + 1e-30, ds + sums + 2.0 ** -22 + np.abs(lse) * 2.0 ** -22


def call(q, k, v, qs, ks, causal, max_q=0, scale=0.0, out="heads", stream=None):
    H, Tq, d = q.shape
    desc = mcs.packed_desc(len(qs) - 1, Tq, k.shape[1], H, k.shape[0], d, q.dtype, causal, max_q, scale)
    o = torch.full((H, Tq, d), 7.0, dtype=q.dtype, device="cuda")
    if out != "heads":
        o = torch.full((Tq, H, d), 7.0, dtype=q.dtype, device="cuda").transpose(0, 1)
    lse = torch.full((H, Tq), 7.0, dtype=torch.float32, device="cuda")
    at = lambda s: torch.tensor(s, dtype=torch.int32, device="cuda")
    mcs.mcs_packed_attn(desc, q, k, v, at(qs), at(ks), o, lse, mcs.packed_attn_workspace(desc), stream)
    return o, lse


def check(q, k, v, qs, ks, causal, max_q=0, scale=None, out="heads"):
    o, lse = call(q, k, v, qs, ks, causal, max_q, scale or 0.0, out)
    mcs.mcs_check_status()
    f = lambda t: t.float().cpu().numpy().astype(np.float64)
    ro, rl, w, spread = orc.packed_attention(f(q), f(k), f(v), qs, ks, causal, scale)
    o, lse = f(o), f(lse)
    outside = np.isnan(rl)
    assert (o[outside] == 7.0).all() and (lse[outside] == 7.0).all()
    empty = np.isneginf(rl)
    assert (o[empty] == 0).all() and np.isneginf(lse[empty]).all()
    rows = ~outside & ~empty
    bo, bl = bound("bf16" if q.dtype == torch.bfloat16 else "f32", q.shape[2], max(1, k.shape[1]), ro[rows], rl[rows], w[rows], spread[rows])
    eo, el = np.abs(o[rows] - ro[rows]), np.abs(lse[rows] - rl[rows])
    assert (eo <= bo).all(), (eo / bo).max()
    assert (el <= bl).all(), (el / bl).max()


# lengths of queries and keys: one token, tile edges, nothing, more queries than keys (rows that see nothing)
PROMPTS = [
    ([1], [1]), ([77], [77]), ([128], [128]), ([129, 1, 0, 64], [129, 1, 0, 64]), ([3, 40, 200], [3, 40, 200]),
    ([5, 0, 30], [0, 17, 7]), ([140, 20], [130, 3]), ([17, 33], [300, 129]), ([1, 1, 1], [513, 1, 0]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(1, 1, 128), (6, 2, 64), (5, 1, 128), (8, 8, 64)])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_against_oracle(dtype, causal, heads, case):
    H, Hk, d = heads
    nq, nk = PROMPTS[case]
    g = torch.Generator(device="cuda").manual_seed(17 * case + H)
    qs, ks = starts(nq, case % 3), starts(nk, case % 2)
    layout = "heads" if case % 2 else "tokens"
    q = view(g, H, qs[-1] + case % 4, d, DT[dtype], layout, 2.0)
    Tk = max(1, ks[-1] + (case + 1) % 3)
    k, v = view(g, Hk, Tk, d, DT[dtype], "heads" if case % 3 else "tokens"), view(g, Hk, Tk, d, DT[dtype], layout)
    check(q, k, v, qs, ks, causal, out="tokens" if case % 2 else "heads")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(3, 3), (6, 2), (8, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_prompts(d, heads, causal):
    """Several tiles of queries and of keys, prompts and chunks, more blocks than items a head and the other way round."""
    H, Hk = heads
    g = torch.Generator(device="cuda").manual_seed(4)
    for nq, nk in (([700, 259, 30], [700, 259, 30]), ([300, 5, 600], [1111, 900, 200])):
        qs, ks = starts(nq), starts(nk)
        q, k, v = view(g, H, qs[-1], d, torch.bfloat16, "tokens", 2.0), view(g, Hk, ks[-1], d, torch.bfloat16, "tokens"), view(g, Hk, ks[-1], d, torch.bfloat16, "heads")
        check(q, k, v, qs, ks, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nk", [([1] * 4, [2000, 700, 5, 1500]), ([3, 1, 2], [900, 0, 2500]), ([40, 7], [1100, 1300])])
@pytest.mark.parametrize("causal", [True, False])
def test_cut_sequences(dtype, d, nq, nk, causal):
    """Few queries over long keys: sequences are cut and joined again."""
    g = torch.Generator(device="cuda").manual_seed(5)
    qs, ks = starts(nq), starts(nk)
    q, k, v = view(g, 8, qs[-1], d, DT[dtype], "tokens", 2.0), view(g, 2, ks[-1], d, DT[dtype], "tokens"), view(g, 2, ks[-1], d, DT[dtype], "heads")
    desc = mcs.packed_desc(len(nq), qs[-1], ks[-1], 8, 2, d, DT[dtype], causal, max(nq))
    assert mcs.packed_attn_workspace(desc).numel() > 16  # the plan cuts
    check(q, k, v, qs, ks, causal, max_q=max(nq))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [3, 7, 33, 64])
def test_groups_that_do_not_fill_a_tile(dtype, group):
    g = torch.Generator(device="cuda").manual_seed(group)
    qs = starts([19, 4])
    q, k, v = view(g, group, 23, 64, DT[dtype], "heads", 2.0), view(g, 1, 23, 64, DT[dtype], "tokens"), view(g, 1, 23, 64, DT[dtype], "tokens")
    check(q, k, v, qs, qs, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores_and_own_scale(dtype):
    """Maxima that grow from tile to tile by more than 2^8, and a scale of the caller's."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (view(g, 2, 400, 64, DT[dtype], "heads", s) for s in (3.0, 1.0, 1.0))
    k *= torch.linspace(0.2, 4.0, 400, device="cuda").to(k.dtype)[None, :, None]
    check(q, k, v, [0, 400], [0, 400], True, scale=0.25)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_masked_values_have_no_effect(dtype, cut, poison):
    """Keys and values behind a sequence, of other sequences and of later tokens may be anything."""
    g = torch.Generator(device="cuda").manual_seed(11)
    nq, nk = ([2, 2, 2], [700, 1000, 600]) if cut else ([40, 70, 150], [40, 70, 150])
    qs, ks = starts(nq), starts(nk)
    Tk = ks[-1] + 9
    q, k, v = (view(g, h, n, 128, DT[dtype], "heads", 2.0) for h, n in ((4, qs[-1]), (2, Tk), (2, Tk)))
    a = call(q, k, v, qs, ks, True, max(nq))
    kp, vp = k.clone(), v.clone()
    for x in (kp, vp):
        x[:, ks[1]:ks[2]] = poison          # the whole second sequence
        x[:, ks[3]:] = poison               # behind the last one
        x[:, ks[3] - 1] = poison            # the third's last key, which only its last query sees
    b = call(q, kp, vp, qs, ks, True, max(nq))
    mcs.mcs_check_status()
    keep = torch.ones(qs[-1], dtype=torch.bool, device="cuda")
    keep[qs[1]:qs[2]] = False
    keep[-1] = False
    for x, y in zip(a, b):
        assert torch.equal(x[:, keep], y[:, keep])
        assert not torch.isfinite(y[:, ~keep].float()).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_values_that_some_rows_see(dtype):
    """An infinity in one element of V reaches exactly the rows that see its key, in its column, with its sign."""
    g = torch.Generator(device="cuda").manual_seed(12)
    q, k, v = (view(g, h, 150, 64, DT[dtype], "heads", 1.0) for h in (2, 2, 2))
    v[0, 60, 5], v[1, 140, 63], v[1, 3, 0] = float("inf"), float("-inf"), float("nan")
    o, _ = call(q, k, v, [0, 150], [0, 150], True)
    want = torch.zeros((2, 150, 64), device="cuda")
    want[0, 60:, 5], want[1, 140:, 63], want[1, 3:, 0] = float("inf"), float("-inf"), float("nan")
    o = o.float()
    assert torch.equal(torch.isfinite(o), torch.isfinite(want))
    assert torch.equal(o[torch.isinf(want)], want[torch.isinf(want)])
    assert torch.isnan(o[torch.isnan(want)]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_of_nan(dtype):
    """A query of NaN gives NaN to its own row and to no other."""
    g = torch.Generator(device="cuda").manual_seed(13)
    q, k, v = (view(g, 2, 90, 64, DT[dtype], "heads", 1.0) for _ in range(3))
    a, la = call(q, k, v, [0, 90], [0, 90], True)
    q[1, 30, 2] = float("nan")
    b, lb = call(q, k, v, [0, 90], [0, 90], True)
    assert torch.isnan(b[1, 30]).all() and torch.isnan(lb[1, 30])
    b[1, 30], lb[1, 30] = a[1, 30], la[1, 30]
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_bounds_are_flagged():
    g = torch.Generator(device="cuda").manual_seed(14)
    q, k, v = (view(g, 2, 60, 64, torch.bfloat16, "heads") for _ in range(3))
    for dt in (torch.bfloat16, torch.float32):
        for qs, ks, most in (([0, 70], [0, 60], 0), ([0, 30, 20, 60], [0, 20, 40, 60], 0), ([0, 60], [0, 61], 0),
                             ([-3, 60], [0, 60], 0), ([0, 60], [-1, 60], 0), ([0, 20, 60], [0, 20, 60], 39)):
            call(q.to(dt), k.to(dt), v.to(dt), qs, ks, True, most)
            with pytest.raises(mcs.McsError) as e:
                mcs.mcs_check_status()
            assert e.value.code == 5
            mcs.mcs_check_status()


def test_output_without_lse_and_equal_bits():
    g = torch.Generator(device="cuda").manual_seed(15)
    q, k, v = (view(g, h, 1500, 128, torch.bfloat16, "tokens", 2.0) for h in (8, 2, 2))
    a, la = call(q, k, v, [0, 700, 1500], [0, 700, 1500], True)
    b, lb = call(q, k, v, [0, 700, 1500], [0, 700, 1500], True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    desc = mcs.packed_desc(2, 1500, 1500, 8, 2, 128, q.dtype)
    st = torch.tensor([0, 700, 1500], dtype=torch.int32, device="cuda")
    c = torch.empty_like(a)
    mcs.mcs_packed_attn(desc, q, k, v, st, st, c, None, mcs.packed_attn_workspace(desc))
    assert torch.equal(a, c)


def test_stream_and_captured_graph():
    """On another stream, and captured with lengths that change between replays."""
    g = torch.Generator(device="cuda").manual_seed(16)
    q, k, v = view(g, 8, 6, 128, torch.bfloat16, "tokens", 2.0), *(view(g, 2, 4000, 128, torch.bfloat16, "tokens") for _ in range(2))
    lengths = [([0, 2, 6], [0, 1000, 4000]), ([0, 5, 6], [0, 3900, 3950]), ([0, 0, 3], [0, 0, 2500])]
    want = [call(q, k, v, a, b, True) for a, b in lengths]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [call(q, k, v, a, b, True) for a, b in lengths]
    s.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    desc = mcs.packed_desc(2, 6, 4000, 8, 2, 128, q.dtype)
    ws = mcs.packed_attn_workspace(desc)
    qs, ks = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    o, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    mcs.mcs_packed_attn(desc, q, k, v, qs, ks, o, lse, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mcs.mcs_packed_attn(desc, q, k, v, qs, ks, o, lse, ws)
    for (a, b), (wo, wl) in zip(lengths, want):
        qs.copy_(torch.tensor(a)), ks.copy_(torch.tensor(b))
        o.fill_(7.0), lse.fill_(7.0)
        ws.fill_(255)  # what is in the workspace does not matter
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(lse, wl)
    mcs.mcs_check_status()


def test_offsets_past_31_bits():
    """Keys and values whose offsets pass 2^31 elements and 2^32 bytes."""
    Tk, Hk, d = 2_200_000, 8, 128
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    g = torch.Generator(device="cuda").manual_seed(18)
    k, v = (torch.empty((Tk, Hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 300
    for x in (k, v):
        x[-n:] = torch.randn((n, Hk, d), generator=g, device="cuda").to(x.dtype)
    q = view(g, 16, 4, d, torch.bfloat16, "tokens", 2.0)
    small = call(q, k[-n:].transpose(0, 1), v[-n:].transpose(0, 1), [0, 4], [0, n], True, 4)
    large = call(q, k.transpose(0, 1), v.transpose(0, 1), [0, 4], [Tk - n, Tk], True, 4)
    mcs.mcs_check_status()
    # the plans differ (cut or not), so equal up to roundings
    assert torch.allclose(small[0].float(), large[0].float(), atol=2.0 ** -6) and torch.allclose(small[1], large[1], atol=1e-5)


def test_many_sequences():
    """More sequences than a warp looks at in one step, most of them empty."""
    g = torch.Generator(device="cuda").manual_seed(19)
    n = [(7 * i) % 3 if i % 5 else 0 for i in range(3000)]
    n[1234] = 40
    st = starts(n)
    for dtype in ("bf16", "f32"):
        q, k, v = (view(g, 2, st[-1], 64, DT[dtype], "tokens", 2.0) for _ in range(3))
        check(q, k, v, st, st, True)


def test_other_device_is_refused():
    if torch.cuda.device_count() > 1:
        pytest.skip("one device here")
    q = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    desc = mcs.packed_desc(1, 8, 8, 2, 2, 64, q.dtype)
    st = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mcs.mcs_packed_attn(desc, q, q, q, st, st, torch.empty_like(q), None, mcs.packed_attn_workspace(desc))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_masked_values_have_no_effect_in_cut_prompts(d, poison):
    """The same where sequences of several tiles are cut along their keys."""
    g = torch.Generator(device="cuda").manual_seed(20)
    nq, nk = [70, 90, 80], [1100, 1300, 900]
    qs, ks = starts(nq), starts(nk)
    Tk = ks[-1] + 9
    q, k, v = (view(g, h, n, d, torch.bfloat16, "heads", 2.0) for h, n in ((4, qs[-1]), (2, Tk), (2, Tk)))
    desc = mcs.packed_desc(3, qs[-1], Tk, 4, 2, d, q.dtype, True, max(nq))
    assert mcs.packed_attn_workspace(desc).numel() > 16  # the plan cuts
    a = call(q, k, v, qs, ks, True, max(nq))
    kp, vp = k.clone(), v.clone()
    for x in (kp, vp):
        x[:, ks[1]:ks[2]] = poison
        x[:, ks[3]:] = poison
        x[:, ks[3] - 1] = poison            # only the last query sees it
    b = call(q, kp, vp, qs, ks, True, max(nq))
    mcs.mcs_check_status()
    keep = torch.ones(qs[-1], dtype=torch.bool, device="cuda")
    keep[qs[1]:qs[2]] = False
    keep[-1] = False
    for x, y in zip(a, b):
        assert torch.equal(x[:, keep], y[:, keep])
        assert not torch.isfinite(y[:, ~keep].float()).any()


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_that_some_rows_see_in_cut_prompts(d):
    """100 queries behind 1,100 kept keys: query i sees the keys up to 1,100 + i."""
    g = torch.Generator(device="cuda").manual_seed(21)
    q, k, v = (view(g, 2, n, d, torch.bfloat16, "heads", 1.0) for n in (100, 1200, 1200))
    q = torch.cat([q, q])  # two query heads a key head
    desc = mcs.packed_desc(1, 100, 1200, 4, 2, d, q.dtype, True, 100)
    assert mcs.packed_attn_workspace(desc).numel() > 16
    v[0, 1150, 5], v[1, 1199, 63], v[1, 10, 0] = float("inf"), float("-inf"), float("nan")
    o, _ = call(q, k, v, [0, 100], [0, 1200], True, 100)
    want = torch.zeros((4, 100, d), device="cuda")
    want[:2, 50:, 5], want[2:, 99:, 63], want[2:, :, 0] = float("inf"), float("-inf"), float("nan")
    o = o.float()
    assert torch.equal(torch.isfinite(o), torch.isfinite(want))
    assert torch.equal(o[torch.isinf(want)], want[torch.isinf(want)])
    assert torch.isnan(o[torch.isnan(want)]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_single_tokens_over_cut_keys(dtype):
    """More sequences than a warp has lanes, a token each or none, over keys that are cut."""
    g = torch.Generator(device="cuda").manual_seed(22)
    nq = [0 if i % 11 == 5 else 1 for i in range(48)]
    nk = [(137 * i * i) % 1900 if i % 7 else 0 for i in range(48)]
    qs, ks = starts(nq), starts(nk)
    q, k, v = view(g, 8, qs[-1], 128, DT[dtype], "tokens", 2.0), view(g, 2, ks[-1], 128, DT[dtype], "tokens"), view(g, 2, ks[-1], 128, DT[dtype], "heads")
    desc = mcs.packed_desc(48, qs[-1], ks[-1], 8, 2, 128, DT[dtype], True, 1)
    assert mcs.packed_attn_workspace(desc).numel() > 16
    check(q, k, v, qs, ks, True, max_q=1)


def test_two_streams_at_once():
    """Calls that may run side by side, each with a workspace of its own."""
    g = torch.Generator(device="cuda").manual_seed(23)
    calls = []
    for nq, nk in (([1] * 6, [2000, 300, 1500, 40, 900, 1111]), ([300, 5, 200], [300, 5, 200])):
        qs, ks = starts(nq), starts(nk)
        q, k, v = view(g, 8, qs[-1], 128, torch.bfloat16, "tokens", 2.0), *(view(g, 2, ks[-1], 128, torch.bfloat16, "tokens") for _ in range(2))
        calls.append((q, k, v, qs, ks, True, max(nq)))
    want = [call(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(20):
        for c, s, out in zip(calls, streams, got):
            with torch.cuda.stream(s):
                out.append(call(*c))
    torch.cuda.synchronize()
    for w, out in zip(want, got):
        assert all(torch.equal(w[0], o) and torch.equal(w[1], l) for o, l in out)


@pytest.mark.parametrize("group,nq,nk", [
    (1, [32, 7, 0, 1], [32, 300, 40, 129]), (5, [6, 1, 3], [700, 900, 640]), (32, [1, 1, 0, 1], [1, 31, 64, 2500]),
    (8, [4, 4], [127, 3]), (2, [16, 5], [1000, 1030]), (4, [0 if i % 11 == 5 else 1 for i in range(48)], [(137 * i * i) % 1900 if i % 7 else 0 for i in range(48)]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_few_rows(group, nq, nk, causal):
    """Up to 32 rows a sequence with d = 64: four warps share a tile's keys."""
    g = torch.Generator(device="cuda").manual_seed(24)
    qs, ks = starts(nq), starts(nk)
    q, k, v = view(g, 2 * group, qs[-1], 64, torch.bfloat16, "tokens", 2.0), view(g, 2, ks[-1], 64, torch.bfloat16, "tokens"), view(g, 2, ks[-1], 64, torch.bfloat16, "heads")
    check(q, k, v, qs, ks, causal, max_q=max(nq))
    check(q, k, v, qs, ks, causal, max_q=max(nq), scale=0.6, out="tokens")


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_few_rows_masked_values_have_no_effect(cut, poison):
    g = torch.Generator(device="cuda").manual_seed(25)
    nq, nk = [2, 2, 2], [700, 1000, 600] if cut else [90, 70, 150]
    qs, ks = starts(nq), starts(nk)
    Tk = ks[-1] + 9
    q, k, v = (view(g, h, n, 64, torch.bfloat16, "heads", 2.0) for h, n in ((4, qs[-1]), (2, Tk), (2, Tk)))
    a = call(q, k, v, qs, ks, True, 2)
    kp, vp = k.clone(), v.clone()
    for x in (kp, vp):
        x[:, ks[1]:ks[2]] = poison
        x[:, ks[3]:] = poison
        x[:, ks[3] - 1] = poison
    b = call(q, kp, vp, qs, ks, True, 2)
    mcs.mcs_check_status()
    keep = torch.ones(qs[-1], dtype=torch.bool, device="cuda")
    keep[qs[1]:qs[2]] = False
    keep[-1] = False
    for x, y in zip(a, b):
        assert torch.equal(x[:, keep], y[:, keep])
        assert not torch.isfinite(y[:, ~keep].float()).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nk", [300, 1200])
def test_few_rows_infinite_values(d, nk):
    """4 queries, of which the i-th sees the keys up to nk - 4 + i: values that are not finite reach the rows that see them,
    in their columns, with their signs; two of unlike sign give NaN."""
    inf, nan = float("inf"), float("nan")
    g = torch.Generator(device="cuda").manual_seed(26)
    q, k, v = (view(g, h, n, d, torch.bfloat16, "heads", 1.0) for h, n in ((4, 4), (2, nk), (2, nk)))
    clean, lse = call(q, k, v, [0, 4], [0, nk], True, 4)
    v[0, 200, 5], v[0, 40, 6], v[0, 41, 6], v[1, 10, 0] = inf, inf, -inf, nan
    v[1, nk - 2, 63], v[1, 7, 31] = -inf, -inf
    o, l = call(q, k, v, [0, 4], [0, nk], True, 4)
    want = clean.float().clone()
    want[:2, :, 5], want[:2, :, 6], want[2:, :, 0], want[2:, 2:, 63], want[2:, :, 31] = inf, nan, nan, -inf, -inf
    assert torch.equal(torch.nan_to_num(o.float(), 123.0, 1e30, -1e30), torch.nan_to_num(want, 123.0, 1e30, -1e30))
    assert torch.equal(l, lse)


def test_few_rows_captured_graph():
    """Lengths that change between replays, with and without cuts."""
    g = torch.Generator(device="cuda").manual_seed(27)
    for most, cases in ((4000, [([0, 2, 6], [0, 1000, 4000]), ([0, 5, 6], [0, 3900, 3950]), ([0, 0, 3], [0, 0, 2500])]),
                        (300, [([0, 2, 6], [0, 100, 300]), ([0, 5, 6], [0, 290, 291]), ([0, 0, 3], [0, 0, 129])])):
        q, k, v = view(g, 8, 6, 64, torch.bfloat16, "tokens", 2.0), *(view(g, 2, most, 64, torch.bfloat16, "tokens") for _ in range(2))
        want = [call(q, k, v, a, b, True) for a, b in cases]
        desc = mcs.packed_desc(2, 6, most, 8, 2, 64, q.dtype)
        ws = mcs.packed_attn_workspace(desc)
        qs, ks = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
        o, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
        graph = torch.cuda.CUDAGraph()
        mcs.mcs_packed_attn(desc, q, k, v, qs, ks, o, lse, ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            mcs.mcs_packed_attn(desc, q, k, v, qs, ks, o, lse, ws)
        for (a, b), (wo, wl) in zip(cases, want):
            qs.copy_(torch.tensor(a)), ks.copy_(torch.tensor(b))
            o.fill_(7.0), lse.fill_(7.0)
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, wo) and torch.equal(lse, wl)
    mcs.mcs_check_status()
