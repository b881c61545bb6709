"""Requests of different lengths through a layer, as they are used together: packed hidden states, the projection with each
request's adapter, norms and rotary positions that start again in every sequence, attention within each sequence, and the
output projection with the adapters from the attention's head-by-head output. Every stage is held against the float64
oracle on the tensors it received; back to back and captured the chain gives the same bits as with a wait after every
stage. And an AttentionBlock whose projections carry adapters."""
import numpy as np
import pytest
import torch

from oracle import packed_oracle as po
from sparse_attention_diffusion_gb300 import mcs, schedule
from tests.test_adapters_gpu import projection_bound
from tests.test_layer_ops_gpu import DT, f64
from tests.test_packed_attn_gpu import bound, starts

pytestmark = pytest.mark.gpu


class Layer:
    """One layer over S packed prompts with grouped heads: 8 query heads on 2 key heads."""

    def __init__(self, dtype, lengths, d=64, H=8, Hk=2, hidden=320, rank=16, count=3, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        dt = DT[dtype]
        self.dtype, self.H, self.Hk, self.d, self.hidden, self.T = dtype, H, Hk, d, hidden, sum(lengths)
        T, F = self.T, (H + 2 * Hk) * d
        self.start = starts(lengths)
        self.which = [i % (count + 1) - 1 for i in range(len(lengths))]
        self.x = rnd(1, T, hidden).to(dt)
        self.w_in, self.w_out = (rnd(F, hidden) / hidden ** 0.5).to(dt), (rnd(hidden, H * d) / (H * d) ** 0.5).to(dt)
        self.wq, self.wk = (1 + 0.2 * rnd(d)).to(dt), (1 + 0.2 * rnd(d)).to(dt)
        lora = lambda i, o: ((rnd(count, rank, i) / i ** 0.5).to(dt), (0.3 * rnd(count, o, rank) / rank ** 0.5).to(dt))
        self.ad_in, self.ad_out = lora(hidden, F), lora(H * d, hidden)
        self.scale = 0.5 + torch.rand((count,), generator=g, device="cuda")
        at = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.d_start, self.d_which = at(self.start), at(self.which)
        self.pos = at(np.concatenate([np.arange(n) for n in lengths])).view(1, T, 1)
        self.rope = mcs.rope_desc((d,), (max(lengths),), style="half")
        self.table = mcs.rope_table(self.rope)
        self.dq, self.dk = mcs.make_desc(1, H, T, d, 64, dt), mcs.make_desc(1, Hk, T, d, 64, dt)
        self.p_in, self.p_out = mcs.linear_desc(1, T, hidden, F, dt), mcs.linear_desc(1, T, H * d, hidden, dt, heads=H)
        self.set = mcs.adapters_desc(count, rank, len(lengths))
        self.attn = mcs.packed_desc(len(lengths), T, T, H, Hk, d, dt, max_q=max(lengths))
        n = max(mcs.linear_adapters_workspace(p, self.set).numel() for p in (self.p_in, self.p_out))
        self.ws = torch.empty(max(n, mcs.packed_attn_workspace(self.attn).numel()), dtype=torch.uint8, device="cuda")
        new = lambda *s: torch.empty(s, dtype=dt, device="cuda")
        self.qkv, self.q, self.k, self.v = new(1, T, H + 2 * Hk, d), new(1, H, T, d), new(1, Hk, T, d), new(1, Hk, T, d)
        self.o, self.lse, self.y = new(1, H, T, d), torch.empty((H, T), device="cuda"), new(1, T, hidden)

    def run(self, after=lambda: None):
        H, Hk = self.H, self.Hk
        project = lambda p, x, w, res, ad, y: mcs.mcs_linear_adapters(p, self.set, x, w, None, None, res, *ad, self.scale,
                                                                      self.d_start, self.d_which, y, self.ws)
        project(self.p_in, self.x, self.w_in, None, self.ad_in, self.qkv.view(1, self.T, -1))
        after()
        rows = self.qkv.transpose(1, 2)  # [1, H + 2 Hk, T, d] views of the packed projection
        q, k, v = rows[:, :H], rows[:, H:H + Hk], rows[:, H + Hk:]
        mcs.mcs_qk_norm_rope(self.dq, self.rope, self.table, self.pos, q, None, None, self.wq, None, 1e-6, self.q, None, None)
        mcs.mcs_qk_norm_rope(self.dk, self.rope, self.table, self.pos, None, k, v, None, self.wk, 1e-6, None, self.k, self.v)
        after()
        mcs.mcs_packed_attn(self.attn, self.q[0], self.k[0], self.v[0], self.d_start, self.d_start, self.o[0], self.lse, self.ws)
        after()
        project(self.p_out, self.o, self.w_out, self.x, self.ad_out, self.y)
        after()
        return self.y


LENGTHS = [[37, 1, 130, 0, 64], [300, 5], [1] * 20, [700, 300]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_stages(dtype, lengths):
    L = Layer(dtype, lengths)
    L.run(torch.cuda.synchronize)
    mcs.mcs_check_status()
    T, H, Hk, d = L.T, L.H, L.Hk, L.d
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23

    def projection(x, w, ad, res, y):
        z, size, extra = po.adapted_projection(x, f64(w), None, L.start, L.which, f64(ad[0]), f64(ad[1]), f64(L.scale))
        tol = projection_bound(dtype, w.shape[1], ad[0].shape[1], size, extra)
        want = z + (0 if res is None else res)
        err = np.abs(f64(y).reshape(T, -1) - want)
        assert (err <= tol + (half + 2.0 ** -22) * (np.abs(want) + np.abs(z)) + 1e-30).all()

    projection(f64(L.x)[0], L.w_in, L.ad_in, None, L.qkv)
    packed = f64(L.qkv)[0].transpose(1, 0, 2)[None]
    pos = L.pos[0].cpu().numpy()
    ang = pos[:, 0][:, None] * 10000.0 ** (-2.0 * np.arange(d // 2) / d)
    for t, w, xin in ((L.q, L.wq, packed[:, :H]), (L.k, L.wk, packed[:, H:H + Hk])):
        r = xin / np.sqrt((xin ** 2).mean(-1, keepdims=True) + 1e-6) * f64(w)
        a, b = r[..., :d // 2], r[..., d // 2:]
        want = np.concatenate([a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)], -1)
        size = np.abs(np.concatenate([a, b], -1)) + np.abs(np.concatenate([b, a], -1))
        # the norm's sum (d products), reciprocal root, table (2^-23 of 1) and two products
        assert (np.abs(f64(t) - want) <= half * np.abs(want) + size * (d + 24) * 2.0 ** -24 + 1e-30).all()
    assert torch.equal(L.v[0], L.qkv[0, :, H + Hk:].transpose(0, 1))
    ro, rl, w, spread = po.packed_attention(f64(L.q)[0], f64(L.k)[0], f64(L.v)[0], L.start, L.start, True)
    bo, bl = bound(dtype, d, max(lengths), ro, rl, w, spread)
    assert (np.abs(f64(L.o)[0] - ro) <= bo).all() and (np.abs(f64(L.lse) - rl) <= bl).all()
    projection(f64(L.o)[0].transpose(1, 0, 2).reshape(T, H * d), L.w_out, L.ad_out, f64(L.x)[0], L.y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_back_to_back_and_captured(dtype, lengths):
    """One workspace for all calls, no waits between them, and a captured graph replayed over other hidden states."""
    L = Layer(dtype, lengths)
    want = L.run(torch.cuda.synchronize).clone()
    for _ in range(3):
        L.ws.fill_(255)
        assert torch.equal(L.run(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run()
    L.x.mul_(-0.5)
    graph.replay()
    got = L.y.clone()
    assert torch.equal(got, L.run(torch.cuda.synchronize))
    mcs.mcs_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_block_with_adapters(dtype):
    """Two samples with an adapter each; without adapters (all negative) the block gives what it gave before."""
    B, H, d, grid, hidden, rank = 2, 2, 64, (3, 5, 9), 128, 8
    N, dt = 135, DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    w = dict(w_qkv=rnd(3 * H * d, hidden) / 11, b_qkv=rnd(3 * H * d), wq=None, wk=None, w_out=rnd(hidden, H * d) / 11, b_out=rnd(hidden))
    x, gate = rnd(B, N, hidden), rnd(B, hidden)
    ad = schedule.BlockAdapters(rnd(2, rank, hidden) / 11, rnd(2, 3 * H * d, rank) / 3, rnd(2, rank, H * d) / 11, rnd(2, hidden, rank) / 3,
                                torch.tensor([0.7, 1.3], device="cuda"), torch.tensor([0, N, 2 * N], dtype=torch.int32, device="cuda"),
                                torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    rope = mcs.rope_desc((24, 20, 20), grid)

    def block(adapters):
        layer = schedule.MetaCacheLayer(mcs.make_desc(B, H, N, d, 64, dt), 40, dt, "cuda")
        return layer, schedule.AttentionBlock(layer, rope, adapters=adapters, **w)

    layer, b = block(ad)
    o = layer.dense(*b.inputs(x)).clone()
    y = b.output(o, x, gate, torch.empty_like(x))
    mcs.mcs_check_status()
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    for rows, wt, bias, dn, up, out, ep in ((f64(x).reshape(B * N, hidden), w["w_qkv"], w["b_qkv"], ad.down_qkv, ad.up_qkv, b.qkv, False),
                                            (f64(o).transpose(0, 2, 1, 3).reshape(B * N, H * d), w["w_out"], w["b_out"], ad.down_out, ad.up_out, y, True)):
        z, size, extra = po.adapted_projection(rows, f64(wt), f64(bias), [0, N, 2 * N], [1, 0], f64(dn), f64(up), f64(ad.scale))
        tol = projection_bound(dtype, wt.shape[1], rank, size + np.abs(f64(bias)), extra)
        want = z
        if ep:
            gt = np.repeat(f64(gate), N, axis=0)
            want, tol = f64(x).reshape(B * N, hidden) + gt * z, np.abs(gt) * tol + 2.0 ** -22 * np.abs(f64(x).reshape(B * N, hidden))
        assert (np.abs(f64(out).reshape(B * N, -1) - want) <= tol + (half + 2.0 ** -22) * (np.abs(want) + np.abs(z)) + 1e-30).all()
    ad.which.fill_(-1)
    plain_layer, plain = block(None)
    q = b.inputs(x)
    for s, t in zip(q, plain.inputs(x)):
        assert torch.equal(s, t)
    assert torch.equal(b.output(o, x, gate, torch.empty_like(x)), plain.output(o, x, gate, torch.empty_like(x)))
