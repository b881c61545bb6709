"""Rotary positions, query/key norms and projections against the float64 oracle.

Tolerances count roundings. u = 2^-24 (half a step of fp32, relative), and the store
rounds once more by at most r |y| with r = 2^-8 (bf16) or 2^-24 (fp32).
  * rotation: products with a rounded cosine and sine, then a sum: 3 u (|x0| + |x1|) a
    pair, counted as 4;
  * norm: 8 sequential adds and 5 shuffle adds of squares (14 u, half of it in rstd), rsqrt
    (2 ulp = 4 u), two products: 15 u on each normalised element, 4 u for the rotation: 20;
  * its gradient: 5 u on g, 15 u on xhat, 14 u for the sum over d, 16 u for dot * xhat,
    15 u for the factor rstd and the subtraction: 72 u of the terms' sizes;
  * weight gradients: 20 u a term, and one u for every add on the longest chain;
  * products: bf16 products are exact in fp32 and each of the K of them enters a sum once,
    with an error of at most 2^-23 of the absolute sum (a truncating adder; fp32 products
    add u): K 2^-23 sum |x w|;
  * activations: slope at most 1.13; exp(t) of a t with 4 u |t| and expf's 2 + 1.2 |t| ulp:
    (8 + 6 |t|) 2^-23 relative; erfc: 8 ulp and 2 z^2 u of its argument's rounding.
Values below fp32's normal range are flushed: 1e-37 absolute is added everywhere.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from sparse_attention_diffusion_gb300 import mcs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STORE = {"bf16": 2.0 ** -8, "f32": U}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mcs.load(build_if_missing=True)


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, bound, what):
    g = f64(got) if isinstance(got, torch.Tensor) else got
    assert g.shape == want.shape, (what, g.shape, want.shape)
    bad = ~(np.abs(g - want) <= bound + 1e-37)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{g[bad][0]} for {want[bad][0]}, allowed {np.broadcast_to(bound, want.shape)[bad][0]}")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape, dtype="f32"):
    return torch.randn(shape, generator=g).to(DT[dtype]).cuda()


def both(dims, lens, **kw):
    """The same rope for the library and for the oracle."""
    r = mcs.rope_desc(dims, lens, **kw)
    return r, mcs.rope_table(r), lo.rope(dims, lens, **kw)


# ---------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("dims,lens,kw", [
    ((24, 20, 20), (3, 4, 5), {}),
    ((64,), (33,), dict(theta=500.0)),
    ((44, 42, 42), (2, 1, 3), dict(start=(1e6, -7.5, 0), scale=(1.0, 0.25, 3.0))),
    ((2, 126), (1, 700), dict(theta=1e6)),
])
def test_table(dims, lens, kw):
    """Each entry within half a step of fp32 of the 64-bit value (angles of 1e6 carry 1e-10)."""
    r, table, _ = both(dims, lens, **kw)
    want = []
    for a, (da, la) in enumerate(zip(dims, lens)):
        p = np.arange(la)[:, None]
        f = kw.get("theta", 10000.0) ** (-2.0 * np.arange(da // 2) / da)
        ang = (kw.get("start", (0, 0, 0))[a] + p) * kw.get("scale", (1, 1, 1))[a] * f
        want.append(np.stack([np.cos(ang), np.sin(ang)], -1).reshape(-1, 2))
    want = np.concatenate(want)
    close(table, want, U * np.abs(want) + 1e-9, "table")


ROPE_CASES = [
    # dtype, B, H, N, d, dims, lens, rope options
    ("bf16", 1, 3, 60, 64, (24, 20, 20), (3, 4, 5), {}),
    ("bf16", 2, 2, 60, 128, (44, 42, 42), (3, 4, 5), dict(style="half")),
    ("bf16", 1, 5, 77, 128, (16, 56, 56), (4, 3, 5), dict(first=9, start=(99991, 0, 0))),
    ("bf16", 2, 1, 33, 64, (30, 34), (3, 11), dict(style="half")),
    ("f32", 1, 2, 41, 64, (64,), (41,), dict(theta=300.0)),
    ("f32", 2, 3, 50, 64, (10, 6), (5, 10), {}),                      # 16 of 64 elements turn
    ("f32", 1, 1, 1, 128, (44, 42, 42), (1, 1, 1), dict(start=(12.5, 3, 4))),
    ("f32", 1, 7, 130, 128, (44, 42, 42), (5, 5, 5), dict(style="half", first=5)),
]
CASE_IDS = [f"{c[0]}-B{c[1]}H{c[2]}N{c[3]}d{c[4]}" for c in ROPE_CASES]


def layouts(B, H, N, d, dtype):
    """Empty [B,H,N,d] views: head by head, token by token, and a slice of a packed buffer."""
    dt = DT[dtype]
    yield torch.zeros(B, H, N, d, dtype=dt, device="cuda")
    yield torch.zeros(B, N, H, d, dtype=dt, device="cuda").transpose(1, 2)
    yield torch.zeros(B, N + 2, 3, H + 1, d, dtype=dt, device="cuda")[:, 1:N + 1, 1, :H].transpose(1, 2)


@pytest.mark.parametrize("inverse", [False, True], ids=["fwd", "inv"])
@pytest.mark.parametrize("case", ROPE_CASES, ids=CASE_IDS)
def test_rope_apply(case, inverse):
    dtype, B, H, N, d, dims, lens, kw = case
    r, table, orc = both(dims, lens, **kw)
    desc = mcs.make_desc(B, H, N, d, 64, DT[dtype])
    data = rand(gen(5), B, H, N, d, dtype=dtype)
    want = lo.rotate(f64(data), orc, inverse=inverse)
    bound = STORE[dtype] * np.abs(want) + 4 * U * lo.pair_size(f64(data), orc)
    first = None
    for x in layouts(B, H, N, d, dtype):
        x.copy_(data)
        for out in layouts(B, H, N, d, dtype):
            mcs.mcs_rope_apply(desc, r, table, None, x, out, inverse)
            close(out, want, bound, "rope")
            first = out if first is None else first
            assert torch.equal(out, first), "layouts differ"
        whole = x._base.clone() if x._base is not None else x.clone()
        mcs.mcs_rope_apply(desc, r, table, None, x, x, inverse)          # in place
        assert torch.equal(x, first)
        if x._base is not None and x._base.numel() > x.numel():          # nothing around the view was touched
            mask = torch.ones_like(whole, dtype=torch.bool)
            mask[:, 1:N + 1, 1, :H] = False
            assert torch.equal(x._base[mask], whole[mask])
    mcs.mcs_check_status()


@pytest.mark.parametrize("style", ["interleaved", "half"])
@pytest.mark.parametrize("dtype,d,axes", [("bf16", 128, 3), ("bf16", 64, 2), ("f32", 64, 3), ("f32", 128, 1)])
def test_rope_listed_positions(dtype, d, axes, style):
    B, H, N = 2, 3, 53
    dims = {1: (d,), 2: (d // 2, d // 2), 3: (d - 2 * 20, 20, 20)}[axes]
    lens = (9, 1, 30)[:axes] if axes != 1 else (1000,)
    r, table, orc = both(dims, lens, style=style, start=(4096, 0, -15))
    g = gen(6)
    pos = torch.stack([torch.randint(0, n, (B, N), generator=g) for n in lens], -1).to(torch.int32)
    x = rand(g, B, H, N, d, dtype=dtype)
    desc = mcs.make_desc(B, H, N, d, 64, DT[dtype])
    out = torch.empty_like(x)
    mcs.mcs_rope_apply(desc, r, table, pos.cuda(), x, out)
    mcs.mcs_check_status()
    want = lo.rotate(f64(x), orc, pos.numpy())
    close(out, want, STORE[dtype] * np.abs(want) + 4 * U * lo.pair_size(f64(x), orc), "listed positions")


def test_rope_positions_out_of_range_are_flagged_and_skipped():
    B, H, N, d = 2, 2, 40, 64
    r, table, orc = both((24, 20, 20), (4, 5, 6))
    g = gen(7)
    pos = torch.stack([torch.randint(0, n, (B, N), generator=g) for n in (4, 5, 6)], -1).to(torch.int32)
    bad = {(0, 3): (4, 0, 0), (0, 39): (0, -1, 0), (1, 0): (0, 0, 2 ** 31 - 1)}
    for (b, n), p in bad.items():
        pos[b, n] = torch.tensor(p)
    x = rand(g, B, H, N, d, dtype="bf16")
    desc = mcs.make_desc(B, H, N, d, 64, torch.bfloat16)
    out = torch.full_like(x, 7.0)
    mcs.mcs_rope_apply(desc, r, table, pos.cuda(), x, out)
    with pytest.raises(mcs.McsError) as e:
        mcs.mcs_check_status()
    assert e.value.code == 5
    mcs.mcs_check_status()
    good = pos.clone()
    for b, n in bad:
        good[b, n] = 0
    want = lo.rotate(f64(x), orc, good.numpy())
    for b, n in bad:
        want[b, :, n] = 7.0
    close(out, want, STORE["bf16"] * np.abs(want) + 4 * U * lo.pair_size(f64(x), orc), "rows beside bad positions")
    # the gradient: bad tokens are left unwritten and add nothing to the weight gradients
    w = rand(g, d, dtype="bf16")
    dy, ws = rand(g, B, H, N, d, dtype="bf16"), mcs.qk_norm_rope_bwd_workspace(desc)
    res = []
    for p, y in ((pos, dy), (good, dy.clone())):
        if p is good:
            for b, n in bad:
                y[b, :, n] = 0
        dx, dw = torch.full_like(x, 7.0), torch.empty(d, device="cuda")
        mcs.mcs_qk_norm_rope_bwd(desc, r, table, p.cuda(), x, None, w, None, EPS, y, None, None, dx, None, None, dw,
                                 None, ws)
        res.append((dx, dw))
    with pytest.raises(mcs.McsError):
        mcs.mcs_check_status()
    for b, n in bad:
        assert bool((res[0][0][b, :, n] == 7.0).all())
        res[1][0][b, :, n] = 7.0
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_rope_infinities_and_nan_stay_in_their_pairs():
    r, table, _ = both((24, 20, 20), (3, 4, 5))
    desc = mcs.make_desc(1, 2, 60, 64, 64, torch.bfloat16)
    x = rand(gen(8), 1, 2, 60, 64, dtype="bf16")
    clean, out = torch.empty_like(x), torch.empty_like(x)
    mcs.mcs_rope_apply(desc, r, table, None, x, clean)
    x[0, 1, 17, 10], x[0, 0, 59, 63] = float("nan"), float("inf")
    mcs.mcs_rope_apply(desc, r, table, None, x, out)
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[0, 1, 17, 10:12] = keep[0, 0, 59, 62:64] = False
    assert torch.equal(out[keep], clean[keep])
    assert bool(out[0, 1, 17, 10:12].isnan().all()) and not bool(out[0, 0, 59, 62:64].isfinite().any())


# ---------------------------------------------------------------- norm + rotation
def norm_bound(x, w, want, dtype, orc):
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    return STORE[dtype] * np.abs(want) + 20 * U * lo.pair_size(x * rstd * w, orc)


@pytest.mark.parametrize("weights", [True, False], ids=["weights", "plain"])
@pytest.mark.parametrize("case", ROPE_CASES, ids=CASE_IDS)
def test_norm_forward(case, weights):
    dtype, B, H, N, d, dims, lens, kw = case
    r, table, orc = both(dims, lens, **kw)
    desc = mcs.make_desc(B, H, N, d, 64, DT[dtype])
    g = gen(9)
    qkv = rand(g, B, N, 3, H, d, dtype=dtype)
    qkv[:, N // 2, 0] = 0                                    # a row of zeros stays zero
    qkv[:, 0, 1] *= 1e-3
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    wq, wk = (rand(g, d, dtype=dtype) for _ in range(2)) if weights else (None, None)
    out = [torch.full((B, H, N, d), 3.0, dtype=DT[dtype], device="cuda") for _ in range(3)]
    mcs.mcs_qk_norm_rope(desc, r, table, None, q, k, v, wq, wk, EPS, *out)
    mcs.mcs_check_status()
    for i, (x, w) in enumerate(((q, wq), (k, wk))):
        xn, wn = f64(x), np.ones(d) if w is None else f64(w)
        want = lo.norm_rotate(xn, wn, EPS, orc)
        close(out[i], want, norm_bound(xn, wn, want, dtype, orc), "qk"[i])
    assert torch.equal(out[2], v)
    # one stream at a time gives the same bits
    for i in range(3):
        alone = torch.full_like(out[i], 3.0)
        args = [None] * 3
        args[i] = (q, k, v)[i]
        outs = [None] * 3
        outs[i] = alone
        mcs.mcs_qk_norm_rope(desc, r, table, None, *args, wq, wk, EPS, *outs)
        assert torch.equal(alone, out[i])


@pytest.mark.parametrize("case", ROPE_CASES, ids=CASE_IDS)
def test_norm_backward(case):
    dtype, B, H, N, d, dims, lens, kw = case
    r, table, orc = both(dims, lens, **kw)
    desc = mcs.make_desc(B, H, N, d, 64, DT[dtype])
    g = gen(10)
    qkv = rand(g, B, N, 3, H, d, dtype=dtype)
    q, k, _ = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    w = [rand(g, d, dtype=dtype) for _ in range(2)]
    dy = [rand(g, B, H, N, d, dtype=dtype) for _ in range(3)]
    grad = torch.full_like(qkv, 5.0)
    dq, dk, dv = (grad[:, :, i].transpose(1, 2) for i in range(3))
    dw = [torch.full((d,), 5.0, device="cuda") for _ in range(2)]
    ws = mcs.qk_norm_rope_bwd_workspace(desc)
    ws.fill_(255)                                            # NaN patterns: its contents on entry do not matter
    mcs.mcs_qk_norm_rope_bwd(desc, r, table, None, q, k, *w, EPS, *dy, dq, dk, dv, *dw, ws)
    mcs.mcs_check_status()
    for i, (x, dx) in enumerate(((q, dq), (k, dk))):
        xn, wn, yn = f64(x), f64(w[i]), f64(dy[i])
        want, wantw = lo.norm_rotate_grad(xn, wn, EPS, yn, orc)
        rstd = 1.0 / np.sqrt((xn * xn).mean(-1, keepdims=True) + EPS)
        G, xh = lo.pair_size(yn, orc), np.abs(xn * rstd)
        size = rstd * (G * np.abs(wn) + xh * (G * np.abs(wn) * xh).mean(-1, keepdims=True))
        close(dx, want, STORE[dtype] * np.abs(want) + 72 * U * size, "d" + "qk"[i])
        # chain: at most B H N terms on a lane, the block's rows and the blocks
        close(dw[i], wantw, (20 + min(B * H * N, 256) + 64) * U * (G * xh).sum((0, 1, 2)), "dw" + "qk"[i])
    assert torch.equal(dv, dy[2])
    again = [torch.empty_like(t) for t in dw]
    grad2 = torch.empty_like(grad)
    mcs.mcs_qk_norm_rope_bwd(desc, r, table, None, q, k, *w, EPS, *dy, *(grad2[:, :, i].transpose(1, 2) for i in range(3)),
                             *again, ws)
    assert torch.equal(grad, grad2) and torch.equal(again[0], dw[0]) and torch.equal(again[1], dw[1])
    # without weights and weight gradients, one stream
    dk3 = torch.empty(B, H, N, d, dtype=DT[dtype], device="cuda")
    kc = k.contiguous()
    mcs.mcs_qk_norm_rope_bwd(desc, r, table, None, None, kc, None, None, EPS, None, dy[1], None, None, dk3, None, None,
                             None, ws)
    want, _ = lo.norm_rotate_grad(f64(k), np.ones(d), EPS, f64(dy[1]), orc)
    rstd = 1.0 / np.sqrt((f64(k) ** 2).mean(-1, keepdims=True) + EPS)
    G, xh = lo.pair_size(f64(dy[1]), orc), np.abs(f64(k) * rstd)
    close(dk3, want, STORE[dtype] * np.abs(want) + 72 * U * rstd * (G + xh * (G * xh).mean(-1, keepdims=True)), "dk alone")


def test_norm_many_heads_and_tokens():
    """More rows than one wave of blocks, heads and tokens that fill no block."""
    B, H, N, d = 1, 41, 1013, 128
    r, table, orc = both((44, 42, 42), (7, 9, 16), style="interleaved", first=3)
    desc = mcs.make_desc(B, H, N, d, 64, torch.bfloat16)
    g = gen(11)
    q = rand(g, B, N, H, d, dtype="bf16").transpose(1, 2)
    w = rand(g, d, dtype="bf16")
    out = torch.empty(B, H, N, d, dtype=torch.bfloat16, device="cuda")
    mcs.mcs_qk_norm_rope(desc, r, table, None, q, None, None, w, None, EPS, out, None, None)
    want = lo.norm_rotate(f64(q), f64(w), EPS, orc)
    close(out, want, norm_bound(f64(q), f64(w), want, "bf16", orc), "q")
    dy, dx, dw = rand(g, B, H, N, d, dtype="bf16"), torch.empty_like(q), torch.empty(d, device="cuda")
    mcs.mcs_qk_norm_rope_bwd(desc, r, table, None, q, None, w, None, EPS, dy, None, None, dx, None, None, dw, None,
                             mcs.qk_norm_rope_bwd_workspace(desc))
    mcs.mcs_check_status()
    want, wantw = lo.norm_rotate_grad(f64(q), f64(w), EPS, f64(dy), orc)
    rstd = 1.0 / np.sqrt((f64(q) ** 2).mean(-1, keepdims=True) + EPS)
    G, xh, wn = lo.pair_size(f64(dy), orc), np.abs(f64(q) * rstd), np.abs(f64(w))
    size = rstd * (G * wn + xh * (G * wn * xh).mean(-1, keepdims=True))
    close(dx, want, STORE["bf16"] * np.abs(want) + 72 * U * size, "dq")
    close(dw, wantw, (20 + 256 + 64) * U * (G * xh).sum((0, 1, 2)), "dwq")


# ---------------------------------------------------------------- projections
def linear_bound(x, w, y, z, act, gate, dtype):
    xt = x if x.ndim == 3 else x.transpose(0, 2, 1, 3).reshape(x.shape[0], x.shape[2], -1)
    ez = (xt.shape[-1] + 2) * 2.0 ** -23 * (np.abs(xt) @ np.abs(w.T)) + 2 * U * np.abs(z)
    if act != "none":
        t = np.abs(z) if act == "silu" else 1.6 * np.abs(z + 0.044715 * z ** 3)
        rel = 8 + (2 * z * z if act == "gelu_erf" else 6 * t)
        ez = 1.13 * ez + rel * 2.0 ** -23 * np.abs(lo.activate(z, act))
    if gate is not None:
        ez = ez * np.abs(gate)[:, None, :] + U * np.abs(gate)[:, None, :] * np.abs(lo.activate(z, act))
    return ez + (STORE[dtype] + U) * np.abs(y)


def check_linear(dtype, B, N, K, O, act="none", bias=False, gate=False, residual=False, heads=0, seed=12):
    g = gen(seed)
    x = rand(g, B, N, K, dtype=dtype) if heads == 0 else rand(g, B, heads, N, K // heads, dtype=dtype)
    w = (torch.randn((O, K), generator=g) / K ** 0.5).to(DT[dtype]).cuda()
    b = rand(g, O, dtype=dtype) if bias else None
    ga = rand(g, B, O, dtype=dtype) if gate else None
    res = rand(g, B, N, O, dtype=dtype) if residual else None
    desc = mcs.linear_desc(B, N, K, O, DT[dtype], act=act, heads=heads)
    guard = torch.full((B * N * O + 64,), 9.0, dtype=DT[dtype], device="cuda")
    y = guard[:B * N * O].view(B, N, O)
    mcs.mcs_linear(desc, x, w, b, ga, res, y)
    mcs.mcs_check_status()
    n = lambda t: None if t is None else f64(t)
    want, z = lo.linear(f64(x), f64(w), n(b), n(ga), n(res), act)
    close(y, want, linear_bound(f64(x), f64(w), want, z, act, n(ga), dtype), "y")
    assert bool((guard[B * N * O:] == 9.0).all()), "written past the last row"
    y2 = torch.empty_like(y) if res is None else res.clone()
    mcs.mcs_linear(desc, x, w, b, ga, None if res is None else y2, y2)        # again, onto the residual
    assert torch.equal(y, y2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 64, 65, 128, 129, 300])
def test_linear_rows(dtype, M):
    check_linear(dtype, 1, M, 200, 136, bias=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,O", [
    (1, 8, 1), (3, 8, 9), (5, 64, 7), (130, 72, 127), (257, 520, 129), (40, 1032, 1000), (1, 4096, 2050), (2, 1536, 40),
    (64, 64, 4096), (515, 136, 264), (260, 2048, 520),
])
def test_linear_shapes(dtype, M, K, O):
    check_linear(dtype, 1, M, K, O, bias=O % 2 == 0, residual=O % 3 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("B,N,K,O", [(1, 70, 264, 200), (3, 5, 128, 72), (2, 131, 128, 33)])
def test_linear_epilogues(dtype, act, B, N, K, O):
    for bias, gate, residual in ((False, False, False), (True, False, True), (True, True, False), (True, True, True)):
        check_linear(dtype, B, N, K, O, act, bias, gate, residual)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,heads,N,d,O", [(1, 1, 1, 64, 8), (2, 3, 61, 64, 96), (1, 2, 260, 128, 200), (3, 2, 129, 128, 264),
                                           (2, 5, 1, 64, 320), (2, 2, 300, 64, 520)])
def test_linear_from_heads(dtype, B, heads, N, d, O):
    check_linear(dtype, B, N, heads * d, O, "none", True, True, True, heads=heads)


@pytest.mark.parametrize("M", [1, 40, 700])
def test_linear_infinities_and_nan_stay_in_their_rows(M):
    g = gen(13)
    K, O = 128, 72
    x, w = rand(g, 1, M, K, dtype="bf16"), rand(g, O, K, dtype="bf16")
    desc = mcs.linear_desc(1, M, K, O, torch.bfloat16, act="silu")
    clean, y = (torch.empty(1, M, O, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mcs.mcs_linear(desc, x, w, None, None, None, clean)
    x[0, M // 2, 5] = float("nan")
    mcs.mcs_linear(desc, x, w, None, None, None, y)
    keep = [m for m in range(M) if m != M // 2]
    assert torch.equal(y[0, keep], clean[0, keep]) and bool(y[0, M // 2].isnan().all())


def test_linear_wide_activations():
    """Logistic gates at arguments where exp over- and underflows."""
    z = torch.tensor([-3e38, -1e30, -300.0, -88.0, -20.0, -4.0, 0.0, 4.0, 20.0, 300.0, 1e30, 3e38])
    n = z.numel()
    x = torch.zeros(1, n, 8, device="cuda")
    x[0, :, 0] = z
    w = torch.zeros(1, 8, device="cuda")
    w[0, 0] = 1.0
    for act in ("gelu_tanh", "gelu_erf", "silu"):
        y = torch.empty(1, n, 1, device="cuda")
        mcs.mcs_linear(mcs.linear_desc(1, n, 8, 1, torch.float32, act=act), x, w, None, None, None, y)
        got = f64(y)[0, :, 0]
        assert np.array_equal(got[:2], [0, 0]) and np.array_equal(got[-3:], f64(z)[-3:]), (act, got)
        zc = f64(z)[3:9]
        t = np.abs(zc) if act == "silu" else 1.6 * np.abs(zc + 0.044715 * zc ** 3)
        want = lo.activate(zc, act)
        rel = 8 + (2 * zc * zc if act == "gelu_erf" else 6 * t)
        assert np.all(np.abs(got[3:9] - want) <= rel * 2.0 ** -23 * np.abs(want) + 1e-36), act


# ---------------------------------------------------------------- streams and graphs
def test_another_stream_and_a_captured_graph():
    B, H, N, d = 1, 3, 200, 64
    r, table, _ = both((24, 20, 20), (5, 5, 8))
    desc = mcs.make_desc(B, H, N, d, 64, torch.bfloat16)
    g = gen(14)
    x = rand(g, B, N, H * d, dtype="bf16")
    w = rand(g, 3 * H * d, H * d, dtype="bf16")
    wn = rand(g, d, dtype="bf16")
    ld = mcs.linear_desc(B, N, H * d, 3 * H * d, torch.bfloat16)
    ws = mcs.qk_norm_rope_bwd_workspace(desc)
    qkv = torch.empty(B, N, 3, H, d, dtype=torch.bfloat16, device="cuda")
    out = [torch.empty(B, H, N, d, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    grad, dw = torch.empty_like(qkv), [torch.empty(d, device="cuda") for _ in range(2)]

    def chain():
        mcs.mcs_linear(ld, x, w, None, None, None, qkv.view(B, N, -1))
        q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
        mcs.mcs_qk_norm_rope(desc, r, table, None, q, k, v, wn, wn, EPS, *out)
        mcs.mcs_qk_norm_rope_bwd(desc, r, table, None, q, k, wn, wn, EPS, *out,
                                 *(grad[:, :, i].transpose(1, 2) for i in range(3)), *dw, ws)

    def results():
        return [t.clone() for t in (qkv, *out, grad, *dw)]

    chain()
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in (qkv, *out, grad, *dw):
            t.zero_()
        chain()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for seed in (15, 16):
        x.copy_(rand(gen(seed), B, N, H * d, dtype="bf16"))
        chain()
        want = results()
        for t in (qkv, *out, grad, *dw):
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    mcs.mcs_check_status()


def test_strides_past_32_bits():
    """Two heads 2^31 elements apart, a few tokens of each."""
    d, N = 64, 5
    span = 2 ** 31 + 64
    buf = torch.empty(span + N * d, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((1, 2, N, d), (0, span, d, 1))
    x.copy_(rand(gen(17), 1, 2, N, d, dtype="bf16"))
    r, table, orc = both((24, 20, 20), (1, 1, 5))
    desc = mcs.make_desc(1, 2, N, d, 64, torch.bfloat16)
    out = torch.empty(1, 2, N, d, dtype=torch.bfloat16, device="cuda")
    mcs.mcs_rope_apply(desc, r, table, None, x, out)
    want = lo.rotate(f64(x), orc)
    close(out, want, STORE["bf16"] * np.abs(want) + 4 * U * lo.pair_size(f64(x), orc), "far head")
    mcs.mcs_rope_apply(desc, r, table, None, x, x)
    assert torch.equal(x, out)
    mcs.mcs_check_status()
