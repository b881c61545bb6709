"""Projections with an adapter for each segment of rows against the float64 oracle: both bf16 kernels and fp32, ragged
and empty segments, rows without an adapter, what another request's rows and adapters hold."""
import numpy as np
import pytest
import torch

from oracle import packed_oracle as orc
from sparse_attention_diffusion_gb300 import mcs

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def projection_bound(dtype, din, R, size, extra):
    """The documented bounds of the sums: of the product with R more columns in two parts, of h, of its rounding. size and
    extra: sums of absolute products (oracle)."""
    if dtype == "bf16":
        tol = ((504 + 5.25 * 2 * (R / 16 + 1)) * 2.0 ** -23 + (din / 1024 + 9) * 2.0 ** -24) * (size + extra)
        return tol + extra * (2.0 ** -16 + (din / 16 + 2) * 5.25 * 2.0 ** -23)
    return (12 * 2.0 ** -23 + (din / 32 + 11) * 2.0 ** -24) * size + extra * (din + R + 8) * 2.0 ** -24 + (size + extra) * 2.0 ** -23


class Case:
    def __init__(self, dtype, B, N, din, dout, rank, start, which, count=3, act="none", heads=0, gated=False, bias=True, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 31 * rank + N)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        dt = DT[dtype]
        self.dtype, self.start, self.which, self.act, self.heads = dtype, start, which, act, heads
        self.x = (rnd(B, heads, N, din // heads) if heads else rnd(B, N, din)).to(dt)
        self.w, self.bias = (rnd(dout, din) / din ** 0.5).to(dt), (rnd(dout).to(dt) if bias else None)
        self.gate = rnd(B, dout).to(dt) if gated else None
        self.residual = rnd(B, N, dout).to(dt) if gated else None
        self.down, self.up = (rnd(count, rank, din) / din ** 0.5).to(dt), (rnd(count, dout, rank) / rank ** 0.5).to(dt)
        self.scale = 0.5 + torch.rand((count,), generator=g, device="cuda")
        self.desc = mcs.linear_desc(B, N, din, dout, dt, act=act, heads=heads)
        self.adapters = mcs.adapters_desc(count, rank, len(which))
        self.y = torch.empty((B, N, dout), dtype=dt, device="cuda")

    def run(self, y=None, stream=None, ws=None, residual=None):
        y = torch.full_like(self.y, 7.0) if y is None else y
        if ws is None:
            ws = mcs.linear_adapters_workspace(self.desc, self.adapters)
            ws.fill_(255)  # NaN: what is in the workspace does not matter
        at = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        mcs.mcs_linear_adapters(self.desc, self.adapters, self.x, self.w, self.bias, self.gate, residual if residual is not None else self.residual,
                                self.down, self.up, self.scale, at(self.start), at(self.which), y, ws, stream)
        return y

    def check(self):
        y = self.run()
        mcs.mcs_check_status()
        f = lambda t: None if t is None else t.float().cpu().numpy().astype(np.float64)
        B, N, dout = self.y.shape
        din, R = self.w.shape[1], self.down.shape[1]
        x = f(self.x.transpose(1, 2) if self.heads else self.x).reshape(B * N, din)
        z, size, extra = orc.adapted_projection(x, f(self.w), f(self.bias), self.start, self.which, f(self.down), f(self.up), f(self.scale))
        if self.bias is not None:
            size = size + np.abs(f(self.bias))
        tol = projection_bound(self.dtype, din, R, size, extra)
        if self.act == "silu":
            v = z / (1 + np.exp(-z))
        elif self.act == "gelu_tanh":
            v = z / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
        else:
            v = z
        if self.act != "none":  # slopes below 1.13; exponential and division
            tol = 1.13 * tol + np.abs(v) * (2.0 ** -14 if self.dtype == "bf16" else 2.0 ** -20) + 1e-30
        if self.gate is not None:
            gate = np.repeat(f(self.gate), N, axis=0)
            v, tol = f(self.residual).reshape(B * N, dout) + gate * v, np.abs(gate) * tol + 2.0 ** -23 * np.abs(f(self.residual).reshape(B * N, dout))
        half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -23
        tol = tol + half * (np.abs(v) + tol) + 1e-30
        err = np.abs(f(y).reshape(B * N, dout) - v)
        assert np.isfinite(err).all() and (err <= tol).all(), (err / tol).max()


SEGMENTS = [  # of 300 rows: one for all; ragged, empty ones, without an adapter, gaps at both ends; a row each at first
    ([0, 300], [1]),
    ([0, 17, 17, 130, 200, 300], [2, 0, -1, 0, 1]),
    ([5, 40, 256, 290], [0, 1, 2]),
    (list(range(0, 41)) + [300], [i % 4 - 1 for i in range(40)] + [2]),
    ([10, 20], [-1]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", range(len(SEGMENTS)))
@pytest.mark.parametrize("rank,din,dout", [(8, 64, 40), (24, 200, 129), (64, 1600, 256), (136, 72, 64), (256, 2048, 96)])
def test_against_oracle(dtype, seg, rank, din, dout):
    start, which = SEGMENTS[seg]
    Case(dtype, 1, 300, din, dout, rank, start, which, seed=seg).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("heads", [0, 3])
def test_epilogue_and_layouts(dtype, act, heads):
    """Batches with a gate each, heads side by side, segments that span batches."""
    Case(dtype, 3, 50, 384, 200, 16, [3, 60, 61, 150], [1, 0, 2], act=act, heads=heads, gated=True).check()


@pytest.mark.parametrize("rows,dout,din,kernel", [(9000, 512, 128, "pairs"), (8600, 250, 1664, "pairs"), (9000, 1024, 256, "pairs"),
                                                  (1, 4096, 4096, "few"), (8, 512, 4096, "few"), (200, 256, 5120, "few")])
@pytest.mark.parametrize("rank", [16, 72])
@pytest.mark.parametrize("heads", [False, True])
def test_kernels(rows, dout, din, kernel, rank, heads):
    """Both kernels of the product, with one and with several accumulators a row, slices of K, tiles of several segments."""
    B, N = (2, rows // 2) if heads and rows > 1 else (1, rows)
    cut = sorted({0, rows // 7, rows // 3, rows // 3 + 1, rows // 2, rows})
    which = [i % 4 - 1 for i in range(1, len(cut))]
    c = Case("bf16", B, N, din, dout, rank, cut, which, heads=din // 128 if heads else 0, gated=heads)
    assert mcs.mcs_linear_plan(c.desc, residual=heads)[0] == kernel
    c.check()


def test_decode_rows_with_their_own_adapters():
    """A row a segment: 70 requests, some without an adapter."""
    Case("bf16", 1, 70, 1024, 1024, 16, list(range(71)), [i % 33 - 1 for i in range(70)], count=32).check()
    Case("f32", 1, 70, 1024, 256, 16, list(range(71)), [i % 33 - 1 for i in range(70)], count=32).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dout,din", [(300, 200, 640), (6000, 512, 256), (5, 512, 2048)])
def test_without_adapters_equals_the_product(dtype, rows, dout, din):
    c = Case(dtype, 1, rows, din, dout, 16, [0, rows], [-1], gated=True, act="silu")
    y = torch.empty_like(c.y)
    mcs.mcs_linear(c.desc, c.x, c.w, c.bias, c.gate, c.residual, y)
    assert torch.equal(c.run(), y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dout,din", [(300, 200, 640), (6000, 512, 256)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["x", "down", "up", "scale"])
def test_other_requests_have_no_effect(dtype, rows, dout, din, poison, what):
    c = Case(dtype, 1, rows, din, dout, 16, [0, rows // 3, rows // 3 + 2, rows], [0, 1, 2])
    a = c.run()
    if what == "x":
        c.x[:, rows // 3:rows // 3 + 2] = poison
    else:
        getattr(c, what)[1].view(-1)[5 if what != "scale" else 0] = poison
    b = c.run()
    mcs.mcs_check_status()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[rows // 3:rows // 3 + 2] = False
    assert torch.equal(a[:, keep], b[:, keep])
    mine = b[:, ~keep].float()
    if what == "up" and dtype == "bf16":
        assert torch.isnan(mine).all()
    else:
        assert not torch.isfinite(mine).all()


def test_residual_in_place_stream_and_equal_bits():
    for rows, dout in ((300, 256), (6000, 512)):
        c = Case("bf16", 1, rows, 512, dout, 32, [0, rows // 2, rows], [0, 2], gated=True)
        y = c.run()
        assert torch.equal(c.run(), y)
        r = c.residual.clone()
        assert torch.equal(c.run(y=r, residual=r), y)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            z = c.run()
        s.synchronize()
        assert torch.equal(z, y)


def test_back_to_back_equals_synchronised():
    """Calls that share a workspace one behind the other: a call's slabs are not overwritten before they are read."""
    cases = [Case("bf16", 1, n, 512, 384, 32, [0, n // 2, n], [0, 2], seed=n) for n in (6000, 40, 300, 5000, 64)]
    ws = torch.empty(max(mcs.linear_adapters_workspace(c.desc, c.adapters).numel() for c in cases), dtype=torch.uint8, device="cuda")
    want = []
    for c in cases:
        want.append(c.run(ws=ws))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [c.run(ws=ws) for c in cases]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_graph(dtype):
    """Segments and adapters that change between replays."""
    c = Case(dtype, 1, 300, 512, 256, 32, [0, 100, 300], [0, 2])
    ws = mcs.linear_adapters_workspace(c.desc, c.adapters)
    st, wh = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (c.start, c.which))
    y = torch.empty_like(c.y)
    call = lambda: mcs.mcs_linear_adapters(c.desc, c.adapters, c.x, c.w, c.bias, None, None, c.down, c.up, c.scale, st, wh, y, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for start, which in (([0, 100, 300], [0, 2]), ([0, 0, 299], [1, 1]), ([30, 31, 32], [-1, 2])):
        st.copy_(torch.tensor(start)), wh.copy_(torch.tensor(which))
        graph.replay()
        c.start, c.which = start, which
        assert torch.equal(y, c.run())
    mcs.mcs_check_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_are_flagged(dtype):
    for start, which in (([0, 301], [0]), ([-1, 300], [0]), ([0, 200, 100], [0, 1]), ([0, 300], [3]), ([0, 10, 300], [0, 99])):
        c = Case(dtype, 1, 300, 128, 64, 8, start, which)
        y = c.run()
        with pytest.raises(mcs.McsError) as e:
            mcs.mcs_check_status()
        assert e.value.code == 5
        mcs.mcs_check_status()
        if which[-1] >= 3:  # no such adapter: the projection alone
            c.which = [w if w < 3 else -1 for w in which]
            assert torch.equal(y, c.run())


def test_many_segments():
    rows = 3000
    start = [i * rows // 2000 for i in range(2001)]
    Case("bf16", 1, rows, 128, 96, 16, start, [i % 6 - 2 for i in range(2000)], count=4).check()
    Case("f32", 1, rows, 128, 96, 16, start, [i % 6 - 2 for i in range(2000)], count=4).check()


def test_two_streams_at_once():
    """Calls that may run side by side, each with a workspace of its own."""
    cases = [Case("bf16", 1, n, 512, 384, 32, [0, n // 2, n], [0, 2], seed=n) for n in (6000, 300)]
    cases.append(Case("bf16", 1, 64, 512, 384, 16, list(range(65)), [i % 3 for i in range(64)], seed=64))
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], [[] for _ in cases]
    for _ in range(20):
        for c, s, out in zip(cases, streams, got):
            with torch.cuda.stream(s):
                out.append(c.run())
    torch.cuda.synchronize()
    for w, out in zip(want, got):
        assert all(torch.equal(w, y) for y in out)


@pytest.mark.parametrize("rows,dout,rank", [(256, 9000, 128), (700, 4096, 256), (60, 12000, 64), (6000, 512, 16)])
def test_large_up_is_looked_over_to_its_end(rows, dout, rank):
    """An element that is not finite anywhere in an adapter's `up` stays in its own rows."""
    cuts = [0, rows // 3, rows // 3 + 2, rows]
    c = Case("bf16", 1, rows, 256, dout, rank, cuts, [0, 1, 2])
    c.check()
    a = c.run()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[cuts[1]:cuts[2]] = False
    up = c.up[1].view(-1)
    for at in (0, up.numel() // 3 + 5, up.numel() // 2 + 7, up.numel() * 63 // 64, up.numel() - 1):
        old = up[at].item()
        up[at] = float("inf")
        b = c.run()
        up[at] = old
        assert torch.equal(a[:, keep], b[:, keep])
        assert not torch.isfinite(b[:, ~keep].float()).all()
    mcs.mcs_check_status()
    assert torch.equal(c.run(), a)


@pytest.mark.parametrize("rank,din,heads", [(4, 132, 0), (24, 640, 5), (64, 2432, 19), (136, 36, 0)])
def test_f32_many_rows(rank, din, heads):
    """fp32 with more rows than the first step takes one by one: ragged segments, rows without an adapter, heads."""
    rows = 2600
    for start, which in (([0, rows], [1]), ([3, 700, 700, 1301, 2599], [2, 1, -1, 0])):
        Case("f32", 2, rows // 2, din, 40, rank, start, which, heads=heads, act="silu", gated=True).check()
