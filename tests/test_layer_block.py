"""A block's attention run together: projection, norms with rotary positions, the
meta-cache schedule's dense, anchor and reuse steps, and the gated output projection.
Every stage is held against the float64 oracle on the tensors it received, with the
stages' own tolerances; a reuse step on the anchor's inputs gives the anchor's result."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from oracle import mcs_oracle as orc
from sparse_attention_diffusion_gb300 import mcs, schedule
from tests import parity
from tests.test_layer_ops_gpu import DT, STORE, close, f64, gen, linear_bound, norm_bound, rand

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, B, H, d, C, grid, text tokens behind it, hidden size, K
    ("f32", 1, 2, 64, 64, (3, 5, 9), 11, 96, 40),
    ("bf16", 2, 3, 128, 128, (4, 8, 10), 23, 256, 96),
    ("bf16", 1, 2, 64, 64, (2, 9, 9), 0, 136, 33),
]


def make(case, seed=30):
    dtype, B, H, d, C, grid, text, hidden, K = case
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    N = int(np.prod(grid)) + text
    desc = mcs.make_desc(B, H, N, d, C, DT[dtype])
    s = 2 * (d // 6)
    dims = (d - 2 * s, s, s)
    g = gen(seed)
    w = dict(w_qkv=(rand(g, 3 * H * d, hidden) / hidden ** 0.5).to(DT[dtype]), b_qkv=rand(g, 3 * H * d, dtype=dtype),
             wq=1 + 0.2 * rand(g, d, dtype=dtype), wk=1 + 0.2 * rand(g, d, dtype=dtype),
             w_out=(rand(g, hidden, H * d) / (H * d) ** 0.5).to(DT[dtype]), b_out=rand(g, hidden, dtype=dtype))
    layer = schedule.MetaCacheLayer(desc, K, DT[dtype], "cuda")
    block = schedule.AttentionBlock(layer, mcs.rope_desc(dims, grid), **w)
    x, gate = rand(g, B, N, hidden, dtype=dtype), 0.5 * rand(g, B, hidden, dtype=dtype)
    return layer, block, w, lo.rope(dims, grid), x, gate


@pytest.mark.parametrize("case", CASES, ids=[c[0] + f"-d{c[3]}" for c in CASES])
def test_stages(case):
    dtype, B, H, d = case[:4]
    layer, block, w, rope, x, gate = make(case)
    q, k, v = block.inputs(x)
    N = x.shape[1]
    want, z = lo.linear(f64(x), f64(w["w_qkv"]), f64(w["b_qkv"]))
    close(block.qkv, want, linear_bound(f64(x), f64(w["w_qkv"]), want, z, "none", None, dtype), "qkv")
    packed = f64(block.qkv).reshape(B, N, 3, H, d)
    for i, (t, wn) in enumerate(((q, w["wq"]), (k, w["wk"]))):
        xin = packed[:, :, i].transpose(0, 2, 1, 3)
        want = lo.norm_rotate(xin, f64(wn), block.eps, rope)
        close(t, want, norm_bound(xin, f64(wn), want, dtype, rope), "qk"[i])
    assert torch.equal(v, block.qkv.view(B, N, 3, H, d)[:, :, 2].transpose(1, 2))
    o = layer.dense(q, k, v)
    for b in range(B):
        for h in range(H):
            ref, _ = orc.dense_attention(f64(q[b, h]), f64(k[b, h]), f64(v[b, h]))
            parity.assert_close(f64(o[b, h]), ref, dtype, f"attention {b} {h}")
    y = block.output(o, x, gate, torch.empty_like(x))
    want, z = lo.linear(f64(o), f64(w["w_out"]), f64(w["b_out"]), f64(gate), f64(x))
    close(y, want, linear_bound(f64(o), f64(w["w_out"]), want, z, "none", f64(gate), dtype), "y")
    mcs.mcs_check_status()


@pytest.mark.parametrize("case", CASES, ids=[c[0] + f"-d{c[3]}" for c in CASES])
def test_schedule_over_a_block(case):
    """Dense warm-up, an anchor, and reuse steps, the hidden states updated in place; while
    they stand still (second half), reuse steps return the anchor's output up to the cached
    residual's and the output's roundings (2e-2 / 1e-5, the attention's own tolerance)."""
    dtype = case[0]
    layer, block, w, _, x, gate = make(case)
    outs = []

    def step(t, kind, o):
        res = x.clone()
        y = block.output(o, x, gate, x if t < 2 else torch.empty_like(x))
        want, z = lo.linear(f64(o), f64(w["w_out"]), f64(w["b_out"]), f64(gate), f64(res))
        close(y, want, linear_bound(f64(o), f64(w["w_out"]), want, z, "none", f64(gate), dtype), f"step {t}")
        outs.append((kind, o.clone()))

    recs = schedule.run(layer, schedule.Schedule(steps=5, warmup=2, period=4), lambda: block.inputs(x), lambda: None, step)
    mcs.mcs_check_status()
    assert [r.kind for r in recs] == ["dense", "dense", "anchor", "reuse", "reuse"]
    for kind, o in outs[3:]:
        parity.assert_close(f64(o), f64(outs[2][1]), dtype, "reuse on the anchor's inputs")


def test_block_in_a_captured_graph():
    """A reuse step of a block, captured and replayed with new hidden states."""
    layer, block, w, _, x, gate = make(CASES[1])
    layer.anchor(*block.inputs(x))
    y = torch.empty_like(x)

    def reuse():
        block.output(layer.reuse(*block.inputs(x)), x, gate, y)

    reuse()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        reuse()
    x.copy_(rand(gen(31), *x.shape, dtype="bf16"))
    reuse()
    want = y.clone()
    y.zero_()
    graph.replay()
    assert torch.equal(y, want)
    mcs.mcs_check_status()
