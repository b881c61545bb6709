"""Meta-cache denoising schedule over the C ABI [MC-Sparse summary: grouping and
exact selection run only on anchor steps; later steps reuse the query groups, the
KV indices and the output residual; groups, indices and residual refresh together].

A schedule of `steps` denoising steps for one attention layer:
  * the first `warmup` steps run dense attention;
  * step `warmup + i*period` is an anchor: PDDP grouping, dense attention + LSE,
    pass-2 column sums + exact top-K, anchor sparse attention + residual store;
    the anchor's output is the dense output;
  * every other step is a reuse step: sparse attention of the current Q/K/V over
    the cached groups and indices, plus the cached residual.
The warm-up length and anchor period are not on the pages; the 118,800-token
schedule workload uses 5 warm-up steps and an anchor every 10 steps.

Inputs drift between steps through a caller-supplied callback (the generator's
variance-preserving drift), which runs outside the per-step kernel timing.
"""
from __future__ import annotations

from dataclasses import dataclass, field

import torch

from . import mcs


@dataclass
class StepRecord:
    kind: str          # "dense" | "anchor" | "reuse"
    ms: float
    stages: dict = field(default_factory=dict)


@dataclass
class Schedule:
    steps: int = 50
    warmup: int = 5
    period: int = 10

    def kind(self, t: int) -> str:
        if t < self.warmup:
            return "dense"
        return "anchor" if (t - self.warmup) % self.period == 0 else "reuse"


class MetaCacheLayer:
    """One attention layer with its caller-owned meta-cache buffers.

    warm_iters: None groups every anchor from the fixed start (desc.pddp_iters
    power iterations); an integer keeps the grouping's per-node directions
    between anchors, so that every anchor after the first starts each node from
    the previous anchor's direction and runs warm_iters iterations ("fast PDDP",
    the amortised grouping). `masses` collects each anchor's mean captured
    attention mass (untimed), the quality measure of the grouping."""

    def __init__(self, desc: mcs.mcs_desc, K: int, dtype, device, warm_iters=None):
        self.desc, self.K = desc, K
        self.cache = mcs.alloc_cache(desc, K, dtype, device=device)
        self.ws = mcs.workspace(desc, K, device=device)
        shape = (desc.B, desc.H, desc.N, desc.d)
        self.o_dense = torch.empty(shape, dtype=dtype, device=device)
        self.lse = torch.empty((desc.B, desc.H, desc.N), dtype=torch.float32, device=device)
        self.out = torch.empty(shape, dtype=dtype, device=device)
        self.warm_iters = warm_iters
        self.masses = []
        self._anchors = 0
        if warm_iters is not None:
            self.dirs = mcs.pddp_dirs(desc, device=device)
            self.desc_warm = mcs.make_desc(desc.B, desc.H, desc.N, desc.d, desc.C, dtype, desc.scale, warm_iters)

    def group(self, q):
        c = self.cache
        if self.warm_iters is None:
            mcs.mcs_group_pddp(self.desc, q, c["perm"], c["group_of"], self.ws)
        elif self._anchors == 0:
            mcs.mcs_group_pddp_warm(self.desc, q, None, self.dirs, c["perm"], c["group_of"], self.ws)
        else:
            mcs.mcs_group_pddp_warm(self.desc_warm, q, self.dirs, self.dirs, c["perm"], c["group_of"], self.ws)
        self._anchors += 1

    def dense(self, q, k, v):
        mcs.mcs_dense_attn(self.desc, q, k, v, self.o_dense, self.lse)
        return self.o_dense

    def anchor(self, q, k, v, timer=None):
        c = self.cache
        t = timer or (lambda name, fn: fn())
        t("pddp", lambda: self.group(q))
        t("dense", lambda: mcs.mcs_dense_attn(self.desc, q, k, v, self.o_dense, self.lse))
        t("select", lambda: mcs.mcs_anchor_select(self.desc, q, k, c["perm"], self.lse, self.K, c["idx"], c["mass"],
                                                  self.ws))
        t("anchor_residual", lambda: mcs.mcs_anchor_residual(self.desc, q, k, v, c["perm"], c["idx"], self.K,
                                                             self.o_dense, c["residual"]))
        return self.o_dense

    def after_step(self, kind, q):
        """Untimed work after a step: the anchor's mean captured mass."""
        if kind == "anchor":
            self.masses.append(float(self.cache["mass"].float().mean()))

    def reuse(self, q, k, v):
        c = self.cache
        mcs.mcs_sparse_attn_gather(self.desc, q, k, v, c["perm"], c["idx"], self.K, c["residual"], self.out)
        return self.out


@dataclass
class BlockAdapters:
    """Low-rank adapters of an AttentionBlock's two projections for the requests of a batch: adapter a adds
    scale[a] * (x down_a^T) up_a^T to a projection of the rows whose segment takes it. start [segments + 1] cuts the rows
    (counted through the batches), which [segments] names each segment's adapter (negative: none); both int32."""
    down_qkv: torch.Tensor   # [count, rank, in]
    up_qkv: torch.Tensor     # [count, 3 * H * d, rank]
    down_out: torch.Tensor   # [count, rank, H * d]
    up_out: torch.Tensor     # [count, in, rank]
    scale: torch.Tensor      # [count] fp32
    start: torch.Tensor
    which: torch.Tensor


class AttentionBlock:
    """The projections around a MetaCacheLayer, from a block's hidden states x
    [B, N, in] and back: packed q, k, v projection, per-head norms of q and k with
    the rotary positions, attention (the layer's dense, anchor or reuse step), output
    projection added to the hidden states through a gate.

    w_qkv: [3 * H * d, in], rows ordered q heads, k heads, v heads; w_out: [in, H * d];
    wq, wk: norm weights [d] or None; biases may be None. adapters: BlockAdapters of the
    requests in the batch, or None; its tensors may be refilled between steps. The block owns
    its buffers; q, k, v are overwritten by every inputs() call. With run():
        run(layer, sched, lambda: block.inputs(x), advance,
            on_output=lambda t, kind, o: block.output(o, x, gate, x))"""

    def __init__(self, layer: MetaCacheLayer, rope, w_qkv, b_qkv, wq, wk, w_out, b_out, eps=1e-6, adapters=None):
        d = layer.desc
        hd, dt, dev = d.H * d.d, layer.out.dtype, layer.out.device
        self.layer, self.rope, self.eps = layer, rope, eps
        self.w_qkv, self.b_qkv, self.wq, self.wk, self.w_out, self.b_out = w_qkv, b_qkv, wq, wk, w_out, b_out
        self.table = mcs.rope_table(rope, device=dev)
        self.proj_in = mcs.linear_desc(d.B, d.N, w_qkv.shape[1], 3 * hd, dt)
        self.proj_out = mcs.linear_desc(d.B, d.N, hd, w_out.shape[0], dt, heads=d.H)
        self.qkv = torch.empty((d.B, d.N, 3 * hd), dtype=dt, device=dev)
        self.q, self.k, self.v = (torch.empty_like(layer.out) for _ in range(3))
        self.adapters = adapters
        if adapters is not None:
            a = adapters
            self.sets = mcs.adapters_desc(a.down_qkv.shape[0], a.down_qkv.shape[1], a.which.shape[0])
            sizes = [mcs.linear_adapters_workspace(p, self.sets, device=dev) for p in (self.proj_in, self.proj_out)]
            self.ws = max(sizes, key=torch.Tensor.numel)

    def _project(self, desc, x, w, bias, gate, residual, y, down, up):
        a = self.adapters
        if a is None:
            mcs.mcs_linear(desc, x, w, bias, gate, residual, y)
        else:
            mcs.mcs_linear_adapters(desc, self.sets, x, w, bias, gate, residual, getattr(a, down), getattr(a, up), a.scale,
                                    a.start, a.which, y, self.ws)

    def inputs(self, x):
        """(q, k, v) [B, H, N, d] of the hidden states x."""
        d = self.layer.desc
        self._project(self.proj_in, x, self.w_qkv, self.b_qkv, None, None, self.qkv, "down_qkv", "up_qkv")
        q, k, v = self.qkv.view(d.B, d.N, 3, d.H, d.d).permute(2, 0, 3, 1, 4)
        mcs.mcs_qk_norm_rope(d, self.rope, self.table, None, q, k, v, self.wq, self.wk, self.eps, self.q, self.k, self.v)
        return self.q, self.k, self.v

    def output(self, o, x, gate, y):
        """y = x + gate * (o w_out^T + b_out) for an attention output o; y may be x."""
        self._project(self.proj_out, o, self.w_out, self.b_out, gate, x, y, "down_out", "up_out")
        return y


def run(layer: MetaCacheLayer, sched: Schedule, inputs, advance, on_output=None):
    """Run the schedule. `inputs()` returns the current (q, k, v); `advance()`
    drifts them to the next step. Returns the per-step records (CUDA-event ms)."""
    stream = torch.cuda.current_stream()
    recs = []
    for t in range(sched.steps):
        q, k, v = inputs()
        kind = sched.kind(t)
        stages = {}
        ev = []

        def timer(name, fn):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record(stream)
            fn()
            b.record(stream)
            ev.append((name, a, b))

        a0, b0 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a0.record(stream)
        if kind == "dense":
            out = layer.dense(q, k, v)
        elif kind == "anchor":
            out = layer.anchor(q, k, v, timer)
        else:
            out = layer.reuse(q, k, v)
        b0.record(stream)
        if hasattr(layer, "after_step"):
            layer.after_step(kind, q)
        if on_output is not None:
            on_output(t, kind, out)
        recs.append((kind, a0, b0, ev))
        advance()
    torch.cuda.synchronize()
    out = []
    for kind, a0, b0, ev in recs:
        out.append(StepRecord(kind, a0.elapsed_time(b0), {n: a.elapsed_time(b) for n, a, b in ev}))
    return out


def anchor_overhead(records, t_dense_ms: float, density: float, warmup: int):
    """Anchor cost spread over the trajectory, as extra density points: the
    post-warm-up time divided by what dense attention would have cost on those
    steps gives an equivalent density; the overhead is that minus the density."""
    post = [r for r in records[warmup:]]
    t_post = sum(r.ms for r in post)
    rho_eq = t_post / (len(post) * t_dense_ms)
    return rho_eq, rho_eq - density
