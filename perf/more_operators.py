"""Requests of different lengths in one batch as measured cases: attention over packed sequences (causal or not,
grouped heads, whole prompts, chunks and single tokens over kept keys), and the projection with each request's own
low-rank adapter.

`own` false computes them in elementary torch operations, in 32 bits; `own` true makes the library's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# the largest listed cases, which bound the drawn ones
MAX_PAIRS = 12 * 32768 * 32769 // 2 * 128        # visible (query, key) pairs x heads x d
MAX_CACHE = 64 * 16384 * 8 * 128                 # elements of keys
MAX_FLOPS = 2 * 75600 * 5120 * 5120
MAX_ELEMS = 75600 * 5120


# ---------------------------------------------------------------- cases
def _attn(name, dtype, S, H, Hk, d, longest_q, longest_k=0, causal=True, layout="packed", mix=0):
    """longest_k 0: a sequence's keys are its own tokens. mix 0: all sequences have the longest length, otherwise they
    are ragged and mix seeds them."""
    return {"name": name, "op": "attn", "dtype": dtype, "S": S, "H": H, "Hk": Hk, "d": d, "longest_q": longest_q,
            "longest_k": longest_k, "causal": causal, "layout": layout, "mix": mix}


def _lora(name, dtype, B, N, din, dout, S, count, rank, act="none", bias=True, gated=False, heads=0, mix=0):
    return {"name": name, "op": "lora", "dtype": dtype, "B": B, "N": N, "in": din, "out": dout, "S": S, "count": count,
            "rank": rank, "act": act, "bias": bias, "gated": gated, "heads": heads, "mix": mix}


def listed():
    return [
        # one short prompt of a small encoder in fp32: call latency
        _attn("attn-prompt-tiny-f32", "f32", 1, 4, 2, 64, 77),
        # one new token of one prompt over its kept keys: the smallest bf16 call
        _attn("attn-token-one", "bf16", 1, 32, 8, 128, 1, 4000),
        # 16 ragged prompts of a text encoder with grouped heads, straight from the packed projection
        _attn("attn-prompts-ragged", "bf16", 16, 32, 8, 128, 900, mix=3),
        # chunks of prompts that continue over kept keys, six heads a key head, d = 64
        _attn("attn-chunks-d64", "bf16", 7, 24, 4, 64, 300, 9000, layout="heads", mix=5),
        # one token for each of 64 requests over ragged caches
        _attn("attn-tokens-64", "bf16", 64, 32, 8, 128, 1, 16384, layout="heads", mix=7),
        # three clips of different length, every token sees its whole clip (no mask), heads of the 480p layer
        _attn("attn-clips-full", "bf16", 3, 12, 12, 128, 20000, causal=False, layout="heads", mix=2),
        # one long prompt of as many tokens as the 480p layer
        _attn("attn-prompt-long", "bf16", 1, 12, 4, 128, 32768),
        # the smallest layer's packed projection in fp32, two requests
        _lora("lora-tiny-f32", "f32", 1, 1024, 64, 192, 2, 2, 4, mix=1),
        # one token of each of 64 requests, each with its own adapter or none
        _lora("lora-tokens-64", "bf16", 1, 64, 4096, 4096, 64, 48, 16, bias=False, mix=4),
        # text embedding of two prompts with two adapters
        _lora("lora-text-gelu", "bf16", 2, 226, 4096, 5120, 2, 3, 32, act="gelu_tanh", mix=2),
        # packed q, k, v projection of the 480p layer, four clips of different length
        _lora("lora-qkv-480p", "bf16", 1, 32768, 1536, 4608, 4, 3, 64, mix=6),
        # output projection of the 720p layer from the attention's output, gated residual, one adapter for all
        _lora("lora-out-720p", "bf16", 1, 75600, 5120, 5120, 1, 1, 32, gated=True, heads=40),
    ]


def _lengths(n, longest, mix, short=1):
    """Lengths of n sequences, the longest first if all are alike."""
    if not mix:
        return [longest] * n
    r = random.Random(mix * 7919 + n)
    return [max(short, min(longest, int(longest * r.random() ** 1.5) + r.randint(0, 3))) for _ in range(n)]


def _attn_lengths(case):
    q = _lengths(case["S"], case["longest_q"], case["mix"])
    if case["longest_k"] == 0:
        return q, q
    # kept keys before the new tokens, which are the last of them
    k = _lengths(case["S"], case["longest_k"], case["mix"] and case["mix"] + 1)
    return q, [a + b for a, b in zip(k, q)]


def _segments(case):
    """Segment bounds over the rows, and the adapter of each segment (-1: none)."""
    S, rows = case["S"], case["B"] * case["N"]
    r = random.Random(case["mix"] * 104729 + S)
    if S == rows:
        start = list(range(rows + 1))
    elif case["mix"] == 0:
        start = [rows * s // S for s in range(S + 1)]
    else:
        start = [0] + sorted(r.randint(0, rows) for _ in range(S - 1)) + [rows]
    which = [0] if S == 1 else [r.randint(-1, case["count"] - 1) if s else 0 for s in range(S)]
    return start, which


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _pairs(nq, nk, causal):
    if not causal:
        return nq * nk
    n = min(nq, nk)  # the last n queries see nk - n + 1 .. nk keys
    return n * (nk - n) + n * (n + 1) // 2


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    mix = rng.randint(1, 1000000)
    if rng.random() < 0.5:
        while True:
            d, Hk, g = rng.choice([64, 128]), _log(rng, 1, 16), rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 8, 16])
            S = _log(rng, 1, 96)
            kind = rng.choice(["prompts", "chunks", "tokens"])
            lq = 1 if kind == "tokens" else _log(rng, 1, 20000 if kind == "prompts" else 600)
            lk = 0 if kind == "prompts" else _log(rng, 1, 20000)
            c = _attn("", dtype, S, Hk * g, Hk, d, lq, lk, rng.random() < 0.7, rng.choice(["packed", "heads"]),
                      rng.choice([0, mix, mix, mix]))
            q, k = _attn_lengths(c)
            pairs = sum(_pairs(a, b, c["causal"]) for a, b in zip(q, k)) * Hk * g * d
            heavy = 1 if dtype == "bf16" else 20
            if pairs * heavy > MAX_PAIRS or sum(k) * Hk * d * (1 if dtype == "bf16" else 4) > MAX_CACHE:
                continue
            if sum(q) * Hk * g * d <= MAX_ELEMS:
                break
    else:
        while True:
            B, N = rng.randint(1, 3), _log(rng, 1, 75600)
            d = rng.choice([64, 128])
            heads = rng.choice([0, 0, _log(rng, 1, 40)])
            din = heads * d if heads else 8 * _log(rng, 8, 640)
            dout = rng.choice([8 * _log(rng, 1, 1280), _log(rng, 1, 2049)])
            S = min(B * N, rng.choice([1, B, _log(rng, 1, 96)]))
            c = _lora("", dtype, B, N, din, dout, S, _log(rng, 1, 64), 8 * _log(rng, 1, 16),
                      rng.choice(["none", "none", "gelu_tanh", "gelu_erf", "silu"]), rng.random() < 0.7,
                      rng.random() < 0.5, heads, mix)
            flops = 2 * B * N * din * dout
            if flops <= (MAX_FLOPS if dtype == "bf16" else MAX_FLOPS // 16) and B * N * max(din, dout) <= MAX_ELEMS:
                break
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _starts(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _prepare_attn(case, g, dt):
    H, Hk, d = case["H"], case["Hk"], case["d"]
    nq, nk = _attn_lengths(case)
    Tq, Tk = sum(nq), sum(nk)
    s = {"case": case, "nq": nq, "nk": nk}
    if case["layout"] == "packed" and case["longest_k"] == 0:
        # the packed projection [tokens, H + 2 Hk, d] as it lies in memory
        qkv = _randn(g, Tq, H + 2 * Hk, d)
        qkv[:, :H] *= 1.5
        qkv = qkv.to(dt).transpose(0, 1)
        s["q"], s["k"], s["v"] = qkv[:H], qkv[H:H + Hk], qkv[H + Hk:]
    elif case["layout"] == "packed":
        s["q"] = (1.5 * _randn(g, Tq, H, d)).to(dt).transpose(0, 1)
        s["k"], s["v"] = (_randn(g, Tk, Hk, d).to(dt).transpose(0, 1) for _ in range(2))
    else:
        s["q"] = (1.5 * _randn(g, H, Tq, d)).to(dt)
        s["k"], s["v"] = (_randn(g, Hk, Tk, d).to(dt) for _ in range(2))
    s["q_start"] = torch.tensor(_starts(nq), dtype=torch.int32, device="cuda")
    s["k_start"] = s["q_start"] if nq == nk else torch.tensor(_starts(nk), dtype=torch.int32, device="cuda")
    if own:
        from sparse_attention_diffusion_gb300 import mcs
        s["desc"] = mcs.packed_desc(case["S"], Tq, Tk, H, Hk, d, dt, causal=case["causal"], max_q=max(nq))
        s["ws"] = mcs.packed_attn_workspace(s["desc"])
    return s


def _prepare_lora(case, g, dt):
    B, N, din, dout, heads = case["B"], case["N"], case["in"], case["out"], case["heads"]
    count, R = case["count"], case["rank"]
    s = {"case": case}
    if heads:
        s["x"] = (0.5 * _randn(g, B, heads, N, din // heads)).to(dt)
    else:
        s["x"] = _randn(g, B, N, din).to(dt)
    s["w"] = (_randn(g, dout, din) / math.sqrt(din)).to(dt)
    s["bias"] = (0.1 * _randn(g, dout)).to(dt) if case["bias"] else None
    s["gate"] = (0.5 * _randn(g, B, dout)).to(dt) if case["gated"] else None
    s["residual"] = (2.0 * _randn(g, B, N, dout)).to(dt) if case["gated"] else None
    s["down"] = (_randn(g, count, R, din) / math.sqrt(din)).to(dt)
    s["up"] = (0.3 * _randn(g, count, dout, R) / math.sqrt(R)).to(dt)
    s["scale"] = 0.5 + torch.rand((count,), generator=g, device="cuda")
    s["bounds"], s["ids"] = _segments(case)
    s["start"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
    s["which"] = torch.tensor(s["ids"], dtype=torch.int32, device="cuda")
    if own:
        from sparse_attention_diffusion_gb300 import mcs
        s["desc"] = mcs.linear_desc(B, N, din, dout, dt, act=case["act"], heads=heads)
        s["adapters"] = mcs.adapters_desc(count, R, case["S"])
        s["ws"] = mcs.linear_adapters_workspace(s["desc"], s["adapters"])
    return s


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    return _prepare_attn(case, g, dt) if case["op"] == "attn" else _prepare_lora(case, g, dt)


# ---------------------------------------------------------------- plain form
def _plain_attn(s):
    case = s["case"]
    H, Hk, d = case["H"], case["Hk"], case["d"]
    g = H // Hk
    dt = DTYPES[case["dtype"]]
    Tq = s["q"].shape[1]
    o = torch.empty((H, Tq, d), dtype=dt, device="cuda")
    lse = torch.empty((H, Tq), dtype=torch.float32, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        step = max(1, (1 << 30) // (g * nk))  # rows at once: their scores stay below 4 GB
        heads = max(1, min(Hk, (1 << 29) // (g * nq * nk)))
        for h in range(0, Hk, heads):
            n = min(heads, Hk - h)
            k = s["k"][h:h + n, None, k0:k0 + nk].float()
            v = s["v"][h:h + n, None, k0:k0 + nk].float()
            for i in range(0, nq, step):
                e = min(nq, i + step)
                q = s["q"][h * g:(h + n) * g, q0 + i:q0 + e].float().reshape(n, g, e - i, d)
                z = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
                if case["causal"] and nq > 1:
                    rows = torch.arange(i, e, device="cuda")[:, None] + (nk - nq)
                    z.masked_fill_(torch.arange(nk, device="cuda")[None, :] > rows, -math.inf)
                m = z.amax(-1, keepdim=True)
                z = torch.exp_(z.sub_(m))
                l = z.sum(-1, keepdim=True)
                o[h * g:(h + n) * g, q0 + i:q0 + e] = ((z @ v) / l).reshape(n * g, e - i, d).to(dt)
                lse[h * g:(h + n) * g, q0 + i:q0 + e] = (m + torch.log(l)).reshape(n * g, e - i)
        q0, k0 = q0 + nq, k0 + nk
    return [o, lse]


def _act(z, act):
    if act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
        return z / (1.0 + torch.exp(-2.0 * u))
    if act == "gelu_erf":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_lora(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    x = s["x"].float()
    if case["heads"]:
        x = x.transpose(1, 2)
    x = x.reshape(-1, case["in"])
    z = x @ s["w"].float().t()
    if s["bias"] is not None:
        z += s["bias"].float()
    for a, lo, hi in zip(s["ids"], s["bounds"][:-1], s["bounds"][1:]):
        if a >= 0 and hi > lo:
            z[lo:hi] += s["scale"][a] * ((x[lo:hi] @ s["down"][a].float().t()) @ s["up"][a].float().t())
    z = _act(z, case["act"]).reshape(case["B"], case["N"], case["out"])
    if s["gate"] is not None:
        z = s["residual"].float() + s["gate"].float()[:, None, :] * z
    return z.to(dt)


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from sparse_attention_diffusion_gb300 import mcs

    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "attn":
        H, Tq, d = s["q"].shape
        o = torch.empty((H, Tq, d), dtype=dt, device="cuda")
        lse = torch.empty((H, Tq), dtype=torch.float32, device="cuda")
        mcs.mcs_packed_attn(s["desc"], s["q"], s["k"], s["v"], s["q_start"], s["k_start"], o, lse, s["ws"])
        return [o, lse]
    y = torch.empty((case["B"], case["N"], case["out"]), dtype=dt, device="cuda")
    mcs.mcs_linear_adapters(s["desc"], s["adapters"], s["x"], s["w"], s["bias"], s["gate"], s["residual"], s["down"],
                            s["up"], s["scale"], s["start"], s["which"], y, s["ws"])
    return y


def run(state):
    if own:
        return _own(state)
    return _plain_attn(state) if state["case"]["op"] == "attn" else _plain_lora(state)


# ---------------------------------------------------------------- 64-bit values
def _exact_attn(case, s):
    """Row by row from the definition: weights by the log-sum-exp of the visible scores."""
    H, g, d = case["H"], case["H"] // case["Hk"], case["d"]
    nq, nk = _attn_lengths(case)
    Tq = sum(nq)
    o = torch.empty((H, Tq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((H, Tq), dtype=torch.float64, device="cuda")
    qs, ks = _starts(nq), _starts(nk)
    for i in range(case["S"]):
        for h in range(H):
            k = s["k"][h // g, ks[i]:ks[i + 1]].double()
            v = s["v"][h // g, ks[i]:ks[i + 1]].double()
            block = max(1, 134217728 // nk[i])
            for r in range(0, nq[i], block):
                e = min(nq[i], r + block)
                last = nk[i] - nq[i] + e if case["causal"] else nk[i]  # keys that any of these rows sees
                z = torch.einsum("qd,kd->qk", s["q"][h, qs[i] + r:qs[i] + e].double(), k[:last]) / d ** 0.5
                if case["causal"]:
                    z += torch.full_like(z, -math.inf).triu(nk[i] - nq[i] + r + 1)
                n = torch.logsumexp(z, -1)
                lse[h, qs[i] + r:qs[i] + e] = n
                o[h, qs[i] + r:qs[i] + e] = torch.einsum("qk,kd->qd", torch.exp(z - n[:, None]), v[:last])
    return [o, lse]


def _exact_lora(case, s):
    B, N, din, dout, heads = case["B"], case["N"], case["in"], case["out"], case["heads"]
    w = s["w"].double()
    y = torch.empty((B * N, dout), dtype=torch.float64, device="cuda")
    bounds, ids = s["bounds"], s["ids"]
    x_all = s["x"].permute(0, 2, 1, 3).reshape(B * N, din) if heads else s["x"].reshape(B * N, din)
    for lo, hi, a in zip(bounds[:-1], bounds[1:], ids):
        eff = w if a < 0 else w + float(s["scale"][a]) * torch.einsum("or,ri->oi", s["up"][a].double(), s["down"][a].double())
        for n in range(lo, hi, 8192):
            m = min(hi, n + 8192)
            z = torch.einsum("nk,mk->nm", x_all[n:m].double(), eff)
            if case["bias"]:
                z += s["bias"].double()
            if case["act"] == "silu":
                z = z * torch.sigmoid(z)
            elif case["act"] == "gelu_erf":
                z = z * torch.special.ndtr(z)
            elif case["act"] == "gelu_tanh":
                z = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
            if case["gated"]:
                batch = torch.arange(n, m, device="cuda") // N
                z = s["residual"].reshape(B * N, dout)[n:m].double() + s["gate"].double()[batch] * z
            y[n:m] = z
    return y.reshape(B, N, dout)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_attn(case, s) if case["op"] == "attn" else _exact_lora(case, s)


# ---------------------------------------------------------------- work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attn":
        H, Hk, d = case["H"], case["Hk"], case["d"]
        nq, nk = _attn_lengths(case)
        pairs = sum(_pairs(a, b, case["causal"]) for a, b in zip(nq, nk))
        return {"bytes": es * d * (2 * H * sum(nq) + 2 * Hk * sum(nk)) + 4 * H * sum(nq), "flops": 4 * H * d * pairs}
    M, din, dout, R = case["B"] * case["N"], case["in"], case["out"], case["rank"]
    bounds, ids = _segments(case)
    used = {a for a, lo, hi in zip(ids, bounds[:-1], bounds[1:]) if a >= 0 and hi > lo}
    rows = sum(hi - lo for a, lo, hi in zip(ids, bounds[:-1], bounds[1:]) if a >= 0)
    n = M * din + dout * din + M * dout + (dout if case["bias"] else 0) + len(used) * R * (din + dout)
    if case["gated"]:
        n += M * dout + case["B"] * dout
    return {"bytes": n * es, "flops": 2 * M * din * dout + 2 * rows * R * (din + dout)}
