"""The operators around the attention layer as measured cases: rotary positions on a
(time, height, width) grid, per-head query/key norms fused with the rotation (forward and
backward), and the matrix product with bias, activation, gate and residual.

`own` false computes them in elementary torch operations, in 32 bits (positions in 64);
`own` true makes the library's calls.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# the largest listed cases, which bound the drawn ones
MAX_ELEMS = 40 * 75600 * 128
MAX_FLOPS = 2 * 75600 * 5120 * 5120


# ---------------------------------------------------------------- cases
def _rope(name, dtype, B, H, d, T, Y, X, extra=0, layout="heads", style="interleaved", inverse=False, listed_pos=False,
          start=0):
    return {"name": name, "op": "rope", "dtype": dtype, "B": B, "H": H, "d": d, "T": T, "Y": Y, "X": X, "extra": extra,
            "layout": layout, "style": style, "inverse": inverse, "listed_pos": listed_pos, "start": start}


def _norm(name, op, dtype, B, H, d, T, Y, X, extra=0, style="interleaved"):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "H": H, "d": d, "T": T, "Y": Y, "X": X, "extra": extra,
            "style": style}


def _linear(name, dtype, B, N, din, dout, act="none", bias=True, gated=False, heads=0):
    return {"name": name, "op": "linear", "dtype": dtype, "B": B, "N": N, "in": din, "out": dout, "act": act,
            "bias": bias, "gated": gated, "heads": heads}


def listed():
    return [
        # the smallest layer of the benchmark, one head of 1,024 tokens: call latency
        _rope("rope-tiny-f32", "f32", 1, 1, 64, 4, 16, 16),
        # queries of the 720p layer, already head by head as the attention takes them
        _rope("rope-720p-bf16", "bf16", 1, 40, 128, 21, 45, 80),
        # gradient through the rotation of regrouped tokens (positions listed), token by token in memory, odd grid
        # of a clip that continues a long video
        _rope("rope-inverse-listed-bf16", "bf16", 2, 16, 64, 11, 37, 41, layout="tokens", style="half", inverse=True,
              listed_pos=True, start=100000),
        # one image with text tokens behind it, two samples (guidance), fp32
        _norm("norm-image-text-f32", "norm", "f32", 2, 16, 64, 1, 31, 47, extra=77, style="half"),
        # projections of the 720p layer, packed q, k, v
        _norm("norm-720p-bf16", "norm", "bf16", 1, 40, 128, 21, 45, 80),
        # training shapes: a small odd clip in fp32, the 480p layer in bf16
        _norm("norm-bwd-odd-f32", "norm_bwd", "f32", 2, 3, 64, 7, 9, 11, extra=5),
        _norm("norm-bwd-480p-bf16", "norm_bwd", "bf16", 1, 12, 128, 16, 32, 64),
        # projections of the smallest layer, fp32
        _linear("linear-tiny-f32", "f32", 1, 1024, 64, 192),
        # six modulation vectors of every sample from the time embedding: one row a sample
        _linear("linear-modulation-bf16", "bf16", 2, 1, 5120, 30720),
        # text embedding of two prompts, ragged row count
        _linear("linear-text-gelu-bf16", "bf16", 2, 226, 4096, 5120, act="gelu_tanh"),
        # packed q, k, v projection of the 480p layer
        _linear("linear-qkv-480p-bf16", "bf16", 1, 32768, 1536, 4608),
        # output projection of the 720p layer from the attention's head-by-head output, gated residual
        _linear("linear-out-720p-bf16", "bf16", 1, 75600, 5120, 5120, gated=True, heads=40),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["rope", "norm", "norm_bwd", "linear", "linear"])
    if op == "linear":
        while True:
            B, N = rng.randint(1, 3), _log(rng, 1, 75600)
            d = rng.choice([64, 128])
            heads = rng.choice([0, 0, _log(rng, 1, 40)])
            din = heads * d if heads else 8 * _log(rng, 8, 640)
            dout = rng.choice([8 * _log(rng, 1, 3840), _log(rng, 1, 2049)])
            flops = 2 * B * N * din * dout
            if flops > (MAX_FLOPS if dtype == "bf16" else MAX_FLOPS // 16):
                continue
            if B * N * max(din, dout) > MAX_ELEMS:
                continue
            c = _linear("", dtype, B, N, din, dout, rng.choice(["none", "gelu_tanh", "gelu_erf", "silu"]),
                        rng.random() < 0.8, rng.random() < 0.5, heads)
            break
    else:
        while True:
            B, H, d = rng.randint(1, 3), _log(rng, 1, 40), rng.choice([64, 128])
            T, Y, X = _log(rng, 1, 33), rng.randint(1, 64), rng.randint(1, 80)
            extra = rng.choice([0, 0, rng.randint(1, 512)])
            es = 1 if dtype == "bf16" else 2
            if es * B * H * (T * Y * X + extra) * d <= MAX_ELEMS:
                break
        style = rng.choice(["interleaved", "half"])
        if op == "rope":
            listed_pos = rng.random() < 0.4
            c = _rope("", dtype, B, H, d, T, Y, X, 0 if listed_pos else extra, rng.choice(["heads", "tokens"]), style,
                      rng.random() < 0.4, listed_pos, rng.choice([0, 0, rng.randint(1, 1000000)]))
        else:
            c = _norm("", op, dtype, B, H, d, T, Y, X, extra, style)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _dims(d):
    """Elements of the head that turn with time, height and width."""
    s = 2 * (d // 6)
    return d - 2 * s, s, s


def _tokens(case):
    return case["T"] * case["Y"] * case["X"] + case["extra"]


def _positions(case, g):
    """Listed positions [B, N, 3] int32: the grid's tokens in another order in every sample."""
    T, Y, X = case["T"], case["Y"], case["X"]
    n = T * Y * X
    rows = []
    for _ in range(case["B"]):
        t = torch.randperm(n, generator=g, device="cuda")
        rows.append(torch.stack([t // (Y * X), (t // X) % Y, t % X], dim=1))
    return torch.stack(rows).to(torch.int32)


def _angles(case, pos, dev="cuda"):
    """Angles in 64 bits, [N, d/2] for the grid or [B, N, d/2] for listed positions; tokens past the grid do not turn."""
    T, Y, X = case["T"], case["Y"], case["X"]
    start = case.get("start", 0)
    if pos is None:
        n = torch.arange(T * Y * X, device=dev)
        p = torch.stack([n // (Y * X), (n // X) % Y, n % X], dim=1)
    else:
        p = pos
    out = []
    for a, da in enumerate(_dims(case["d"])):
        j = torch.arange(da // 2, device=dev, dtype=torch.float64)
        f = THETA ** (-2.0 * j / da)
        pa = p[..., a].to(torch.float64) + (start if a == 0 else 0)
        out.append(pa[..., None] * f)
    ang = torch.cat(out, dim=-1)
    if case["extra"]:
        pad = torch.zeros(case["extra"], ang.shape[-1], device=dev, dtype=torch.float64)
        ang = torch.cat([ang, pad], dim=0)
    return ang


def _packed(case, g, n):
    """Packed projections [B, N, 3, H, d] as a projection writes them: channels of different size."""
    B, H, d = case["B"], case["H"], case["d"]
    x = _randn(g, B, n, 3, H, d)
    x *= torch.exp(0.4 * _randn(g, 3, H, d))
    return x.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "linear":
        B, N, din, dout, heads = case["B"], case["N"], case["in"], case["out"], case["heads"]
        if heads:
            s["x"] = (0.5 * _randn(g, B, heads, N, din // heads)).to(dt)
        else:
            x = _randn(g, B, N, din)
            x *= torch.exp(0.3 * _randn(g, din))
            s["x"] = x.to(dt)
            del x
        s["w"] = (_randn(g, dout, din) / math.sqrt(din)).to(dt)
        s["bias"] = (0.1 * _randn(g, dout)).to(dt) if case["bias"] else None
        s["gate"] = (0.5 * _randn(g, B, dout)).to(dt) if case["gated"] else None
        s["residual"] = (2.0 * _randn(g, B, N, dout)).to(dt) if case["gated"] else None
        if own:
            from sparse_attention_diffusion_gb300 import mcs
            s["desc"] = mcs.linear_desc(B, N, din, dout, dt, act=case["act"], heads=heads)
        return s
    B, H, d, n = case["B"], case["H"], case["d"], _tokens(case)
    s["pos"] = _positions(case, g) if case.get("listed_pos") else None
    if case["op"] == "rope":
        if case["layout"] == "heads":
            s["x"] = _randn(g, B, H, n, d).to(dt)
        else:
            s["x"] = _randn(g, B, n, H, d).to(dt).transpose(1, 2)
    else:
        s["qkv"] = _packed(case, g, n)
        s["wq"] = (1.0 + 0.2 * _randn(g, d)).to(dt)
        s["wk"] = (1.0 + 0.2 * _randn(g, d)).to(dt)
        if case["op"] == "norm_bwd":
            s["dout"] = [_randn(g, B, H, n, d).to(dt) for _ in range(3)]
    if own:
        from sparse_attention_diffusion_gb300 import mcs
        s["desc"] = mcs.make_desc(B, H, n, d, 64, dt)
        s["rope"] = mcs.rope_desc(_dims(d), (case["T"], case["Y"], case["X"]), theta=THETA,
                                  start=(case.get("start", 0), 0, 0), style=case["style"])
        s["table"] = mcs.rope_table(s["rope"])
        if case["op"] == "norm_bwd":
            s["ws"] = mcs.qk_norm_rope_bwd_workspace(s["desc"])
    else:
        ang = _angles(case, s["pos"])
        if s["pos"] is not None:
            ang = ang[:, None]
        s["cos"], s["sin"] = torch.cos(ang).float(), torch.sin(ang).float()
    return s


# ---------------------------------------------------------------- plain form
def _turn(x, cos, sin, style):
    """Rotate the pairs of the last axis: neighbours ("interleaved") or halves ("half")."""
    if style == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)


def _act(z, act):
    if act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
        return z / (1.0 + torch.exp(-2.0 * u))
    if act == "gelu_erf":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "linear":
        x = s["x"].float()
        if case["heads"]:
            x = x.transpose(1, 2).flatten(2)
        z = x @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        z = _act(z, case["act"])
        if s["gate"] is not None:
            z = s["residual"].float() + s["gate"].float()[:, None, :] * z
        return z.to(dt)
    cos, sin, style = s["cos"], s["sin"], case["style"]
    if case["op"] == "rope":
        return _turn(s["x"].float(), cos, -sin if case["inverse"] else sin, style).to(dt)
    q, k, v = (s["qkv"][:, :, i].transpose(1, 2) for i in range(3))
    if case["op"] == "norm":
        out = []
        for x, w in ((q, s["wq"]), (k, s["wk"])):
            x = x.float()
            r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
            out.append(_turn(x * r * w.float(), cos, sin, style).to(dt))
        return [out[0], out[1], v.contiguous()]
    dqkv = torch.empty_like(s["qkv"])
    dws = []
    for i, (x, w) in enumerate(((q, s["wq"]), (k, s["wk"]))):
        x = x.float()
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        gr = _turn(s["dout"][i].float(), cos, -sin, style)
        dws.append((gr * xh).sum((0, 1, 2)))
        gw = gr * w.float()
        dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
        dqkv[:, :, i] = dx.to(dt).transpose(1, 2)
    dqkv[:, :, 2] = s["dout"][2].transpose(1, 2)
    return [dqkv, dws[0], dws[1]]


def _own(s):
    from sparse_attention_diffusion_gb300 import mcs

    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "linear":
        y = torch.empty((case["B"], case["N"], case["out"]), dtype=dt, device="cuda")
        mcs.mcs_linear(s["desc"], s["x"], s["w"], s["bias"], s["gate"], s["residual"], y)
        return y
    if case["op"] == "rope":
        y = torch.empty_like(s["x"])
        mcs.mcs_rope_apply(s["desc"], s["rope"], s["table"], s["pos"], s["x"], y, inverse=case["inverse"])
        return y
    q, k, v = (s["qkv"][:, :, i].transpose(1, 2) for i in range(3))
    shape = (case["B"], case["H"], _tokens(case), case["d"])
    if case["op"] == "norm":
        out = [torch.empty(shape, dtype=dt, device="cuda") for _ in range(3)]
        mcs.mcs_qk_norm_rope(s["desc"], s["rope"], s["table"], s["pos"], q, k, v, s["wq"], s["wk"], EPS, *out)
        return out
    dqkv = torch.empty_like(s["qkv"])
    dq, dk, dv = (dqkv[:, :, i].transpose(1, 2) for i in range(3))
    dwq = torch.empty(case["d"], dtype=torch.float32, device="cuda")
    dwk = torch.empty_like(dwq)
    mcs.mcs_qk_norm_rope_bwd(s["desc"], s["rope"], s["table"], s["pos"], q, k, s["wq"], s["wk"], EPS, *s["dout"],
                             dq, dk, dv, dwq, dwk, s["ws"])
    return [dqkv, dwq, dwk]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64-bit values
def _exact_linear(case, s):
    B, N, din, heads = case["B"], case["N"], case["in"], case["heads"]
    w = s["w"].double()
    y = torch.empty((B, N, case["out"]), dtype=torch.float64, device="cuda")
    step = 8192
    for b in range(B):
        for n0 in range(0, N, step):
            if heads:
                x = s["x"][b, :, n0:n0 + step].double().permute(1, 0, 2).reshape(-1, din)
            else:
                x = s["x"][b, n0:n0 + step].double()
            z = torch.einsum("nk,mk->nm", x, w)
            if case["bias"]:
                z += s["bias"].double()
            if case["act"] == "silu":
                z = z * torch.sigmoid(z)
            elif case["act"] == "gelu_erf":
                z = z * torch.special.ndtr(z)
            elif case["act"] == "gelu_tanh":
                z = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
            if case["gated"]:
                z = s["residual"][b, n0:n0 + step].double() + s["gate"][b].double() * z
            y[b, n0:n0 + step] = z
    return y


def _complex_pairs(x, style):
    if style == "interleaved":
        return torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous())
    h = x.shape[-1] // 2
    return torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous())


def _from_pairs(z, style):
    if style == "interleaved":
        return torch.view_as_real(z).flatten(-2)
    return torch.cat([z.real, z.imag], dim=-1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "linear":
        return _exact_linear(case, s)
    s.pop("cos"), s.pop("sin")
    style, d = case["style"], case["d"]
    ang = _angles(case, s["pos"])
    unit = torch.polar(torch.ones_like(ang), ang)        # [N, d/2] or [B, N, d/2]

    def phases(b):
        return unit if s["pos"] is None else unit[b]

    def heads_of(make, like):
        out = torch.empty(like, dtype=torch.float64, device="cuda")
        for b in range(like[0]):
            for h in range(like[1]):
                out[b, h] = make(b, h)
        return out

    shape = (case["B"], case["H"], _tokens(case), d)
    if case["op"] == "rope":
        def one(b, h):
            u = phases(b)
            return _from_pairs(_complex_pairs(s["x"][b, h].double(), style) * (u.conj() if case["inverse"] else u), style)
        return heads_of(one, shape)
    qkv = s["qkv"]
    if case["op"] == "norm":
        def normed(i, w):
            def one(b, h):
                x = qkv[b, :, i, h].double()
                x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w.double()
                return _from_pairs(_complex_pairs(x, style) * phases(b), style)
            return heads_of(one, shape)
        return [normed(0, s["wq"]), normed(1, s["wk"]), qkv[:, :, 2].transpose(1, 2).double()]
    grad = torch.empty(qkv.shape, dtype=torch.float64, device="cuda")
    dws = []
    for i, w in enumerate((s["wq"], s["wk"])):
        dw = torch.zeros(d, dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            for h in range(case["H"]):
                x = qkv[b, :, i, h].double()
                g = _from_pairs(_complex_pairs(s["dout"][i][b, h].double(), style) * phases(b).conj(), style)
                ms = x.square().sum(-1, keepdim=True) / d + EPS
                dw += (g * x / ms.sqrt()).sum(0)
                gw = g * w.double()
                grad[b, :, i, h] = gw / ms.sqrt() - x * (gw * x).sum(-1, keepdim=True) / (d * ms * ms.sqrt())
        dws.append(dw)
    grad[:, :, 2] = s["dout"][2].transpose(1, 2)
    return [grad, dws[0], dws[1]]


# ---------------------------------------------------------------- work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        M, din, dout = case["B"] * case["N"], case["in"], case["out"]
        n = M * din + dout * din + M * dout + (dout if case["bias"] else 0)
        if case["gated"]:
            n += M * dout + case["B"] * dout
        return {"bytes": n * es, "flops": 2 * M * din * dout}
    n = case["B"] * case["H"] * _tokens(case) * case["d"]
    pos = 12 * case["B"] * _tokens(case) if case.get("listed_pos") else 0
    if case["op"] == "rope":
        return {"bytes": 2 * n * es + pos, "flops": 3 * n}
    if case["op"] == "norm":
        return {"bytes": 6 * n * es, "flops": 14 * n}
    return {"bytes": 8 * n * es, "flops": 28 * n}
