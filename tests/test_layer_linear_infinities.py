"""Infinite elements in the matrix product: their outputs are what the products and their sum
are, whatever the number of rows, and no other output changes."""
import numpy as np
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import f64, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 8, 9, 200, 4200])
def test_infinities_as_in_a_plain_sum(M, dtype):
    """Infinite elements give what their products and sums are: infinities where their signs agree, NaN for opposite
    ones and beside a zero; everything else keeps its bits."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    g = gen(92)
    K, O, inf = 96, 72, float("inf")
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, w = torch.randn(1, M, K, generator=g).to(dt), torch.randn(O, K, generator=g).to(dt)
    w[11, 5] = 0.0

    def run(a, b):
        y = torch.empty(1, M, O, dtype=dt, device="cuda")
        mcs.mcs_linear(mcs.linear_desc(1, M, K, O, dt), a.cuda(), b.cuda(), None, None, None, y)
        mcs.mcs_check_status()
        return f64(y)[0]

    clean = run(x, w)
    x[0, M // 2, 5] = inf                    # one infinity: its sign times w's, NaN at the zero
    if M > 8:
        x[0, M - 1, 5], x[0, M - 1, 90] = -inf, inf
    w[40, 7] = -inf
    y = run(x, w)
    with np.errstate(invalid="ignore"):
        want = (f64(x)[0, :, None, :] * f64(w)[None]).sum(-1) if M <= 200 else None
    rows = sorted({M // 2, M - 1, 0}) if M > 8 else [M // 2]
    for m in range(M) if M <= 200 else rows:
        with np.errstate(invalid="ignore"):
            r = want[m] if want is not None else (f64(x)[0, m] * f64(w)).sum(-1)
        hard = ~np.isfinite(r)
        assert np.array_equal(np.isnan(y[m]), np.isnan(r)), m
        assert np.array_equal(y[m][hard & ~np.isnan(r)], r[hard & ~np.isnan(r)]), m
        assert np.array_equal(y[m][~hard], clean[m][~hard]), m


@pytest.mark.parametrize("heads,d,O", [(3, 64, 70), (2, 128, 260), (0, 1540, 33)])
def test_infinities_through_the_whole_epilogue(heads, d, O):
    """From heads, over batches, K slices and an in-place gated residual; the finite numbers beside them within fp32."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    g = gen(93)
    B, N, K, inf = 2, 150, max(heads, 1) * d, float("inf")
    x = torch.randn(B, heads, N, d, generator=g) if heads else torch.randn(B, N, d, generator=g)
    w, bias, gate = torch.randn(O, K, generator=g), torch.randn(O, generator=g), torch.randn(B, O, generator=g)
    res = torch.randn(B, N, O, generator=g)
    if heads:
        x[1, heads - 1, 149, d - 1], x[0, 0, 3, 0] = inf, -inf
    else:
        x[1, 149, d - 1], x[0, 3, 0] = inf, -inf
    w[O - 1, 1] = inf
    y = res.cuda()
    desc = mcs.linear_desc(B, N, K, O, torch.float32, heads=heads)
    mcs.mcs_linear(desc, x.cuda(), w.cuda(), bias.cuda(), gate.cuda(), y, y)
    mcs.mcs_check_status()
    got = f64(y)
    xt = f64(x).transpose(0, 2, 1, 3).reshape(B, N, K) if heads else f64(x)
    with np.errstate(invalid="ignore"):
        z = np.stack([(xt[b, n] * f64(w)).sum(-1) for b in range(B) for n in range(N)]).reshape(B, N, O) + f64(bias)
        want = f64(res) + f64(gate)[:, None] * z
    hard = ~np.isfinite(want)
    assert hard.sum() == 2 * O + B * N - 2
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[hard & ~np.isnan(want)], want[hard & ~np.isnan(want)])
    size = np.abs(f64(gate))[:, None] * (np.nan_to_num(np.abs(xt), posinf=0) @ np.nan_to_num(np.abs(f64(w)), posinf=0).T + 8)
    assert np.all(np.abs(got[~hard] - want[~hard]) <= ((19 * 2.0 ** -23 + (K / 32 + 12) * 2.0 ** -24) * size
                                               + 2.0 ** -23 * (np.abs(f64(res)) + np.abs(np.where(hard, 0, want))))[~hard])
