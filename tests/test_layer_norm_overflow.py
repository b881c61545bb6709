"""The norm and its gradient for rows whose sum of squares leaves fp32, for large and tiny
gradients, and for rows that are large and small in one call.

A row whose sum of squares overflows counts as infinitely long: its normalised values are 0, so
its outputs and its gradient are 0 and it adds nothing to the weight gradient. Rows of ordinary
length keep the tolerances of ordinary calls at any size of the gradient that keeps every term
of the formula in fp32's normal range.
"""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import DT, STORE, U, both, close, f64, gen, rand

pytestmark = pytest.mark.gpu
B, H, N, D = 1, 2, 60, 64


def run(x, w, dy, eps, style="interleaved"):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    r, table, orc = both((24, 20, 20), (3, 4, 5), style=style)
    b, h, n, d = x.shape
    desc = mcs.make_desc(b, h, n, d, 64, x.dtype)
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(d, device="cuda")
    mcs.mcs_qk_norm_rope(desc, r, table, None, x, None, None, w, None, eps, y, None, None)
    mcs.mcs_qk_norm_rope_bwd(desc, r, table, None, x, None, w, None, eps, dy, None, None, dx, None, None, dw, None,
                             mcs.qk_norm_rope_bwd_workspace(desc))
    mcs.mcs_check_status()
    return y, dx, dw, orc


def check(x, w, dy, eps, y, dx, dw, orc, dtype):
    """Against the oracle, whose rows longer than fp32 can square are taken out (zeros)."""
    eps = float(np.float32(eps))
    xn, wn, yn = f64(x), f64(w), f64(dy)
    live = (xn * xn).sum(-1, keepdims=True) < 2.0 ** 128
    xn = np.where(live, xn, 0.0)
    rstd = np.where(live, 1.0 / np.sqrt((xn * xn).mean(-1, keepdims=True) + eps), 0.0)
    want = lo.norm_rotate(xn, wn, eps, orc)
    close(y, want, STORE[dtype] * np.abs(want) + 20 * U * lo.pair_size(xn * rstd * wn, orc), "y")
    want, wantw = lo.norm_rotate_grad(xn, wn, eps, yn, orc)
    want = np.where(live, want, 0.0)
    G, xh = lo.pair_size(yn, orc), np.abs(xn * rstd)
    size = rstd * (G * np.abs(wn) + xh * (G * np.abs(wn) * xh).mean(-1, keepdims=True))
    close(dx, want, STORE[dtype] * np.abs(want) + 72 * U * size, "dx")
    close(dw, wantw, (20 + 256 + 64) * U * (G * xh).sum((0, 1, 2)), "dw")


@pytest.mark.parametrize("style", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size,g", [(2e19, 1.0), (3e36, 1.0), (3.3e38, 2.0), (3.3e38, 1e20)])
def test_rows_beyond_fp32_squares(dtype, size, g, style):
    """Rows of all signs at `size` between ordinary ones: zeros there, ordinary results elsewhere."""
    r = gen(71)
    x, w = rand(r, B, H, N, D, dtype=dtype), rand(r, D, dtype=dtype)
    dy = (rand(r, B, H, N, D) * g).to(DT[dtype])
    for h, n in ((0, 0), (0, 17), (1, 18), (1, 59)):
        sign = torch.where(torch.arange(D) % 3 == 0, -1.0, 1.0).cuda()
        x[0, h, n] = (size * sign).to(DT[dtype])
        dy[0, h, n] = dy[0, h, n].abs()
    check(x, w, dy, 1e-6, *run(x, w, dy, 1e-6, style), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,eps,g", [
    (1e16, 1e-6, 1e-12), (1e17, 1e-6, 1e-10), (1e16, 1e-6, 1e5), (1.0, 1e-6, 1e-25), (1.0, 1e-6, 1e30),
    (1e-13, 1e-20, 1e5), (1e-13, 1e-20, 1e-20), (1e-17, 1e-34, 1e5), (1e-17, 1e-34, 1e-12),
])
def test_sizes_of_the_gradient(dtype, scale, eps, g):
    r = gen(72)
    x = (rand(r, B, H, N, D) * scale).to(DT[dtype])
    w, dy = rand(r, D, dtype=dtype), (rand(r, B, H, N, D) * g).to(DT[dtype])
    check(x, w, dy, eps, *run(x, w, dy, eps), dtype)
