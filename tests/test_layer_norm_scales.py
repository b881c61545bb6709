"""Norm, rotation and their gradient for rows far from 1: large rows, whose reciprocal norm
has a cube below fp32's range, and small ones beside eps. Tolerances as at scale 1; the
gradient's reciprocal norm enters as a product of bounded factors."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import DT, STORE, U, both, close, f64, gen, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,eps", [(1e16, 1e-6), (1e13, 1e-6), (1e-3, 1e-6), (1e-13, 1e-20), (1e-17, 1e-34)])
def test_norm_scales(dtype, scale, eps):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    B, H, N, d = 1, 2, 60, 64
    r, table, orc = both((24, 20, 20), (3, 4, 5))
    desc = mcs.make_desc(B, H, N, d, 64, DT[dtype])
    g = gen(70)
    x = (rand(g, B, H, N, d) * scale).to(DT[dtype])
    w, dy = rand(g, d, dtype=dtype), rand(g, B, H, N, d, dtype=dtype)
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(d, device="cuda")
    mcs.mcs_qk_norm_rope(desc, r, table, None, x, None, None, w, None, eps, y, None, None)
    mcs.mcs_qk_norm_rope_bwd(desc, r, table, None, x, None, w, None, eps, dy, None, None, dx, None, None, dw, None,
                             mcs.qk_norm_rope_bwd_workspace(desc))
    mcs.mcs_check_status()
    eps = float(np.float32(eps))
    xn, wn, yn = f64(x), f64(w), f64(dy)
    rstd = 1.0 / np.sqrt((xn * xn).mean(-1, keepdims=True) + eps)
    want = lo.norm_rotate(xn, wn, eps, orc)
    close(y, want, STORE[dtype] * np.abs(want) + 20 * U * lo.pair_size(xn * rstd * wn, orc), "y")
    want, wantw = lo.norm_rotate_grad(xn, wn, eps, yn, orc)
    G, xh = lo.pair_size(yn, orc), np.abs(xn * rstd)
    size = rstd * (G * np.abs(wn) + xh * (G * np.abs(wn) * xh).mean(-1, keepdims=True))
    close(dx, want, STORE[dtype] * np.abs(want) + 72 * U * size, "dx")
    close(dw, wantw, (20 + 256 + 64) * U * (G * xh).sum((0, 1, 2)), "dw")
