"""Projections with adapters: the erf form of GELU in both bf16 products, row by row and in fp32, and the smallest sizes."""
import numpy as np
import pytest
import torch
from scipy.special import erfc

from oracle import packed_oracle as orc
from sparse_attention_diffusion_gb300 import mcs
from tests.test_adapters_gpu import Case, projection_bound

pytestmark = pytest.mark.gpu


def check_erf(c):
    y = c.run()
    mcs.mcs_check_status()
    f = lambda t: t.float().cpu().numpy().astype(np.float64)
    B, N, dout = c.y.shape
    din, R = c.w.shape[1], c.down.shape[1]
    x = f(c.x.transpose(1, 2) if c.heads else c.x).reshape(B * N, din)
    z, size, extra = orc.adapted_projection(x, f(c.w), f(c.bias), c.start, c.which, f(c.down), f(c.up), f(c.scale))
    tol = projection_bound(c.dtype, din, R, size + np.abs(f(c.bias)), extra)
    v = 0.5 * z * erfc(-z / np.sqrt(2.0))
    # The function's slope is below 1.13. Its own error: the argument z / sqrt(2) is off by 2^-23 of itself (a constant and a
    # product), which moves erfc by a factor of at most 1 +- (z^2 + 1.5 |z| + 1) 2^-23; erfcf by 4 units of 2^-23, two products.
    tol = 1.13 * tol + np.abs(v) * (z * z + 1.5 * np.abs(z) + 6) * 2.0 ** -23 + 1e-30
    if c.gate is not None:
        gate, res = np.repeat(f(c.gate), N, axis=0), f(c.residual).reshape(B * N, dout)
        v, tol = res + gate * v, np.abs(gate) * tol + 2.0 ** -23 * np.abs(res)
    half = 2.0 ** -8 if c.dtype == "bf16" else 2.0 ** -23
    tol = tol + half * (np.abs(v) + tol) + 1e-30
    err = np.abs(f(y).reshape(B * N, dout) - v)
    assert np.isfinite(err).all() and (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dtype,rows,din,dout,kernel", [
    ("bf16", 9000, 256, 512, "pairs"), ("bf16", 8600, 1664, 250, "pairs"), ("bf16", 200, 640, 129, "few"), ("bf16", 8, 4096, 512, "few"),
    ("f32", 300, 200, 129, "f32_parts"), ("f32", 5, 2048, 96, "f32_rows"), ("f32", 2600, 512, 64, "f32_parts")])
@pytest.mark.parametrize("gated", [False, True])
def test_gelu_erf(dtype, rows, din, dout, kernel, gated):
    cuts = [0, rows // 3, rows // 3 + 1, rows]
    c = Case(dtype, 1, rows, din, dout, 24, cuts, [2, -1, 0], act="gelu_erf", gated=gated)
    assert mcs.mcs_linear_plan(c.desc, residual=gated)[0] == kernel
    check_erf(c)


def test_gelu_erf_row_by_row():
    """Rows with adapters of their own."""
    for dtype in ("bf16", "f32"):
        check_erf(Case(dtype, 1, 70, 512, 200, 16, list(range(71)), [i % 33 - 1 for i in range(70)], count=32, act="gelu_erf"))


@pytest.mark.parametrize("rows", [1, 2, 300, 9000])
@pytest.mark.parametrize("dout", [1, 3])
def test_smallest_sizes(rows, dout):
    """The narrowest rows, outputs and adapters."""
    Case("bf16", 1, rows, 8, dout, 8, [0, rows], [1]).check()
    Case("bf16", rows, 1, 8, dout, 8, [0, rows // 2, rows], [1, 0], gated=True).check()
    Case("f32", 1, rows, 4, dout, 4, [0, rows], [1]).check()
    Case("f32", rows, 1, 4, dout, 4, [0, rows // 2, rows], [1, 0], gated=True).check()
