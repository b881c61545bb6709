"""Outputs of more than 2^31 elements: rows at the start, around the 32-bit limit and at the
end of a projection, against float64 (tolerances as in the smaller tests)."""
import pytest
import torch

from oracle import layer_oracle as lo
from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import close, f64, linear_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,N,K,O", [("bf16", 270000, 64, 8192), ("bf16", 270000, 64, 8191), ("f32", 270000, 36, 8192)])
def test_linear_past_32_bits(dtype, N, K, O):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(60)
    x = torch.randn(1, N, K, generator=g, device="cuda").to(dt)
    w = torch.randn(O, K, generator=g, device="cuda").to(dt)
    y = torch.empty(1, N, O, dtype=dt, device="cuda")
    mcs.mcs_linear(mcs.linear_desc(1, N, K, O, dt, act="silu"), x, w, None, None, None, y)
    mcs.mcs_check_status()
    edge = 2 ** 31 // O
    rows = [0, 1, 255, edge - 1, edge, edge + 1, N - 2, N - 1]
    xr = f64(x[:, rows])
    want, z = lo.linear(xr, f64(w), act="silu")
    close(y[:, rows], want, linear_bound(xr, f64(w), want, z, "silu", None, dtype), "rows")
    del y
    torch.cuda.empty_cache()
