"""Projections with adapters: rows of other requests keep their bits whatever a request's adapter holds, in columns too where
the shared weights themselves hold infinities."""
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_adapters_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dout,din", [(300, 200, 640), (40, 129, 2048), (6000, 512, 256), (300, 64, 8)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_infinite_weights_beside_an_adapter_that_is_not_finite(dtype, rows, dout, din, poison):
    cuts = [0, rows // 3, rows // 3 + 2, rows]
    c = Case(dtype, 1, rows, din, dout, 16, cuts, [0, 1, 2])
    for o, k in ((0, 0), (5, 3), (dout - 1, 1)):
        c.w[o, k] = float("inf")
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[cuts[1]:cuts[2]] = False
    a = c.run()
    assert torch.isinf(a[:, keep][:, :, [0, 5, dout - 1]].float()).all()  # x is nowhere 0
    c.up[1].view(-1)[7] = poison
    b = c.run()
    mcs.mcs_check_status()
    assert torch.equal(a[:, keep], b[:, keep])
    assert not torch.isfinite(b[:, ~keep].float()).all()
