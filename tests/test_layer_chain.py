"""Calls whose launches overlap their predecessor's end, each reading what the one
before it wrote (and overwriting what the one before that read): a chain over all the
layer's kernels without a synchronisation in between gives the bits of the same chain
synchronised after every call."""
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import DT, gen, rand

pytestmark = pytest.mark.gpu


def chain(dtype, N, sync, rounds=12):
    B, H, d = 1, 4, 64
    hid = H * d
    desc = mcs.make_desc(B, H, N, d, 64, DT[dtype])
    g = gen(50)
    rope = mcs.rope_desc((24, 20, 20), (N, 1, 1))
    table = mcs.rope_table(rope)
    w1, w2 = ((rand(g, o, i) / i ** 0.5).to(DT[dtype]) for o, i in ((3 * hid, hid), (hid, hid)))
    wn, x = rand(g, d, dtype=dtype), rand(g, B, N, hid, dtype=dtype)
    up = mcs.linear_desc(B, N, hid, 3 * hid, DT[dtype], act="silu")
    out = mcs.linear_desc(B, N, hid, hid, DT[dtype], heads=H)
    qkv = torch.empty(B, N, 3, H, d, dtype=DT[dtype], device="cuda")
    q, k, v, r = (torch.empty(B, H, N, d, dtype=DT[dtype], device="cuda") for _ in range(4))
    grad, dw = torch.empty_like(qkv), torch.empty(d, device="cuda")
    ws = mcs.qk_norm_rope_bwd_workspace(desc)
    views = lambda t: [t[:, :, i].transpose(1, 2) for i in range(3)]
    calls = [
        lambda: mcs.mcs_linear(up, x, w1, None, None, None, qkv.view(B, N, 3 * hid)),
        lambda: mcs.mcs_qk_norm_rope(desc, rope, table, None, *views(qkv), wn, None, 1e-6, q, k, v),
        lambda: mcs.mcs_rope_apply(desc, rope, table, None, q, r, True),
        lambda: mcs.mcs_qk_norm_rope_bwd(desc, rope, table, None, *views(qkv)[:2], wn, wn, 1e-6, r, k, v, *views(grad), dw,
                                         None, ws),
        lambda: mcs.mcs_linear(out, r, w2, None, None, x, x),
        lambda: mcs.mcs_dense_attn(desc, q, k, v, r, None),
        lambda: mcs.mcs_linear(out, r, w2, None, None, None, x),
    ]
    for _ in range(rounds):
        for call in calls:
            call()
            if sync:
                torch.cuda.synchronize()
    mcs.mcs_check_status()
    return [t.clone() for t in (x, qkv, q, k, v, r, grad, dw)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 7, 60, 700, 3001])
def test_back_to_back_equals_synchronised(dtype, N):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    want = chain(dtype, N, True)
    assert all(bool(t.isfinite().all()) for t in want)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(dtype, N, False), want))
