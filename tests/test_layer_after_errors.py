"""A call that failed on the host leaves nothing behind that the next call reports as its own."""
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import f64, gen, rand

pytestmark = pytest.mark.gpu


def linear(M=40, K=128, O=72, dtype="bf16"):
    g = gen(110)
    x, w = rand(g, 1, M, K, dtype=dtype), rand(g, O, K, dtype=dtype)
    y = torch.empty(1, M, O, dtype=x.dtype, device="cuda")
    mcs.mcs_linear(mcs.linear_desc(1, M, K, O, x.dtype), x, w, None, None, None, y)
    return y


def test_calls_after_a_failed_one():
    """mcs_check_status waits for its stream, which a stream under capture refuses: the capture is lost and the call
    fails; everything after it works."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    want = linear()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin()
        with pytest.raises(mcs.McsError):
            mcs.mcs_check_status()
        with pytest.raises(Exception):
            graph.capture_end()
    got = linear()
    mcs.mcs_check_status()
    assert torch.equal(got, want)
    rope = mcs.rope_desc((64,), (5,))
    table = mcs.rope_table(rope)
    x = torch.ones(1, 1, 5, 64, device="cuda")
    out = torch.empty_like(x)
    mcs.mcs_rope_apply(mcs.make_desc(1, 1, 5, 64, 64, torch.float32), rope, table, None, x, out)
    mcs.mcs_check_status()
    assert abs(float((f64(out) ** 2).sum()) - 5 * 64) < 1e-3
