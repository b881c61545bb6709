"""Matrix products of long rows back to back, each reading what the one before it wrote and writing
onto what it read: the bits of the same chain synchronised after every call, and of a captured one."""
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import DT, gen, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,M,K,kernel", [("bf16", 300, 1800, "few"), ("bf16", 1300, 2056, "pairs"),
                                              ("bf16", 12000, 1800, "pairs"), ("bf16", 3, 8192, "few"), ("f32", 150, 1800, "f32_parts")])
def test_back_to_back(dtype, M, K, kernel):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    desc = mcs.linear_desc(1, M, K, K, DT[dtype], act="silu")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert mcs.mcs_linear_plan(desc, False, sms)[0] == kernel
    g = gen(120)
    w = [(rand(g, K, K) / K ** 0.5).to(DT[dtype]) for _ in range(2)]
    start = rand(g, 1, M, K, dtype=dtype)
    a, b = torch.empty_like(start), torch.empty_like(start)

    def chain(sync):
        a.copy_(start)
        for _ in range(6):
            mcs.mcs_linear(desc, a, w[0], None, None, None, b)
            if sync:
                torch.cuda.synchronize()
            mcs.mcs_linear(desc, b, w[1], None, None, a, a)
            if sync:
                torch.cuda.synchronize()

    chain(True)
    want = (a.clone(), b.clone())
    assert all(bool(t.isfinite().all()) for t in want)
    for _ in range(3):
        chain(False)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(False)
    a.zero_(), b.zero_()
    graph.replay()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    mcs.mcs_check_status()
