"""The bf16 matrix product on CTA pairs and with wide token tiles against the float64 oracle:
several k steps, ring turns and accumulators, several tiles a pair, residual pieces that cross
tiles, gates that change inside a tile, head-by-head inputs of several batches, all activations,
odd outputs. Every case says which kernel it is meant for, and that is checked first."""
import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import check_linear, gen, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mcs.load(build_if_missing=True)


def check(kernel, B, N, K, O, act="none", bias=False, gate=False, residual=False, heads=0, wide=0, long=False):
    """check_linear after a look at the plan: the kernel, tiles of at least `wide`, several accumulators if `long`."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plan = mcs.mcs_linear_plan(mcs.linear_desc(B, N, K, O, torch.bfloat16, act=act, heads=heads), residual, sms)
    assert plan[0] == kernel and plan[1] >= wide and (plan[3] > 1) == long, plan
    check_linear("bf16", B, N, K, O, act, bias, gate, residual, heads=heads)


@pytest.mark.parametrize("N,K,O", [(4097, 64, 8), (5000, 320, 520), (5000, 1032, 33), (5000, 1032, 1002), (12000, 1096, 72),
                                   (20000, 136, 1560)])
def test_pairs(N, K, O):
    check("pairs", 1, N, K, O, bias=True, residual=True)
    check("pairs", 1, N, K, O)


@pytest.mark.parametrize("N,K,O,wide", [(4500, 2056, 264, 96), (12000, 1800, 72, 96), (20000, 1640, 777, 224),
                                        (30000, 2600, 520, 192), (1000, 1800, 2056, 128), (400, 4096, 5120, 160)])
def test_pairs_long_rows(N, K, O, wide):
    """Rows of several accumulators, in narrow and wide tiles, several tiles a pair and fewer than pairs."""
    check("pairs", 1, N, K, O, bias=True, residual=True, wide=wide, long=True)
    check("pairs", 1, N, K, O, "gelu_erf", wide=wide, long=True)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("B,N,K,O", [(3, 1500, 328, 296), (2, 2100, 136, 131), (5, 1001, 72, 50), (3, 1500, 1800, 296),
                                     (2, 2100, 3208, 131), (2, 9000, 1800, 456)])
def test_pairs_epilogues(act, B, N, K, O):
    """Batch boundaries, and so gates, inside row tiles."""
    check("pairs", B, N, K, O, act, True, True, True, long=K > 1536)
    check("pairs", B, N, K, O, act, False, True, False, long=K > 1536)


@pytest.mark.parametrize("B,heads,N,d,O", [(2, 3, 4500, 64, 200), (2, 2, 4500, 128, 136), (1, 18, 4200, 64, 328),
                                           (1, 1, 4200, 64, 77), (2, 26, 4500, 64, 200), (1, 16, 4200, 128, 328),
                                           (2, 15, 5000, 128, 999)])
def test_pairs_from_heads(B, heads, N, d, O):
    check("pairs", B, N, heads * d, O, "none", True, True, True, heads=heads, long=heads * d > 1536)


@pytest.mark.parametrize("M,K,O,wide,long", [
    (224, 2048, 2560, 112, False), (160, 2048, 5120, 160, False), (128, 5120, 5120, 128, True), (128, 13824, 1000, 128, True),
    (192, 5120, 5120, 192, True), (224, 5120, 5128, 224, True), (256, 5120, 5120, 256, True), (300, 5120, 2560, 160, True),
    (512, 8192, 1000, 128, True), (100, 40000, 4104, 112, True),
])
def test_wide_token_tiles(M, K, O, wide, long):
    check("few", 1, M, K, O, "gelu_tanh", True, True, True, wide=wide, long=long)


@pytest.mark.parametrize("O", [20480, 20487])
def test_two_rows_of_many_accumulators(O):
    check("few", 2, 1, 32768, O, "silu", True, True, True, long=True)


def test_wide_token_tiles_from_heads():
    check("few", 2, 128, 40 * 128, 5000, "none", True, True, True, heads=40, wide=128, long=True)


def test_nan_stays_in_its_row_on_pairs():
    g = gen(95)
    M, K, O = 4600, 1100 * 8, 264
    x, w = rand(g, 1, M, K, dtype="bf16"), rand(g, O, K, dtype="bf16")
    desc = mcs.linear_desc(1, M, K, O, torch.bfloat16, act="gelu_erf")
    clean, y = (torch.empty(1, M, O, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mcs.mcs_linear(desc, x, w, None, None, None, clean)
    x[0, 4099, K - 1] = float("nan")
    mcs.mcs_linear(desc, x, w, None, None, None, y)
    keep = [m for m in range(M) if m != 4099]
    assert torch.equal(y[0, keep], clean[0, keep]) and bool(y[0, 4099].isnan().all())
