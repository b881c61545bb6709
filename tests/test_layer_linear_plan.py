"""The matrix product's plan on the host: refusals, and which kernel the kinds of sizes take. CPU only."""
import ctypes

import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs


@pytest.fixture(scope="module")
def lib():
    return mcs.load(build_if_missing=True)


def plan(B, N, K, O, dtype=torch.bfloat16, heads=0, **kw):
    return mcs.mcs_linear_plan(mcs.linear_desc(B, N, K, O, dtype, heads=heads), **kw)


def test_refusals(lib):
    d, c = mcs.linear_desc(1, 4, 128, 96, torch.bfloat16), mcs.mcs_linear_choice()
    assert lib.mcs_linear_plan(None, 0, 152, ctypes.byref(c)) == 1
    assert lib.mcs_linear_plan(ctypes.byref(d), 0, 152, None) == 1
    assert lib.mcs_linear_plan(ctypes.byref(d), 0, 7, ctypes.byref(c)) == 1
    assert lib.mcs_linear_plan(ctypes.byref(d), 0, 1025, ctypes.byref(c)) == 1
    with pytest.raises(mcs.McsError):
        plan(1, 4, 68, 96)


def test_kernels(lib):
    assert plan(1, 8, 128, 96, torch.float32)[0] == "f32_rows"
    assert plan(1, 9, 128, 96, torch.float32)[0] == "f32_parts"
    assert plan(1, 1, 5120, 5120)[0] == "few"
    for N in (4097, 75600):                                # more rows a section than the few-rows kernel takes
        assert plan(1, N, 64, 8)[0] == "pairs" and plan(2, N, 128, 200, heads=2)[0] == "pairs"


@pytest.mark.parametrize("B,N,heads", [(1, 1, 0), (1, 300, 0), (3, 200, 40), (1, 5000, 0)])
def test_one_accumulator_takes_1536_columns_at_most(lib, B, N, heads):
    for K in (64, 1536, 1600, 5120, 1 << 17, 1 << 20):
        K = K - K % 2560 if heads and K > 2560 else K
        h = K // 64 if heads else 0
        kernel, tile, slices, accs = plan(B, N, K, 1000, heads=h)
        assert 16 <= tile <= 256 and 1 <= slices <= 8
        steps = -(-(-(-K // 64)) // slices)
        assert accs == (1 if steps <= 24 else -(-steps // 16))


@pytest.mark.parametrize("sms", [8, 9, 12, 132, 1024])
def test_any_number_of_sms(lib, sms):
    for dtype in (torch.bfloat16, torch.float32):
        for N in (1, 64, 700, 5000):
            for K in (64, 512, 5120):
                kernel, tile, slices, accs = plan(1, N, K, 1000, dtype, num_sms=sms)
                assert 1 <= slices <= 8 and tile >= 2 and accs >= 1
