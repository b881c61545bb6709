"""Activations of the matrix product over their negative tails, down to the smallest normal
numbers, in both types and by each kernel's way out.

fp32: expf is right to 2 ulp, taken twice at half the argument (4 ulp), and five more operations
round: 8 * 2^-23 relative. The argument of GELU's tanh form has 6 roundings (3 * 2^-23 |t|), that
of its erf form two (z^2 * 2^-23, counted twice). bf16: the store's 2^-8 and at most 2^-14 of the
fast exponential and of the same arguments.
"""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from sparse_attention_diffusion_gb300 import mcs
from tests.test_layer_ops_gpu import f64

pytestmark = pytest.mark.gpu


def product(x, w, act):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    mcs.load(build_if_missing=True)
    B, M, K = x.shape
    y = torch.empty(B, M, w.shape[0], dtype=x.dtype, device="cuda")
    mcs.mcs_linear(mcs.linear_desc(B, M, K, w.shape[0], x.dtype, act=act), x, w, None, None, None, y)
    mcs.mcs_check_status()
    return y


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("M", [8, 64])
def test_activations_keep_their_digits(M, act):
    z = torch.linspace(-91, 12, 64 * 16).float().reshape(16, 64)
    for row in z if M == 64 else z.reshape(-1, 8):
        x = torch.zeros(1, M, 8)
        x[0, :, 0] = row
        w = torch.zeros(1, 8)
        w[0, 0] = 1.0
        got, zn = f64(product(x.cuda(), w.cuda(), act))[0, :, 0], f64(row)
        want = lo.activate(zn, act)
        rel = {"silu": 8 + 0 * zn, "gelu_tanh": 8 + 3 * 1.6 * np.abs(zn + 0.044715 * zn ** 3),
               "gelu_erf": 8 + 2 * zn * zn}[act]
        seen = np.abs(want) >= 2.0 ** -126
        off = np.abs(got - want)
        assert np.all(off[seen] <= (rel * 2.0 ** -23 * np.abs(want))[seen]), (act, zn[seen][np.argmax(off[seen] / np.abs(want[seen]))])
        assert np.all(off[~seen] <= 2.0 ** -126)


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu_erf", "silu"])
@pytest.mark.parametrize("M", [8, 300, 4600])
def test_bf16_tails(M, act):
    z = torch.linspace(-91, 12, M).bfloat16()
    x = torch.zeros(1, M, 8, dtype=torch.bfloat16)
    x[0, :, 0] = z
    w = torch.zeros(8, 8, dtype=torch.bfloat16)
    w[:, 0] = 1.0
    got = f64(product(x.cuda(), w.cuda(), act))[0]
    want = lo.activate(f64(z), act)[:, None]
    seen = (np.abs(want) >= 2.0 ** -126)[:, 0]
    assert np.all(np.abs(got - want)[seen] <= (2.0 ** -8 + 2.0 ** -14) * np.abs(want)[seen]), f64(z)[seen][
        np.argmax((np.abs(got - want)[seen] / np.abs(want)[seen]).max(1))]
    assert np.all(np.abs(got - want)[~seen] <= 2.0 ** -126)
