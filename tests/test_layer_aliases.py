"""Outputs that alias inputs (or one another) where kernels would read what others have written are
refused on the host. CPU only: validation returns before the first CUDA call."""
import ctypes

import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs

INVALID = 1
B, H, N, D = 2, 3, 60, 64
BLOCK = 2 * B * H * N * D                                # bytes of a bf16 tensor
BASE = 1 << 20


def at(offset):
    return ctypes.c_void_p(BASE + offset)


@pytest.fixture(scope="module")
def lib():
    return mcs.load(build_if_missing=True)


def disjoint(n, size):
    return [at(i * size) for i in range(n)]


@pytest.mark.parametrize("which,offset", [
    (0, 0), (0, 64), (0, -64), (1, 0), (1, 16), (2, 0), (3, 0), (4, 16), (4, -16),
])
def test_linear(lib, which, offset):
    """y against x, w, bias, gate (any overlap) and residual (any but the whole)."""
    d = mcs.linear_desc(2, 64, 128, 128, torch.bfloat16)
    p = disjoint(6, 1 << 18)                            # x, w, bias, gate, residual, y
    p[5] = ctypes.c_void_p(p[which].value + offset)
    assert lib.mcs_linear(ctypes.byref(d), *p, None) == INVALID


def norm(lib, src, dst, st):
    d, r = mcs.make_desc(B, H, N, D, 64, torch.bfloat16), mcs.rope_desc((24, 20, 20), (3, 4, 5))
    return lib.mcs_qk_norm_rope(ctypes.byref(d), ctypes.byref(r), at(1 << 28), None, *src, st, None, None, 1e-6, *dst, None)


def test_norm(lib):
    p = disjoint(6, 1 << 20)
    packed = mcs.mcs_strides(3 * N * H * D, D, 3 * H * D)
    for i in range(3):
        for j in range(3):
            dst = list(p[3:])
            dst[i] = p[j]
            if i != j:                                   # another stream's input
                assert norm(lib, p[:3], dst, None) == INVALID
            assert norm(lib, p[:3], dst, packed) == INVALID   # rows in another order
            dst[i] = ctypes.c_void_p(p[j].value + 2 * D)
            assert norm(lib, p[:3], dst, None) == INVALID
            if i != j:
                dst = list(p[3:])
                dst[i] = dst[j]
                assert norm(lib, p[:3], dst, None) == INVALID


def test_norm_gradient(lib):
    d, r = mcs.make_desc(B, H, N, D, 64, torch.bfloat16), mcs.rope_desc((24, 20, 20), (3, 4, 5))
    need = lib.mcs_qk_norm_rope_bwd_workspace_size(ctypes.byref(d))
    p = disjoint(12, 1 << 20)

    def bwd(dx, dwq=p[8], dwk=p[9], dy=p[2:5], st=None):
        return lib.mcs_qk_norm_rope_bwd(ctypes.byref(d), ctypes.byref(r), at(1 << 28), None, p[0], p[1], st, None, None,
                                        1e-6, *dy, *dx, dwq, dwk, p[10], need, None)

    packed = mcs.mcs_strides(3 * N * H * D, D, 3 * H * D)
    assert bwd(p[5:8], dwk=p[8]) == INVALID              # both weight gradients in one place
    for i in range(3):
        for j in range(3):
            dx = list(p[5:8])
            if i != j:
                dx[i] = dx[j]
                assert bwd(dx) == INVALID
                dx[i] = p[2 + j]                         # another stream's gradient
                assert bwd(dx) == INVALID
                if j < 2:
                    dx[i] = p[j]                         # another stream's input
                    assert bwd(dx) == INVALID
            dx[i] = p[2 + j]
            assert bwd(dx, st=packed) == INVALID         # rows in another order
