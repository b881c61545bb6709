"""Rotary positions, query/key norms and projections reject bad arguments on the host,
before any launch. CPU only: validation returns before the first CUDA call."""
import ctypes

import pytest
import torch

from sparse_attention_diffusion_gb300 import mcs

A, MIS = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return mcs.load(build_if_missing=True)


def desc(**kw):
    base = dict(B=2, H=3, N=60, d=64, C=64, dtype=torch.bfloat16)
    base.update(kw)
    return mcs.make_desc(*[base[k] for k in ("B", "H", "N", "d", "C", "dtype")])


def rope(**kw):
    base = dict(dims=(24, 20, 20), lens=(3, 4, 5))
    base.update(kw)
    return mcs.rope_desc(**base)


def test_table_size(lib):
    assert lib.mcs_rope_table_size(ctypes.byref(rope())) == 8 * (3 * 12 + 4 * 10 + 5 * 10)
    assert lib.mcs_rope_table_size(ctypes.byref(rope(dims=(64,), lens=(7,)))) == 8 * 7 * 32
    assert lib.mcs_rope_table_size(None) == 0
    assert lib.mcs_rope_table(ctypes.byref(rope()), None, None) == INVALID
    assert lib.mcs_rope_table(ctypes.byref(rope()), MIS, None) == INVALID


BAD_ROPES = [
    (dict(dims=(23, 20, 20)), UNSUPPORTED),            # odd
    (dict(dims=(0, 20, 20)), UNSUPPORTED),
    (dict(dims=(130, 20, 20)), UNSUPPORTED),
    (dict(lens=(0, 4, 5)), INVALID),
    (dict(first=-1), INVALID),
    (dict(theta=0.0), INVALID),
    (dict(theta=float("inf")), INVALID),
    (dict(start=(float("nan"), 0, 0)), INVALID),
    (dict(scale=(1, float("inf"), 1)), INVALID),
    (dict(dims=(64,), lens=(2 ** 30,)), UNSUPPORTED),  # table past 2^31 entries
]


@pytest.mark.parametrize("kw,code", BAD_ROPES)
def test_bad_ropes(lib, kw, code):
    r, d = rope(**kw), desc()
    assert lib.mcs_rope_table_size(ctypes.byref(r)) == 0
    assert lib.mcs_rope_table(ctypes.byref(r), A, None) == code
    assert lib.mcs_rope_apply(ctypes.byref(d), ctypes.byref(r), A, None, A, None, A, None, 0, None) == code
    assert lib.mcs_qk_norm_rope(ctypes.byref(d), ctypes.byref(r), A, None, A, None, None, None, None, None, 1e-6, A,
                                None, None, None) == code


def test_rope_axes_and_style_out_of_range(lib):
    for field, value, code in (("axes", 0, INVALID), ("axes", 4, INVALID), ("style", 2, UNSUPPORTED)):
        r = rope()
        setattr(r, field, value)
        assert lib.mcs_rope_table(ctypes.byref(r), A, None) == code
    with pytest.raises(ValueError):
        rope(style="thirds")
    with pytest.raises(ValueError):
        rope(dims=(24, 20), lens=(3, 4, 5))


def apply(lib, d=None, r=None, table=A, pos=None, x=A, xs=None, out=A, os=None):
    d, r = d or desc(), r or rope()
    return lib.mcs_rope_apply(ctypes.byref(d), ctypes.byref(r), table, pos, x, xs, out, os, 0, None)


def test_apply_refusals(lib):
    assert apply(lib, table=None) == INVALID
    assert apply(lib, x=None) == INVALID
    assert apply(lib, out=MIS) == INVALID
    assert apply(lib, pos=MIS) == INVALID
    assert apply(lib, r=rope(lens=(3, 4, 6))) == INVALID                           # grid of 72 tokens, N = 60
    assert apply(lib, r=rope(first=1)) == INVALID                                  # grid ends at 61
    assert apply(lib, r=rope(lens=(2 ** 15, 2 ** 15, 2 ** 15))) == INVALID         # token count past 64-bit ranges
    assert apply(lib, r=rope(dims=(24, 22, 20))) == UNSUPPORTED                    # 66 > d
    assert apply(lib, r=rope(dims=(22, 20, 20), style="half")) == UNSUPPORTED      # halves need the whole head
    assert apply(lib, d=desc(d=96)) == UNSUPPORTED
    assert apply(lib, d=desc(N=0)) == INVALID
    S = mcs.mcs_strides
    assert apply(lib, xs=S(11520, 3840, 68)) == INVALID                            # token stride of 136 bytes
    assert apply(lib, xs=S(11520, -3840, 64)) == INVALID
    assert apply(lib, os=S(0, 3840, 64)) == INVALID                                # batches written on each other
    assert apply(lib, os=S(11520, 3840, 32)) == INVALID                            # rows overlap
    assert apply(lib, os=S(11520, 64, 128)) == INVALID                             # three heads, room for two
    assert apply(lib, xs=S(11520, 3840, 64), os=S(11520, 64, 192)) == INVALID      # in place with other strides


def norm(lib, q=A, k=A, v=A, qo=A, ko=A, vo=A, wq=A, wk=A, eps=1e-6, st=None):
    return lib.mcs_qk_norm_rope(ctypes.byref(desc()), ctypes.byref(rope()), A, None, q, k, v, st, wq, wk, eps, qo, ko,
                                vo, None)


def test_norm_refusals(lib):
    assert norm(lib, q=None) == INVALID                 # output without input
    assert norm(lib, ko=None) == INVALID
    assert norm(lib, None, None, None, None, None, None) == INVALID
    assert norm(lib, v=MIS) == INVALID
    assert norm(lib, wq=MIS) == INVALID
    assert norm(lib, wk=MIS) == INVALID
    assert norm(lib, eps=0.0) == INVALID
    assert norm(lib, eps=float("nan")) == INVALID
    assert norm(lib, st=mcs.mcs_strides(11520, 3840, 4)) == INVALID


def test_norm_bwd_refusals(lib):
    d = desc()
    need = lib.mcs_qk_norm_rope_bwd_workspace_size(ctypes.byref(d))
    assert need > 0 and lib.mcs_qk_norm_rope_bwd_workspace_size(ctypes.byref(desc(d=96))) == 0

    def bwd(q=A, k=A, st=None, dqo=A, dko=A, dvo=A, dq=A, dk=A, dv=A, dwq=A, dwk=A, ws=A, n=need, eps=1e-6):
        return lib.mcs_qk_norm_rope_bwd(ctypes.byref(d), ctypes.byref(rope()), A, None, q, k, st, A, A, eps, dqo, dko,
                                        dvo, dq, dk, dv, dwq, dwk, ws, n, None)

    assert bwd(q=None) == INVALID                       # gradient without the forward's input
    assert bwd(dqo=None) == INVALID
    assert bwd(dv=None) == INVALID
    assert bwd(q=None, dqo=None, dq=None) == INVALID    # weight gradient of an absent stream
    assert bwd(dwk=MIS) == INVALID
    assert bwd(eps=-1.0) == INVALID
    assert bwd(st=mcs.mcs_strides(0, 3840, 64)) == INVALID
    assert bwd(ws=None) == WORKSPACE
    assert bwd(ws=MIS) == WORKSPACE
    assert bwd(n=need - 1) == WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(in_features=0), INVALID), (dict(out_features=0), INVALID),
    (dict(heads=-1), INVALID), (dict(dtype=5), UNSUPPORTED), (dict(act=4), UNSUPPORTED), (dict(act=-1), UNSUPPORTED),
    (dict(in_features=68), UNSUPPORTED), (dict(in_features=66, dtype=0), UNSUPPORTED),
    (dict(in_features=2 ** 20 + 8), UNSUPPORTED), (dict(out_features=2 ** 20 + 1), UNSUPPORTED),
    (dict(B=2 ** 16, N=2 ** 15), UNSUPPORTED), (dict(heads=3), UNSUPPORTED), (dict(heads=4), UNSUPPORTED),
])
def test_bad_linears(lib, kw, code):
    base = dict(B=1, N=4, in_features=128, out_features=96, heads=0, dtype=1, act=0)
    base.update(kw)
    d = mcs.mcs_linear_desc(**base)
    assert lib.mcs_linear(ctypes.byref(d), A, A, A, A, A, A, None) == code


def test_linear_bad_pointers(lib):
    d = mcs.linear_desc(1, 4, 128, 96, torch.bfloat16)
    for bad in range(6):
        for p in (MIS, None):
            if p is None and bad in (2, 3, 4):
                continue                                # bias, gate and residual may be absent
            args = [A] * 6
            args[bad] = p
            assert lib.mcs_linear(ctypes.byref(d), *args, None) == INVALID
    assert lib.mcs_linear(None, A, A, A, A, A, A, None) == INVALID
    with pytest.raises(ValueError):
        mcs.linear_desc(1, 4, 128, 96, torch.bfloat16, act="relu")


def test_binding_refuses_host_and_misshapen_tensors():
    d, r = desc(), rope()
    table = torch.empty(126, 2)
    x = torch.empty(2, 3, 60, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected"):
        mcs.mcs_rope_apply(d, r, table, None, x[:, :, :59], x)
    with pytest.raises(ValueError, match="current device"):
        mcs.mcs_rope_apply(d, r, table, None, x, x)
    with pytest.raises(ValueError, match="table"):
        mcs.mcs_rope_apply(d, r, table[:100], None, x, x)
    with pytest.raises(ValueError, match="pos"):
        mcs.mcs_rope_apply(d, r, table, torch.zeros(2, 60, 2, dtype=torch.int32), x, x)
    with pytest.raises(ValueError, match="wq"):
        mcs.mcs_qk_norm_rope(d, r, table, None, x, x, x, torch.empty(64), None, 1e-6, x, x, x)
    ld = mcs.linear_desc(2, 60, 192, 96, torch.bfloat16, heads=3)
    w = torch.empty(96, 192, dtype=torch.bfloat16)
    y = torch.empty(2, 60, 96, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x: expected"):
        mcs.mcs_linear(ld, torch.empty(2, 60, 192, dtype=torch.bfloat16), w, None, None, None, y)
    with pytest.raises(ValueError, match="gate"):
        mcs.mcs_linear(ld, x, w, None, torch.empty(1, 96, dtype=torch.bfloat16), None, y)
    with pytest.raises(ValueError, match="device tensors"):
        mcs.mcs_linear(ld, x, w, None, None, None, y)


@pytest.mark.parametrize("kw", [dict(start=(1e308, 0, 0), scale=(100.0, 1, 1)), dict(theta=1e-307, start=(1e10, 0, 0))])
def test_infinite_angles(lib, kw):
    r = rope(**kw)
    assert lib.mcs_rope_table_size(ctypes.byref(r)) == 0
    assert lib.mcs_rope_table(ctypes.byref(r), A, None) == INVALID
