"""What mcs_packed_attn refuses before it launches anything (CPU only: pointers are never read)."""
import ctypes

import pytest

from sparse_attention_diffusion_gb300 import mcs

FIELDS = ("S", "Tq", "Tk", "H", "Hk", "d", "dtype", "causal", "max_q", "scale")
GOOD = dict(S=2, Tq=100, Tk=100, H=8, Hk=2, d=64, dtype=mcs.MCS_BF16, causal=1, max_q=0, scale=0.0)


@pytest.fixture(scope="module")
def lib():
    return mcs.load(build_if_missing=True)


def desc(**kw):
    return mcs.mcs_packed_desc(*[{**GOOD, **kw}[f] for f in FIELDS])


@pytest.mark.parametrize("kw", [
    dict(S=0), dict(Tq=0), dict(Tk=0), dict(H=0), dict(Hk=0), dict(H=7), dict(d=96), dict(d=32), dict(dtype=3),
    dict(H=130, Hk=2), dict(max_q=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(Tq=(1 << 30) + 1),
    dict(Tk=(1 << 30) + 1), dict(H=1 << 21, Hk=1 << 21),
])
def test_descriptions(lib, kw):
    assert lib.mcs_packed_attn_workspace_size(ctypes.byref(desc(**kw))) == 0
    assert run(lib, desc(**kw)) in (1, 2)


def test_missing_description(lib):
    assert lib.mcs_packed_attn_workspace_size(None) == 0


def run(lib, d, strides=(None,) * 4, **kw):
    """The call with made-up addresses far apart."""
    a = dict(q=1 << 40, k=2 << 40, v=3 << 40, q_start=4 << 40, k_start=5 << 40, o=6 << 40, lse=7 << 40, ws=8 << 40, n=1 << 38)
    a.update(kw)
    st = [None if s is None else mcs.mcs_strides(0, *s) for s in strides]
    return lib.mcs_packed_attn(ctypes.byref(d), a["q"], st[0], a["k"], st[1], a["v"], st[2], a["q_start"], a["k_start"],
                               a["o"], st[3], a["lse"], a["ws"], a["n"], None)


@pytest.mark.parametrize("name", ["q", "k", "v", "q_start", "k_start", "o"])
def test_pointers(lib, name):
    assert run(lib, desc(), **{name: None}) == 1
    assert run(lib, desc(), **{name: (9 << 40) + 8}) == 1


def test_workspace(lib):
    d = desc(Tk=9000, max_q=1)
    n = lib.mcs_packed_attn_workspace_size(ctypes.byref(d))
    assert n > 16
    assert run(lib, d, n=n - 1) == 3
    assert run(lib, d, ws=None) == 3
    assert run(lib, d, ws=(8 << 40) + 4) == 3


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("s", [(64, 63), (-64, 512), (100 * 64, 68), (32, 512), (50 * 64, 64), (1 << 50, 64), (64, 7 * 64)])
def test_strides(lib, which, s):
    """Not of 16 bytes, negative, rows that overlap (8 heads of queries, 2 of keys)."""
    heads = 8 if which in (0, 3) else 2
    if heads == 2 and s == (64, 7 * 64):
        return  # two heads fit in that row
    st = [None] * 4
    st[which] = s
    assert run(lib, desc(), st) == 1


@pytest.mark.parametrize("out", ["o", "lse", "ws"])
@pytest.mark.parametrize("of", ["q", "k", "v", "q_start", "k_start", "o", "lse", "ws"])
def test_outputs_overlap_nothing(lib, out, of):
    if out == of:
        return
    at = {"q": 1 << 40, "k": 2 << 40, "v": 3 << 40, "q_start": 4 << 40, "k_start": 5 << 40, "o": 6 << 40, "lse": 7 << 40, "ws": 8 << 40}
    d = desc(Tk=9000, max_q=1)
    need = lib.mcs_packed_attn_workspace_size(ctypes.byref(d))
    assert run(lib, d, n=need, **{out: at[of]}) == 1
