"""What mcs_linear_adapters refuses before it launches anything (CPU only: pointers are never read)."""
import ctypes

import pytest

from sparse_attention_diffusion_gb300 import mcs


@pytest.fixture(scope="module")
def lib():
    return mcs.load(build_if_missing=True)


def descs(dtype="bf16", **kw):
    a = {**dict(B=2, N=100, i=512, o=256, heads=0, act="none", count=3, rank=16, segments=4), **kw}
    return (mcs.linear_desc(a["B"], a["N"], a["i"], a["o"], dtype, act=a["act"], heads=a["heads"]),
            mcs.adapters_desc(a["count"], a["rank"], a["segments"]))


AT = {n: (i + 1) << 40 for i, n in enumerate(("x", "w", "bias", "gate", "residual", "down", "up", "scale", "start", "which", "y", "ws"))}


def run(lib, d, a, n=1 << 38, **kw):
    p = {**AT, **kw}
    return lib.mcs_linear_adapters(ctypes.byref(d), None if a is None else ctypes.byref(a), p["x"], p["w"], p["bias"], p["gate"],
                                   p["residual"], p["down"], p["up"], p["scale"], p["start"], p["which"], p["y"], p["ws"], n, None)


@pytest.mark.parametrize("kw", [dict(count=0), dict(rank=0), dict(rank=12), dict(rank=264), dict(segments=0), dict(count=(1 << 20) + 1),
                                dict(segments=(1 << 20) + 1), dict(N=0), dict(i=511), dict(o=0), dict(heads=3)])
def test_descriptions(lib, kw):
    d, a = descs(**kw)
    assert lib.mcs_linear_adapters_workspace_size(ctypes.byref(d), ctypes.byref(a)) == 0
    assert run(lib, d, a) in (1, 2)


def test_rank_by_type(lib):
    d, a = descs("f32", rank=12)
    assert lib.mcs_linear_adapters_workspace_size(ctypes.byref(d), ctypes.byref(a)) > 0
    d, a = descs("f32", rank=6)
    assert run(lib, d, a) == 2
    assert lib.mcs_linear_adapters_workspace_size(ctypes.byref(d), None) == 0
    assert run(lib, d, None) == 1


@pytest.mark.parametrize("name", sorted(AT))
def test_pointers(lib, name):
    d, a = descs()
    code = 3 if name == "ws" else 1
    if name not in ("bias", "gate", "residual"):
        assert run(lib, d, a, **{name: None}) == code
    assert run(lib, d, a, **{name: AT[name] + 8}) == code


def test_workspace(lib):
    for dtype in ("bf16", "f32"):
        d, a = descs(dtype)
        n = lib.mcs_linear_adapters_workspace_size(ctypes.byref(d), ctypes.byref(a))
        assert run(lib, d, a, n=n - 1) == 3


@pytest.mark.parametrize("out", ["y", "ws"])
@pytest.mark.parametrize("of", sorted(AT))
def test_outputs_overlap_nothing(lib, out, of):
    if out == of or (out, of) == ("y", "residual"):
        return
    d, a = descs()
    n = lib.mcs_linear_adapters_workspace_size(ctypes.byref(d), ctypes.byref(a))
    assert run(lib, d, a, n=n, **{out: AT[of]}) == 1


def test_y_beside_its_residual(lib):
    d, a = descs()
    assert run(lib, d, a, y=AT["residual"] + 16) == 1
