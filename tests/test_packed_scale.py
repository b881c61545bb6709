"""mcs_packed_attn refuses a scale that leaves fp32's range in the units the kernels take (CPU only)."""
import ctypes

import pytest

from tests.test_packed_refusals import desc, lib, run  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_scale_times_log2_e(lib, scale):  # noqa: F811
    """Scores are taken in powers of two: scale * 1.4427 has to be finite, or scores of 0 were NaN."""
    assert lib.mcs_packed_attn_workspace_size(ctypes.byref(desc(scale=scale))) == 0
    assert run(lib, desc(scale=scale)) == 1


def test_largest_scale(lib):  # noqa: F811
    assert lib.mcs_packed_attn_workspace_size(ctypes.byref(desc(scale=2.35e38))) > 0
