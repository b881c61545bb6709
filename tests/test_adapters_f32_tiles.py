"""fp32 projections with adapters whose first step goes by tiles of 64 rows although the rows are few: high ranks."""
import pytest

from tests.test_adapters_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,rank", [(400, 256), (700, 256), (1100, 136), (1900, 64)])
@pytest.mark.parametrize("din,heads", [(36, 0), (640, 5), (1536, 0)])
def test_few_rows_of_high_rank(rows, rank, din, heads):
    """One adapter for all, and ragged segments with rows that have none; K in one slice and shared by a cluster."""
    for start, which in (([0, rows], [1]), ([3, rows // 4, rows // 4, rows // 2 + 1, rows - 1], [2, 1, -1, 0])):
        Case("f32", 2, rows // 2, din, 40, rank, start, which, heads=heads, act="silu", gated=True).check()
