"""Workspace of a table's gradient without a GPU: every part that the kernels use has its bytes."""
import pytest

from quantized_weight_out_gb300 import binding as rg
from quantized_weight_out_gb300 import build as rgbuild


@pytest.fixture(scope="module")
def lib():
    rgbuild.build()
    return rg.load()


def up(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("N,pairs", [(1, 0), (1023, 0), (1024, 1), (32000, 1), ((1 << 20) - 1, 1), (1 << 20, 2),
                                     ((1 << 31) - 1, 2)])
@pytest.mark.parametrize("n", [1, 32, 33, 4097, 1 << 20])
@pytest.mark.parametrize("K", [8, 64, 4104])
def test_rows_back_workspace(lib, N, pairs, n, K):
    """The order and the sorted ids, two pieces of F32 rows a window of 32 ids, and what lies between the sort's passes:
    pairs of 8 bytes, once for two passes, twice for more (ids of N and one more take 10 bits a pass)."""
    windows = -(-n // 32)
    want = 2 * up(4 * n) + 2 * up(4 * windows * K) + pairs * up(8 * n)
    assert rg.rg_get_rows_back_workspace_bytes(n, N, K) == want
