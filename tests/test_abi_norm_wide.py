"""Workspace of the layer norm's gradient for rows of more than 16384 channels, without a GPU: one value a
row, and from 129 rows on the sums of at most 608 parts of the rows for weight and bias."""
import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._builder().build()
    import bit_linear_gb300 as bl
    return bl


@pytest.mark.parametrize("n,parts", [(1, 0), (128, 0), (129, 2), (256, 2), (257, 3), (608 * 128, 608), (608 * 128 + 1, 608), ((1 << 31) - 2049, 608)])
@pytest.mark.parametrize("D", [16385, 20002, 1 << 22])
def test_workspace(lib, n, parts, D):
    assert lib.tern_norm_bwd_workspace(n, D) == 4 * (n + 2 * parts * D)
