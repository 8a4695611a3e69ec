"""Where tern_orthogonalize takes its steps two at a time, by the workspace that this asks for (two more
matrices of the smaller side, of two planes): not where the products saved are fewer than those added."""
import pytest


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._builder().build()
    import bit_linear_gb300 as bl
    return bl


def _matrices(lib, K, N):
    """The matrices of the smaller side in the workspace (each rounded up, beside two X and some bytes)."""
    up = lambda x, to: (x + to - 1) // to * to  # noqa: E731
    m = min(K, N)
    x, a = 4 * up(K * up(N, 8) * 2, 256), 2 * up(m * up(m, 8) * 2, 256)
    return (lib.tern_orthogonalize_workspace(K, N) - x) // a


@pytest.mark.parametrize("K,N", [(512, 2600), (600, 2400), (4096, 5000), (12288, 4096), (1024, 1536), (1800, 1024), (1200, 2100)])
def test_pairs(lib, K, N):
    assert _matrices(lib, K, N) == 4


@pytest.mark.parametrize("K,N", [(512, 2048), (1000, 1530), (1023, 1600), (1025, 1600), (1100, 1650), (1900, 1100), (1152, 1728), (1280, 1920),
                                 (1250, 1900), (2048, 2048), (3000, 3180)])
def test_single_steps(lib, K, N):
    assert _matrices(lib, K, N) == 2
