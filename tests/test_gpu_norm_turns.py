"""Layer norm over so many rows that every group of threads takes four turns or more: the rings that rows are
copied through are refilled within the loop, and their places used again.

The bounds are those of single rows (tests/test_gpu_norm.py).  Their terms, of the kernels that run here: a
sum over a row adds at most 32 terms in a thread, 5 over lanes and 16 over warps, under 64; a column's sum
at most 2 ceil(n / (2 152 R)) = 14 rows in a group of threads, 2 over lanes, R <= 16 groups beside one
another (a warp's rows joined), and the blocks' sums by 5 in a lane, 5 over lanes and 5 over warps: 47, under 128."""
import pytest
import torch

from test_gpu_norm import IDS, NAMES, TYPES, _inputs, _near, _ref, _run

pytestmark = pytest.mark.gpu


def _row_threads(D):
    t = 8
    while t * 16 < D:
        t *= 2
    return t


def _check(bl, n, D, tx, ty):
    x, w, b, dy = _inputs(n, D, tx, ty, n + D)
    got, refs = _run(bl, x, w, b, dy), _ref(x, w, b, 1e-5, dy)
    for g, ref, name in zip(got, refs, NAMES):
        _near(g, ref, name)
    assert all(torch.equal(p, q) for p, q in zip(got, _run(bl, x, w, b, dy)))


@pytest.mark.parametrize("n,D", [(60001, 64), (20001, 512), (10001, 1024), (5203, 2048), (2603, 4096), (1301, 8192),
                                 (60001, 62), (10001, 1022), (2603, 4094), (1301, 8190)])
@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
def test_gradient(cuda_lib, n, D, tx, ty):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # pairs of rows that the GPU takes at a time: at most 512 threads an SM
    assert n > 3 * 2 * sms * 512 // _row_threads(D)
    _check(cuda_lib, n, D, tx, ty)


@pytest.mark.parametrize("n,D", [(120001, 64), (60001, 256), (40001, 512), (13001, 1024), (9001, 2048), (4001, 4096)])
def test_forward(cuda_lib, n, D):
    """bf16 to bf16, whose forward takes pairs of rows: so many blocks of an SM by the threads of a row."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = _row_threads(D)
    blocks = {64: 10, 256: 3}.get(T, 6)
    assert n > 3 * 2 * sms * blocks * max(1, 128 // T if T <= 32 else 1)
    _check(cuda_lib, n, D, torch.bfloat16, torch.bfloat16)
