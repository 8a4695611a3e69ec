"""Packed documents stay apart in both directions: whatever a NaN or an infinity does to its own
document, the others' outputs and gradients keep their bits."""
import numpy as np
import pytest
import torch

from test_gpu_scan import Case

pytestmark = pytest.mark.gpu

# blocks of four warps without a cluster, clusters of eight-warp blocks, narrow tiles in clusters of 16,
# odd widths: all the shapes that a step's rows are joined in
SHAPES = [(330, 300, 32), (3, 700, 64), (1, 3000, 64), (2, 600, 35)]


def _check(bl, B, T, D, dtype, name, bad, first, second, at):
    """`bad` at row `at` of one document, rows first..second-1, of the middle of three (None: at all of its rows); everything outside keeps its bits."""
    starts = np.zeros((B, T), bool)
    starts[:, first] = starts[:, second] = True
    clean = Case(bl, B, T, D, dtype, 21, starts=starts).run()
    case = Case(bl, B, T, D, dtype, 21, starts=starts)
    getattr(case, name)[:, first if at is None else at:second if at is None else at + 1] = bad
    case.run()
    for k in ("y", "df", "dv", "dr"):
        got, ref = getattr(case, k), getattr(clean, k)
        assert torch.equal(got[:, :first], ref[:, :first]), (k, "before", first, at)
        assert torch.equal(got[:, second:], ref[:, second:]), (k, "after", second, at)
    assert torch.equal(case.dh0, clean.dh0) and torch.equal(case.hT, clean.hT), (first, second, at)


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", ["f", "v", "r", "dy"])
def test_a_nan_stays_in_its_document(cuda_lib, B, T, D, dtype, name):
    """The row is in the segment of its document's start, and segments, warps, blocks and steps after it."""
    for first, second, at in ((33, T - 20, 33), (33, T - 20, 34), (33, T - 20, 40), (33, T - 20, 75), (33, T - 20, T - 21),
                              (T // 2 - 1, T - 1, T // 2), (1, T // 2, T // 2 - 1), (64, 65, 64), (33, T - 20, None), (100, T // 2, None)):
        _check(cuda_lib, B, T, D, dtype, name, float("nan"), first, second, at)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["v", "r", "dy"])
def test_an_infinity_stays_in_its_document(cuda_lib, name, bad):
    for B, T, D in SHAPES[1:3]:
        for first, second, at in ((33, T - 20, 40), (33, T - 20, T - 21)):
            _check(cuda_lib, B, T, D, torch.float32, name, bad, first, second, at)


def test_a_nan_gate_and_padding(cuda_lib):
    """The same beside uneven lengths: the document of the NaN ends in padding."""
    B, T, D = 4, 500, 64
    starts = np.zeros((B, T), bool)
    starts[:, 100] = True
    lengths = [101, 150, 333, 500]
    clean = Case(cuda_lib, B, T, D, torch.float32, 22, lengths=lengths, starts=starts).run()
    case = Case(cuda_lib, B, T, D, torch.float32, 22, lengths=lengths, starts=starts)
    for b, n in enumerate(lengths):
        case.f[b, n - 1] = float("nan")
    case.run()
    for k in ("y", "df", "dv", "dr"):
        assert torch.equal(getattr(case, k)[:, :100], getattr(clean, k)[:, :100]), k
    assert torch.equal(case.dh0, clean.dh0)
