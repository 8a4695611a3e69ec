"""Distillation at the ends of the temperature's range and with teacher entries near the ends of fp32: only an
entry of -inf itself is left out, and only differences to the row's largest count.  Bounds as in
tests/test_gpu_logits.py."""
import math

import pytest
import torch

from test_gpu_logits import IDS, TYPES, _check_distill, _close, _distill_ref, _gen, _teacher

pytestmark = pytest.mark.gpu

WIDTHS = [40, 700, 5000, 70000]   # a warp's row, blocks, blocks that share a row


@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("T", [1e-6, 1e-3, 1e3, 1e6])
def test_temperatures(cuda_lib, V, dtype, T):
    """Logits of the temperature's size, so that neither distribution is degenerate."""
    randn, _ = _gen(V)
    ids, top, w = _teacher(6, V, 5, V, repeat=True)
    _check_distill(cuda_lib, (randn(6, V) * 3 * T).to(dtype), ids, top * T, w, T, place=True)


@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("T", [1e-6, 0.5, 1.0, 1e6])
def test_entries_near_the_types_ends(cuda_lib, V, T):
    """Rows whose entries are all the lowest value (equal: uniform), the highest, the highest beside the lowest, and
    masks of the lowest beside ordinary ones: as rows of small entries with the same probabilities."""
    bl = cuda_lib
    randn, _ = _gen(V)
    low, high, far = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max, -1e4 * T
    rows = [([low] * 4, [0.0] * 4), ([high] * 4, [0.0] * 4), ([high, low, low, low], [0.0, far, far, far]), ([0.0, low, T, low], [0.0, far, T, far]),
            ([3e38, 1e38, 1e38, -math.inf], [0.0, far, far, -math.inf])]
    top, same = (torch.tensor([r[i] for r in rows], device="cuda") for i in range(2))
    n = len(rows)
    x = randn(n, V) * T
    ids, _, w = _teacher(n, V, 4, V)
    ref = _distill_ref(x, ids, same, w, T)
    loss, lse, d, d2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    bl.tern_distill(x, ids, top, loss, lse=lse, dlogits=d, weight=w, temperature=T)
    _close(loss, ref[0], ref[1], "loss")
    _close(d, ref[4], ref[5], "dlogits")
    bl.tern_distill(x, ids, same, loss, lse=lse, dlogits=d2, weight=w, temperature=T)
    assert torch.equal(d, d2)                                    # the same probabilities, bit for bit
    bl.tern_distill_bwd(x, ids, top, lse, d, weight=w, temperature=T)
    bl.tern_distill_bwd(x, ids, same, lse, d2, weight=w, temperature=T)
    assert torch.equal(d, d2)
