"""tern_orthogonalize where the gradient's norm is far below eps, so that G / (|G|_F + eps) starts far
below 1: every step multiplies such values by up to 3.4445, until they reach the rest of the quintic.

Tolerance, in the norm of the whole result: rounding out to bf16 leaves what rounding the fp64 result
leaves; the arithmetic adds at most `arithmetic_bound` of test_gpu_orthogonalize_precision."""
import pytest
import torch

from test_gpu_orthogonalize import _gradient, _reference, _run
from test_gpu_orthogonalize_precision import arithmetic_bound, excess

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N", [(1, 1), (1, 9), (40, 72), (72, 40), (200, 530), (1024, 1600), (130, 8300), (8300, 130), (1500, 1500)])
@pytest.mark.parametrize("steps", [1, 2, 5, 11])
def test_norms_far_below_eps(cuda_lib, K, N, steps):
    G = _gradient(K, N, seed=K + steps)
    G /= G.double().norm().float()
    # |G|_F and eps: ratios of 1/2 down to 2^-90, the smallest with norms near the end of fp32's range
    for norm, eps in ((1.0, 1.0), (1e-7, 1e-7), (1e-10, 1e-7), (1e-14, 1e-7), (1e-16, 1e-7), (1.0, 1e9), (1e-20, 1e-7), (1e-27, 1.0)):
        H = G * norm
        # the gain keeps the result in bf16's range
        gain = float(min(max(1.0, eps / norm), 1e30))
        out, ref = _run(cuda_lib, H, steps=steps, eps=eps, gain=gain), _reference(H, steps=steps, eps=float(torch.tensor(eps)), gain=gain)
        assert excess(out, ref) <= arithmetic_bound(K, N, steps), (norm, eps)
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


def test_results_below_the_range_are_zeros(cuda_lib):
    G = _gradient(40, 72)
    out = _run(cuda_lib, G * 1e-33, eps=1e30)
    assert torch.all(out == 0)
    z = _run(cuda_lib, torch.zeros(40, 72, device="cuda"), eps=1e30, steps=64)
    assert torch.all(z == 0)
    for bad in (float("nan"), float("inf")):
        G[2, 3] = bad
        assert torch.isnan(_run(cuda_lib, G, eps=1e9)).all()


def test_growth_through_many_steps(cuda_lib):
    """From 2^-40 of the largest value up to the quintic's fixed range, and on: finite, and near 1."""
    G = _gradient(64, 160, seed=3)
    G = (G / G.double().norm().float()) * 2.0 ** -40
    for steps in (20, 26, 40, 64):
        out, ref = _run(cuda_lib, G, steps=steps, eps=1.0), _reference(G, steps=steps, eps=1.0)
        s, r = torch.linalg.svdvals(out.double()), torch.linalg.svdvals(ref)
        assert s.max() <= 1.21 + 2.0 ** -6 and abs(s.max() - r.max()) <= 2.0 ** -6 + 0.6 * (steps > 26)
