"""tern_orthogonalize where the norm or eps is infinite or at the ends of its range."""
import pytest
import torch

from test_gpu_orthogonalize import _gradient, _reference, _run

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("K,N", [(40, 72), (1024, 1600)])
def test_an_infinite_eps_gives_zeros_and_an_infinite_gradient_nan(cuda_lib, K, N):
    G = _gradient(K, N)
    assert torch.all(_run(cuda_lib, G, eps=INF) == 0)
    G[3, 4] = INF
    for eps in (1e-30, 1e-7, 1.0, 3e38):
        assert torch.isnan(_run(cuda_lib, G, eps=eps)).all(), eps
    assert torch.isnan(_run(cuda_lib, G, eps=INF)).all()
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


@pytest.mark.parametrize("value,eps", [(3e38, 1e-30), (3e38, 3e38), (1e-38, 1e-30), (1e-45, 1e-30), (1e-45, 3e38)])
def test_a_single_value_of_any_size(cuda_lib, value, eps):
    """Rank one: the quintic of |G| / (|G| + eps), to a bf16 step."""
    G = torch.zeros(24, 40, device="cuda")
    G[5, 7] = value
    out, ref = _run(cuda_lib, G, eps=eps), _reference(G, eps=float(torch.tensor(eps)))
    assert torch.count_nonzero(out) <= 1
    assert abs(out[5, 7].double() - ref[5, 7]) <= abs(ref[5, 7]) * 2.0 ** -8 + 2.0 ** -133
