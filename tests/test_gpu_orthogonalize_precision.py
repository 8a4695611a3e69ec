"""How precise tern_orthogonalize's products are, in the norm of the whole result, over every tile
shape, wide and tall: a bound that operands of one binary16 plane exceed.

The result is G's, rounded to bf16.  Rounding leaves the same error on the kernel's values as on the
fp64 ones, so what the arithmetic adds is the excess of |out - ref|^2 over |bf16(ref) - ref|^2.  Bound:
operands of two planes are good to 2^-22, grown by up to 3.4445 a step (2^-13 after five); the tensor
cores add 3 depth / 16 times into an fp32 accumulator and cut each sum towards zero, by half of 2^-23
on average, which lowers A and X by a factor, and a singular value moves by at most eight times that
over the steps (the quintic's derivative is below 3.5, and from 1/2 on below 1.5 in magnitude)."""
import pytest
import torch

from test_gpu_orthogonalize import A, B, C, _gradient, _reference, _run

pytestmark = pytest.mark.gpu


def arithmetic_bound(K, N, steps=5):
    return A ** min(steps, 5) * 2.0 ** -22 + 8 * (3 * max(K, N) / 16) * 2.0 ** -24


def excess(out, ref):
    size = ref.norm()
    both = ((out.double() - ref).norm() / size) ** 2 - ((ref.to(torch.bfloat16).double() - ref).norm() / size) ** 2
    return float(both.clamp(min=0).sqrt())


def _planes(x, scale, planes):
    """x rounded to that many binary16 planes at a scale."""
    hi = (x * scale).half()
    lo = ((x * scale) - hi.double()).half() if planes == 2 else torch.zeros_like(hi)
    return (hi.double() + lo.double()) / scale


def _emulated(G, planes, steps=5):
    """The steps in fp64, each matrix rounded once."""
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = _planes(X / (X.norm() + 1e-7), 16384, planes)
    eye = torch.eye(X.shape[0], dtype=torch.float64, device="cuda")
    for _ in range(steps):
        S = _planes(X @ X.T, 8192, planes)
        X = _planes(_planes(A * eye + B * S + C * (S @ S), 8192, planes) @ X, 16384, planes)
    return (X.T if tall else X).to(torch.bfloat16)


# single CTAs of 128 x 64 and clusters of 2, 4 and 8 of them; of 128 x 128; pairs of 256 x 256; steps one
# and two at a time
SHAPES = [(130, 8300), (8300, 130), (260, 4400), (4400, 260), (77, 5000), (5000, 77), (512, 512), (512, 2048), (2048, 512),
          (900, 1300), (1300, 900), (1025, 2100), (2100, 1025), (1100, 4200), (4200, 1100), (1500, 1500), (1500, 4000),
          (4000, 1500), (2049, 2049), (2560, 2816), (2816, 2560), (2900, 3100)]


@pytest.mark.parametrize("K,N", SHAPES)
def test_products_are_more_precise_than_one_plane(cuda_lib, K, N):
    G = _gradient(K, N, seed=K + 2 * N)
    ref, bound = _reference(G), arithmetic_bound(K, N)
    assert excess(_run(cuda_lib, G), ref) <= bound
    assert excess(_emulated(G, 2), ref) <= bound < excess(_emulated(G, 1), ref)


@pytest.mark.parametrize("K,N", [(640, 256), (700, 900), (900, 700), (1500, 1100), (1500, 1500), (1500, 4000), (4000, 1500), (2560, 2816),
                                 (2816, 2560)])
def test_weak_directions_in_every_tile(cuda_lib, K, N):
    """Singular values from 1 down to 1e-3 of the largest: within the weakest quarter of the directions
    the arithmetic adds less than 2^-10 to what rounding out leaves there (8.3e-4); one plane adds 2^-9."""
    m = min(K, N)
    g = torch.Generator(device="cuda").manual_seed(K + N)
    U = torch.linalg.qr(torch.randn(m, m, device="cuda", generator=g, dtype=torch.float64))[0]
    V = torch.linalg.qr(torch.randn(max(K, N), m, device="cuda", generator=g, dtype=torch.float64))[0]
    G = ((U * torch.logspace(0, -3, m, device="cuda", dtype=torch.float64)) @ V.T).float()
    if K > N:
        G = G.T.contiguous()
    ref = _reference(G)

    def weak(out):
        err = out.double() - ref
        return ((U[:, -(m // 4):].T @ err if K <= N else err @ U[:, -(m // 4):]).norm() / ref.norm()) ** 2

    rounding = weak(ref.to(torch.bfloat16))
    assert weak(_run(cuda_lib, G)) <= rounding + 2.0 ** -20 < weak(_emulated(G, 1))
