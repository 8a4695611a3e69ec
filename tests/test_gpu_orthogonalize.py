"""tern_orthogonalize against the definition in fp64, over square, wide, tall and ragged shapes.

Tolerance.  An error left in a direction of weak singular values grows by up to 3.4445 a step.  A
step's roundings are 2^-22 of an operand (two binary16 planes and the dropped lo*lo), and its fp32
sums of depth/16 tensor-core additions add up to depth/16 * 2^-24; both are relative to a spectral
norm of about 1, so tau = 3.4445^steps * (16 + depth/16) * 2^-24 bounds an element's error before
out is rounded to bf16 (2^-8 of it)."""
import numpy as np
import pytest
import torch

from _reference import check

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315


def _reference(G, steps=5, eps=1e-7, gain=1.0):
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / (torch.sqrt((X * X).sum()) + eps)
    for _ in range(steps):
        S = X @ X.T
        X = A * X + (B * S + C * (S @ S)) @ X
    return gain * (X.T if tall else X)


def _run(bl, G, steps=5, eps=1e-7, gain=1.0, out=None, stream=None):
    K, N = G.shape
    out = torch.full((K, N), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = torch.full((bl.tern_orthogonalize_workspace(K, N),), 0x7F, dtype=torch.uint8, device="cuda")
    bl.tern_orthogonalize(G, out, ws, steps=steps, eps=eps, gain=gain, stream=stream)
    return out


def _check(got, ref, steps=5, gain=1.0):
    depth = max(ref.shape)
    tau = A ** steps * (16 + depth / 16) * 2.0 ** -24 * abs(gain)
    r = ref.cpu().numpy()
    check("out", got.float().cpu().numpy(), r, np.abs(r) * 2.0 ** -8 * 1.01 + tau)


def _gradient(K, N, seed=0, scale=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = max(1, min(K, N) // 16)
    w = torch.arange(1, r + 1, device="cuda", dtype=torch.float32) ** -0.5
    low = (torch.randn(K, r, device="cuda", generator=g) * w) @ torch.randn(r, N, device="cuda", generator=g)
    return (low + 0.5 * torch.randn(K, N, device="cuda", generator=g)) * scale


SHAPES = [(1, 1), (1, 7), (9, 1), (8, 8), (16, 200), (200, 16), (33, 65), (65, 33), (129, 257), (300, 130), (512, 512),
          (384, 1000), (1000, 384), (77, 5000), (5000, 77)]


@pytest.mark.parametrize("K,N", SHAPES)
def test_orthogonalize_shapes(cuda_lib, K, N):
    G = _gradient(K, N, seed=K + N)
    _check(_run(cuda_lib, G, gain=0.7), _reference(G, gain=0.7), gain=0.7)
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


@pytest.mark.parametrize("K,N", [(1100, 4200), (4200, 1100), (1500, 1500), (2900, 3100), (3100, 2900)])
def test_orthogonalize_large_tiles(cuda_lib, K, N):
    """Sizes that take the larger tiles and the CTA pairs in each of the products."""
    G = _gradient(K, N, seed=K)
    _check(_run(cuda_lib, G), _reference(G))
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_orthogonalize_steps(cuda_lib, steps):
    G = _gradient(120, 200, seed=steps)
    _check(_run(cuda_lib, G, steps=steps), _reference(G, steps=steps), steps=steps)


@pytest.mark.parametrize("K,N", [(130, 8300), (8300, 130), (260, 4400), (1025, 2100), (900, 1300)])
@pytest.mark.parametrize("steps", [1, 2, 5])
def test_orthogonalize_long_sides(cuda_lib, K, N, steps):
    """Both sides of the rule by which steps are taken two at a time, whole pairs and a last single one."""
    G = _gradient(K, N, seed=K + steps)
    _check(_run(cuda_lib, G, steps=steps), _reference(G, steps=steps), steps=steps)
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


@pytest.mark.parametrize("N", [4500, 700])
def test_orthogonalize_keeps_weak_directions_of_long_sides(cuda_lib, N):
    """As below, with steps two at a time and one at a time."""
    g = torch.Generator(device="cuda").manual_seed(N)
    U = torch.linalg.qr(torch.randn(256, 256, device="cuda", generator=g, dtype=torch.float64))[0]
    V = torch.linalg.qr(torch.randn(N, 256, device="cuda", generator=g, dtype=torch.float64))[0]
    G = ((U * torch.logspace(0, -3, 256, device="cuda", dtype=torch.float64)) @ V.T).float()
    out, ref = _run(cuda_lib, G), _reference(G)
    _check(out, ref)
    assert (U[:, -64:].T @ (out.double() - ref)).norm() <= 2.0 ** -8 * ref.norm()


def test_orthogonalize_keeps_weak_directions(cuda_lib):
    """Singular values from 1 down to 1e-3 of the largest: the weak ones keep their directions."""
    g = torch.Generator(device="cuda").manual_seed(4)
    U = torch.linalg.qr(torch.randn(256, 256, device="cuda", generator=g, dtype=torch.float64))[0]
    V = torch.linalg.qr(torch.randn(640, 256, device="cuda", generator=g, dtype=torch.float64))[0]
    s = torch.logspace(0, -3, 256, device="cuda", dtype=torch.float64)
    G = ((U * s) @ V.T).float()
    out, ref = _run(cuda_lib, G), _reference(G)
    _check(out, ref)
    err = (out.double() - ref)
    weak = U[:, -64:].T @ err            # the error within the weak directions is rounding of out alone
    assert weak.norm() <= 2.0 ** -8 * ref.norm()


def test_orthogonalize_is_scale_free_and_repeatable(cuda_lib):
    G = _gradient(300, 700, seed=9)
    first = _run(cuda_lib, G, eps=1e-30)
    assert torch.equal(first, _run(cuda_lib, G, eps=1e-30))
    for k in (-60, 40):
        assert torch.equal(first, _run(cuda_lib, G * 2.0 ** k, eps=1e-30))
    _check(_run(cuda_lib, G.T.contiguous(), eps=1e-30).T, _reference(G))


def test_orthogonalize_special_values(cuda_lib):
    z = torch.zeros(40, 72, device="cuda")
    assert torch.all(_run(cuda_lib, z) == 0)
    for bad in (float("nan"), float("inf"), -float("inf")):
        G = _gradient(40, 72)
        G[3, 5] = bad
        assert torch.isnan(_run(cuda_lib, G)).all()
    one = torch.zeros(40, 72, device="cuda")
    one[7, 70] = -1e30                   # a single element: rank one, and far from the others' range
    out = _run(cuda_lib, one)
    _check(out, _reference(one))
    assert torch.count_nonzero(out) == 1
    tiny = torch.full((24, 24), 1e-38, device="cuda")
    _check(_run(cuda_lib, tiny, eps=1e-30), _reference(tiny, eps=1e-30))
    e = torch.empty(0, 5, device="cuda")
    cuda_lib.tern_orthogonalize(e, e.bfloat16(), None)


def test_orthogonalize_odd_addresses_stream_and_graph(cuda_lib):
    bl = cuda_lib
    K, N = 90, 136
    G = _gradient(K, N, seed=2)
    first = _run(bl, G)
    buf = torch.zeros(K * N + 1, device="cuda")
    Go = buf[1:].view(K, N)
    Go.copy_(G)
    oo = torch.zeros(K * N + 1, dtype=torch.bfloat16, device="cuda")[1:].view(K, N)
    assert torch.equal(_run(bl, Go, out=oo), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    ws = torch.empty(bl.tern_orthogonalize_workspace(K, N), dtype=torch.uint8, device="cuda")
    call = bl.Orthogonalize(G, out, ws)
    torch.cuda.synchronize()
    call(s)
    s.synchronize()
    assert torch.equal(out, first)
    out.fill_(0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_orthogonalize_refusals(cuda_lib):
    bl = cuda_lib
    G = torch.zeros(8, 16, device="cuda")
    out = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(bl.tern_orthogonalize_workspace(8, 16), dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError):
        bl.tern_orthogonalize(G.bfloat16(), out, ws)
    with pytest.raises(TypeError):
        bl.tern_orthogonalize(G, out.float(), ws)
    with pytest.raises(ValueError):
        bl.tern_orthogonalize(G.t().contiguous().t(), out, ws)
    with pytest.raises(ValueError):
        bl.tern_orthogonalize(G, out[:4], ws)
    for kw in (dict(steps=0), dict(steps=65), dict(eps=0.0), dict(eps=float("nan"))):
        with pytest.raises(bl.TernError) as e:
            bl.tern_orthogonalize(G, out, ws, **kw)
        assert e.value.status == bl.TERN_ERR_ARG
    for w in (None, ws[:-1]):
        with pytest.raises(bl.TernError) as e:
            bl.tern_orthogonalize(G, out, w)
        assert e.value.status == bl.TERN_ERR_WORKSPACE
    big = torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(bl.TernError) as e:
        bl.tern_orthogonalize(G, out, big[16:])
    assert e.value.status == bl.TERN_ERR_ALIGN
