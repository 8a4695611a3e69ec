"""Layer norm and the gated feed-forward layer over more than 2^32 elements: the first and the last rows against
the formulas in fp64.  Bounds as in tests/test_gpu_norm.py and tests/test_gpu_glu.py."""
import pytest
import torch

import test_gpu_glu as glu
import test_gpu_norm as norm

pytestmark = pytest.mark.gpu


def _fill(t):
    for i, part in enumerate(t.split(1 << 17)):
        part.normal_(generator=torch.Generator(device="cuda").manual_seed(i))
    return t


@pytest.mark.parametrize("n,D", [(1050001, 4096), (1050001, 4095), (220001, 20000)])
def test_norm(cuda_lib, n, D):
    assert n * D > 1 << 32
    bl = cuda_lib
    x, dy = (_fill(torch.empty(n, D, dtype=torch.bfloat16, device="cuda")) for _ in range(2))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    w, b = 1 + 0.3 * torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    mean, rstd, dw, db = (torch.empty(k, device="cuda") for k in (n, n, D, D))
    ws = torch.empty(bl.tern_norm_bwd_workspace(n, D), dtype=torch.uint8, device="cuda")
    bl.tern_norm_fwd(x, y, weight=w, bias=b, mean=mean, rstd=rstd)
    bl.tern_norm_bwd(x, dy, mean, rstd, dx, ws, weight=w, dweight=dw, dbias=db)
    for r in (slice(0, 3), slice(n - 3, n)):
        refs = norm._ref(x[r], w, b, 1e-5, dy[r])
        for got, ref, name in zip((y, mean, rstd, dx), refs, norm.NAMES):
            norm._near(got[r], ref, name)
    # a column's sum: at most ceil(n / 152) = 6908 rows one after another (rows beside one another, runs and
    # parts of wide rows make it less), and 128 more to join them
    total, size = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for part in dy.split(1 << 14):
        total += part.double().sum(0)
        size += part.double().abs().sum(0)
    assert torch.all((db.double() - total).abs() <= (6908 + 128) * norm.U * size)


def test_gated_layer(cuda_lib):
    bl = cuda_lib
    M, K, N = 700001, 16, 3200
    assert 2 * M * N > 1 << 32
    _, q, scale, _ = glu._inputs(1, K, N, 5)
    tiles = glu._tiles(bl, q, scale)
    X = _fill(torch.empty(M, K, dtype=torch.bfloat16, device="cuda"))
    dH = _fill(torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
    H, pair, dY = (torch.empty(M, k, dtype=torch.bfloat16, device="cuda") for k in (N, 2 * N, 2 * N))
    bl.tern_glu_fwd(X, tiles, scale, H, saved=pair)
    bl.tern_glu_bwd(dH, dY, X=X, tiles=tiles, scale=scale)
    rows = [slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)]
    for r in rows:
        h, fg, fu = glu._ref(X[r], q, scale, "silu")
        d = dH[r].double()
        glu._near(H[r], *h, 1, "H")
        glu._near(pair[r, :N], *fg, 1, "factor of dG")
        glu._near(pair[r, N:], *fu, 1, "factor of dU")
        glu._near(dY[r, :N], fg[0] * d, fg[1] * d.abs(), 1, "dG")
        glu._near(dY[r, N:], fu[0] * d, fu[1] * d.abs(), 1, "dU")
    bl.tern_glu_bwd(dH, dY, saved=pair)
    for r in rows:
        assert torch.equal(dY[r, :N], (dH[r].float() * pair[r, :N].float()).bfloat16())
        assert torch.equal(dY[r, N:], (dH[r].float() * pair[r, N:].float()).bfloat16())
    assert bl.tern_device_status() == bl.TERN_OK
