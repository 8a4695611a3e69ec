"""The layer norm's gradient of rows of more than 16384 channels, over many rows: the sums of a column are
of bounded runs of rows.

Bound of a column's sum, u = 2^-24: a run adds at most 128 rows, a block of them ceil(n / 608 / 128) runs (one
here), and the blocks' sums, at most 608, are added by ceil(608 / 32) = 19 in a lane, 5 steps over lanes and 5
over warps: under 160 u of the sum of magnitudes (of n rows one after another up to n u: 4096 u here)."""
import pytest
import torch

from test_gpu_norm import IDS, NAMES, TYPES, U, _near, _ref, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,D", [(128, 16400), (129, 16385), (300, 20002), (4096, 16385)])
@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
def test_sums_of_one_sign(cuda_lib, n, D, tx, ty):
    """dy of one sign, nearly the same down a column: what a long sum rounds away has one sign too."""
    g = torch.Generator(device="cuda").manual_seed(n + D)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = (r(1, D) + 0.01 * r(n, 1)).to(tx)
    dy = (0.1 + 0.05 * torch.rand(1, D, device="cuda", generator=g) + 0.001 * torch.rand(n, 1, device="cuda", generator=g)).to(ty)
    w, b = 1 + 0.3 * r(D), 0.5 * r(D)
    got, refs = _run(cuda_lib, x, w, b, dy), _ref(x, w, b, 1e-5, dy)
    for i, name in enumerate(NAMES):
        val, tol = refs[i]
        if name == "dbias":
            tol = 160 * U * dy.double().abs().sum(0)
        elif name == "dweight":
            xhat = (x.double() - x.double().mean(1, keepdim=True)) * refs[2][0][:, None]
            tol = tol + 32 * U * (dy.double() * xhat).abs().sum(0)      # 160 for the 128 that it has
        _near(got[i], (val, tol), name)
    assert all(torch.equal(p, q) for p, q in zip(got, _run(cuda_lib, x, w, b, dy)))


def test_strided_rows_and_one_sum(cuda_lib):
    """Rows between NaN, and each of the sums alone: the same bits, nothing else written."""
    bl = cuda_lib
    n, D = 700, 16387
    g = torch.Generator(device="cuda").manual_seed(7)
    x, dy = (torch.randn(n, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    w, b = torch.rand(D, device="cuda", generator=g), torch.zeros(D, device="cuda")
    want = _run(bl, x, w, b, dy)
    wide = [torch.full((n, D + 5), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    wide[0][:, :D], wide[1][:, :D] = x, dy
    got = _run(bl, wide[0][:, :D], w, b, wide[1][:, :D], dx=wide[2][:, :D])
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and wide[2][:, D:].isnan().all()
    need = bl.tern_norm_bwd_workspace(n, D)
    for k in range(2):
        sums, dx = [None, None], torch.empty_like(x)
        sums[k] = torch.full((D,), 9.0, device="cuda")
        ws = torch.full((need + 64,), 77, dtype=torch.uint8, device="cuda")
        bl.tern_norm_bwd(x, dy, want[1], want[2], dx, ws[:need], weight=w, dweight=sums[0], dbias=sums[1])
        assert torch.equal(sums[k], want[4 + k]) and torch.equal(dx, want[3]) and torch.all(ws[need:] == 77)
