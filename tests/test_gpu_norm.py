"""Layer norm and its gradient on the GPU against the formulas in fp64.

Bounds, with u = 2^-24 (half a step of fp32) and h the half step of the output's type: a sum over a row
adds at most 16 terms in a thread (D / 1024 in the widest rows), 5 in a warp and 32 over warps, so it is off by less than 64 u
times the sum of magnitudes; xhat by the roundings of x - mean and rstd (whose variance has such a sum)
and by delta's sum; the mean by its rounding and delta's sum, or by a delta of at most 16 u deviations.  Sums over rows add at most ceil(n / 608) rows a block, 4 side by side, and 38 + 16
blocks: under 128 for the sizes here."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)]
IDS = ["bf16-bf16", "f32-bf16", "bf16-f32", "f32-f32"]


def _ref(x, w, b, eps, dy=None):
    """y, mean, rstd and, with dy, dx, dw, db in fp64, each with its bound (without the output's rounding)."""
    x, w, b = x.double(), w.double(), b.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / (d.square().mean(1, keepdim=True) + eps).sqrt()
    xhat = d * rstd
    md = d.abs().mean(1, keepdim=True)
    off = U * (80 * xhat.abs() + 64 * md * rstd)
    y = xhat * w + b
    out = [(y, w.abs() * off + 2 * U * (y.abs() + (w * xhat).abs())), (mean[:, 0], (U * (mean.abs() + 64 * md + 16 / rstd))[:, 0]), (rstd[:, 0], 40 * U * rstd[:, 0])]
    if dy is None:
        return out
    dy = dy.double()
    g = dy * w
    mg, mgx = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    ag, agx = g.abs().mean(1, keepdim=True), (g * xhat).abs().mean(1, keepdim=True)
    dx = rstd * (g - mg - xhat * mgx)
    tol = rstd * U * (48 * (g.abs() + mg.abs() + (xhat * mgx).abs()) + 64 * ag + 130 * xhat.abs() * agx) + off * rstd * mgx.abs() + rstd * xhat.abs() * (off * g.abs()).mean(1, keepdim=True)
    out += [(dx, tol), ((dy * xhat).sum(0), (dy.abs() * (128 * U * xhat.abs() + off)).sum(0)), (dy.sum(0), 128 * U * dy.abs().sum(0))]
    return out


def _near(got, ref, name):
    val, tol = ref
    err = (got.double() - val).abs()
    bound = tol + HALF[got.dtype] * (val.abs() + tol)
    assert torch.all(err <= bound), (name, float((err - bound).max()))


def _inputs(n, D, tx, ty, seed, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return (r(n, D) * (0.2 + 3 * torch.rand(n, 1, device="cuda", generator=g)) + shift).to(tx), 1 + 0.3 * r(D), 0.5 * r(D), (0.1 * r(n, D)).to(ty)


# Enough rows for the kernels that take pairs of them, odd counts and uneven ends among them; sums over up to
# 14 rows a block in turn, 16 side by side, then 19 and 32: under 128 too
@pytest.mark.parametrize("n,D", [(9999, 8), (9999, 2), (6001, 62), (6001, 64), (5001, 130), (2601, 254), (1300, 510), (2605, 602), (703, 1030), (702, 2058), (401, 4102), (5001, 128), (5003, 136), (2600, 256), (2501, 264), (1303, 512), (700, 520), (2611, 600), (2600, 1024), (611, 1032), (402, 2048), (705, 2056),
                                 (403, 4096), (350, 4104), (309, 8192), (320, 8200)])
@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
def test_many_rows(cuda_lib, n, D, tx, ty):
    x, w, b, dy = _inputs(n, D, tx, ty, n + D)
    got, refs = _run(cuda_lib, x, w, b, dy), _ref(x, w, b, 1e-5, dy)
    for g, ref, name in zip(got, refs, NAMES):
        _near(g, ref, name)
    assert all(torch.equal(p, q) for p, q in zip(got, _run(cuda_lib, x, w, b, dy)))
    # strided, with NaN between the rows; nothing else written
    wide = torch.full((n, D + 8), float("nan"), dtype=tx, device="cuda")
    wide[:, :D] = x
    dx = torch.full((n, D + 8), 5.0, dtype=tx, device="cuda")
    again = _run(cuda_lib, wide[:, :D], w, b, dy, dx=dx[:, :D])
    assert all(torch.equal(p, q) for p, q in zip(got, again)) and torch.all(dx[:, D:] == 5.0)


def _run(bl, x, w, b, dy, eps=1e-5, y=None, dx=None):
    n, D = x.shape
    f32 = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    y = torch.full((n, D), float("nan"), dtype=dy.dtype, device="cuda") if y is None else y
    dx = torch.full((n, D), float("nan"), dtype=x.dtype, device="cuda") if dx is None else dx
    mean, rstd, dw, db = f32(n), f32(n), f32(D), f32(D)
    ws = f32(bl.tern_norm_bwd_workspace(n, D) // 4)
    bl.tern_norm_fwd(x, y, weight=w, bias=b, eps=eps, mean=mean, rstd=rstd)
    bl.tern_norm_bwd(x, dy, mean, rstd, dx, ws, weight=w, dweight=dw, dbias=db)
    return y, mean, rstd, dx, dw, db


NAMES = ("y", "mean", "rstd", "dx", "dweight", "dbias")


@pytest.mark.parametrize("n,D", [(7001, 63), (6501, 127), (3501, 255), (6301, 301), (3201, 515), (1601, 2047), (640, 4097), (333, 8191), (1601, 2046), (333, 8190)])
@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
def test_many_rows_off_words(cuda_lib, n, D, tx, ty):
    """More rows than the forward's blocks that stay, of widths that no 16-byte words hold."""
    x, w, b, dy = _inputs(n, D, tx, ty, n + D)
    got, refs = _run(cuda_lib, x, w, b, dy), _ref(x, w, b, 1e-5, dy)
    for g, ref, name in zip(got, refs, NAMES):
        _near(g, ref, name)
    assert all(torch.equal(p, q) for p, q in zip(got, _run(cuda_lib, x, w, b, dy)))


@pytest.mark.parametrize("n,D", [(15001, 136), (7501, 264), (7401, 508), (3703, 520), (1901, 1032), (1001, 2056), (501, 4104), (501, 8192)])
@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
def test_more_rows_than_fit(cuda_lib, n, D, tx, ty):
    """More rows than are resident with 16 elements a thread: the forward gives each 32."""
    x, w, b, dy = _inputs(n, D, tx, ty, n + D)
    got, refs = _run(cuda_lib, x, w, b, dy), _ref(x, w, b, 1e-5, dy)
    for g, ref, name in zip(got, refs, NAMES):
        _near(g, ref, name)
    assert all(torch.equal(p, q) for p, q in zip(got, _run(cuda_lib, x, w, b, dy)))


@pytest.mark.parametrize("n,D", [(1, 1), (1, 512), (3, 2), (5, 31), (7, 32), (2500, 64), (9, 511), (33, 512), (10, 513), (4, 1000), (700, 2048),
                                 (6, 2049), (5, 4096), (3, 4100), (2, 8191), (3, 8200), (2, 16384), (2, 16385), (3, 20002)])
@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
def test_norm_and_gradient(cuda_lib, n, D, tx, ty):
    x, w, b, dy = _inputs(n, D, tx, ty, n * 7 + D)
    for got, ref, name in zip(_run(cuda_lib, x, w, b, dy), _ref(x, w, b, 1e-5, dy), NAMES):
        _near(got, ref, name)


@pytest.mark.parametrize("D", [64, 512, 2049, 4096, 20000])
def test_rows_far_from_zero(cuda_lib, D):
    """A mean of 3000 with a spread near 1: what the rounded mean leaves must not reach the results."""
    x, w, b, dy = _inputs(5, D, torch.float32, torch.float32, D, shift=3000.0)
    for got, ref, name in zip(_run(cuda_lib, x, w, b, dy), _ref(x, w, b, 1e-5, dy), NAMES):
        _near(got, ref, name)


@pytest.mark.parametrize("D", [1, 7, 8, 64, 513, 1026])
@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
def test_rows_at_every_address(cuda_lib, D, tx, ty):
    """Rows that start at every element of a 16-byte word, strided, with NaN around them: the aligned call's
    bits in y, and nothing else written."""
    n = 9
    x0, w, b, dy0 = _inputs(n, D, tx, ty, D)
    refs = _ref(x0, w, b, 1e-5, dy0)
    for off in range(8):
        ld = D + (0, 3, 8)[off % 3]
        place = lambda dt, src=None: torch.full((n * ld + 9,), float("nan"), dtype=dt, device="cuda")  # noqa: E731
        bufs = [place(t) for t in (tx, ty, ty, tx)]
        x, dy, y, dx = (t[off:off + n * ld].as_strided((n, D), (ld, 1), off) for t in bufs)
        x.copy_(x0), dy.copy_(dy0)
        for got, ref, name in zip(_run(cuda_lib, x, w, b, dy, y=y, dx=dx), refs, NAMES):
            _near(got, ref, name)
        assert all(int(t.isnan().sum()) == t.numel() - n * D for t in bufs[2:])


def test_parts_of_the_call(cuda_lib):
    bl = cuda_lib
    x, w, b, dy = _inputs(50, 300, torch.float32, torch.bfloat16, 3)
    y, mean, rstd, dx, dw, db = _run(bl, x, w, b, dy)
    plain = torch.empty_like(y)
    bl.tern_norm_fwd(x, plain)                                    # neither weight nor bias, nothing kept
    one, zero = torch.ones(300, device="cuda"), torch.zeros(300, device="cuda")
    _near(plain, _ref(x, one, zero, 1e-5)[0], "y")
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    bl.tern_norm_bwd(x, dy, mean, rstd, dx2, weight=w)            # no sums, no workspace
    assert torch.equal(dx2, dx)
    ws = torch.empty(bl.tern_norm_bwd_workspace(50, 300), dtype=torch.uint8, device="cuda")
    bl.tern_norm_bwd(x, dy, mean, rstd, dx2, ws, weight=w, dweight=dw2)
    bl.tern_norm_bwd(x, dy, mean, rstd, dx2, ws, weight=w, dbias=db2)
    assert torch.equal(dw2, dw) and torch.equal(db2, db)
    for D in (300, 20000):                                        # sums over no rows are zeros
        e, dwe, dbe = torch.empty(0, D, device="cuda"), torch.full((D,), 7.0, device="cuda"), torch.full((D,), 7.0, device="cuda")
        v = torch.empty(0, device="cuda")
        bl.tern_norm_fwd(e, torch.empty_like(e))
        bl.tern_norm_bwd(e, e, v, v, torch.empty_like(e), None, dweight=dwe, dbias=dbe)
        assert not dwe.any() and not dbe.any()


@pytest.mark.parametrize("n,D", [(3000, 64), (5000, 1024), (40, 20000)])
def test_same_bits_every_time(cuda_lib, n, D):
    x, w, b, dy = _inputs(n, D, torch.bfloat16, torch.bfloat16, 1)
    first = _run(cuda_lib, x, w, b, dy)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, _run(cuda_lib, x, w, b, dy)))


def test_rows_that_are_not_finite_or_constant(cuda_lib):
    """NaN and infinities stay in their rows; constant rows give the bias and the gradient's finite values."""
    x, w, b, dy = _inputs(6, 700, torch.float32, torch.float32, 5)
    x[1, 3], x[2, 4], x[4] = float("nan"), float("inf"), 2.5
    y, mean, rstd, dx, _, db = _run(cuda_lib, x, w, b, dy)
    for r in (1, 2):
        assert y[r].isnan().all() and dx[r].isnan().all() and rstd[r].isnan()
    keep = [0, 3, 4, 5]
    refs = _ref(x[keep], w, b, 1e-5, dy[keep])
    for got, ref, name in ((y[keep], refs[0], "y"), (mean[keep], refs[1], "mean"), (rstd[keep], refs[2], "rstd"), (dx[keep], refs[3], "dx")):
        _near(got, ref, name)
    assert torch.allclose(y[4], b, rtol=0, atol=0)


def test_gradient_against_differences(cuda_lib):
    """dx, dweight and dbias against differences of sum(dy y) of the forward's definition in fp64."""
    x, w, b, dy = _inputs(3, 40, torch.float32, torch.float32, 11)
    _, _, _, dx, dw, db = _run(cuda_lib, x, w, b, dy)
    loss = lambda x, w, b: float((dy.double() * _ref(x, w, b, 1e-5)[0][0]).sum())  # noqa: E731
    g, args, eps = torch.Generator().manual_seed(2), [x.double(), w.double(), b.double()], 1e-4
    for i, d in enumerate((dx, dw, db)):
        for _ in range(4):
            v = torch.randn(args[i].shape, generator=g, dtype=torch.float64).cuda()
            at = lambda s: loss(*[a + s * eps * v if k == i else a for k, a in enumerate(args)])  # noqa: E731
            diff, mag = (at(1) - at(-1)) / (2 * eps), float((v * d.double()).abs().sum())
            # the differences' third-order term at steps of 1e-4 of the spread, beside fp32's roundings
            assert abs(diff - float((v * d.double()).sum())) <= 1e-5 * mag


def test_streams_and_graphs(cuda_lib):
    bl = cuda_lib
    x, w, b, dy = _inputs(600, 512, torch.bfloat16, torch.bfloat16, 8)
    want = _run(bl, x, w, b, dy)
    n, D = x.shape
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    mean, rstd, dw, db = (torch.empty(k, device="cuda") for k in (n, n, D, D))
    fwd = bl.NormForward(x, y, w, b, mean=mean, rstd=rstd)
    bwd = bl.NormBackward(x, dy, mean, rstd, dx, torch.empty(bl.tern_norm_bwd_workspace(n, D), dtype=torch.uint8, device="cuda"), w, dw, db)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        fwd()
        bwd()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, (y, mean, rstd, dx, dw, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd()
        bwd()
    x2, _, _, dy2 = _inputs(600, 512, torch.bfloat16, torch.bfloat16, 9)
    want = _run(bl, x2, w, b, dy2)
    x.copy_(x2), dy.copy_(dy2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, (y, mean, rstd, dx, dw, db)))


def test_refusals(cuda_lib):
    bl = cuda_lib
    x, y = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    with pytest.raises(TypeError):
        bl.tern_norm_fwd(x.half(), y)
    with pytest.raises(TypeError):
        bl.tern_norm_fwd(x.cpu(), y)
    with pytest.raises(ValueError):
        bl.tern_norm_fwd(x, y[:3])
    with pytest.raises(ValueError):
        bl.tern_norm_fwd(x.t().contiguous().t(), y)
    with pytest.raises(ValueError):
        bl.tern_norm_fwd(x, y, weight=torch.zeros(7, device="cuda"))
    with pytest.raises(bl.TernError):
        bl.tern_norm_fwd(x, torch.zeros(1, 8, device="cuda").expand(4, 8))   # rows of y on one another
    with pytest.raises(bl.TernError):
        bl.tern_norm_fwd(x, y, eps=0.0)
    with pytest.raises(bl.TernError):
        v = torch.zeros(4, device="cuda")
        bl.tern_norm_bwd(x, y, v, v, torch.empty_like(x), dweight=torch.zeros(8, device="cuda"))   # no workspace
