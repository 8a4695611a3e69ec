"""The gated feed-forward layer and its gradient on the GPU against the formulas in fp64.

Bounds: a tensor core adds K / 16 groups of exact products, each addition off by at most 2^-22 of the
sum of magnitudes (truncation of the aligned terms), so g and u are off by d = (K / 16 + 4) 2^-22
times that sum.  act moves by (|act'| + 2 d) d (|act''| <= 2 for each), plus 2^-19 relative of the
special functions and for gelu 1.5e-7 |g|; act' by 2 d and 2^-19 (1 + |act|).  Then one rounding to bf16, 2^-8,
or two where the gradient multiplies stored factors."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

H8 = 2.0 ** -8
ACTS = ["silu", "gelu", "relu2", "sigmoid"]


def _act(g, name):
    if name == "relu2":
        r = g.clamp(min=0)
        return r * r, 2 * r
    if name == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    return (s, s * c) if name == "sigmoid" else (g * s, s + g * s * c)


def _ternary(q):
    return torch.where(q.abs() >= 2, torch.sign(q), torch.zeros_like(q)).double()


def _ref(X, q, scale, act, dH=None):
    """(value, bound before rounding) of H, the factors of dG and dU."""
    K, N = q.shape[0], q.shape[1] // 2
    T, X, s = _ternary(q), X.double(), scale.double()
    y, off = (X @ T) * s, (X.abs() @ T.abs()) * s.abs() * (K / 16 + 4) * 2.0 ** -22
    g, u, dg, du = y[:, :N], y[:, N:], off[:, :N], off[:, N:]
    a, d = _act(g, act)
    ea = (d.abs() + 2 * dg) * dg + 2.0 ** -19 * a.abs() + (1.5e-7 * g.abs() if act == "gelu" else 0)
    ed = 2 * dg + 2.0 ** -19 * (1 + a.abs())
    H = (a * u, ea * (u.abs() + du) + a.abs() * du)
    fg = (d * u, ed * (u.abs() + du) + d.abs() * du)
    return H, fg, (a, ea)


def _near(got, val, tol, roundings, name):
    assert not got.isnan().any(), name
    err, bound = (got.double() - val).abs(), tol + roundings * H8 * (val.abs() + tol) * (1 + H8) + 1e-38
    assert torch.all(err <= bound), (name, float((err - bound).max()))


def _inputs(M, K, N, seed, zeros=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(-7, 8, (K, 2 * N), dtype=torch.int8, device="cuda", generator=g)
    if zeros:
        q[:, 1] = 0                       # a gate column and a value column without a weight
        q[:, N + 5] = 0
    scale = (0.5 + torch.rand(2 * N, device="cuda", generator=g)) * torch.where(torch.rand(2 * N, device="cuda", generator=g) < 0.2, -1.0, 1.0) * (1.5 / math.sqrt(K))
    X = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    return X, q, scale, torch.randn(M, N, device="cuda", generator=g).bfloat16()


def _tiles(bl, q, scale, **kw):
    t = bl.Tiles.empty(*q.shape, hi_lo=False, **kw)
    bl.tern_materialize(q, scale, t, 2, 7)
    return t


def _new(M, N):
    """[M, N] bf16 with two guard rows behind it."""
    buf = torch.full((M + 2, N), 99.0, dtype=torch.bfloat16, device="cuda")
    return buf[:M], buf[M:]


SIZES = [(1, 16, 16), (3, 48, 32), (8, 512, 2048), (9, 512, 160), (16, 4096, 208), (16, 64, 16), (17, 32, 16), (5, 1040, 1008), (100, 80, 144),
         (128, 64, 128), (129, 512, 272), (256, 128, 128), (300, 1040, 400), (1000, 512, 1360)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_forward_and_both_gradients(cuda_lib, M, K, N, act):
    bl = cuda_lib
    X, q, scale, dH = _inputs(M, K, N, M + K + N)
    tiles = _tiles(bl, q, scale)
    H, fg, fu = _ref(X, q, scale, act)
    out, guard = _new(M, N)
    bl.tern_glu_fwd(X, tiles, scale, out, act=act)
    _near(out, *H, 1, "H")
    out2, guard2 = _new(M, N)
    pair, guard3 = _new(M, 2 * N)
    bl.tern_glu_fwd(X, tiles, scale, out2, saved=pair, act=act)
    _near(out2, *H, 1, "H with factors")
    _near(pair[:, :N], *fg, 1, "factor of dG")
    _near(pair[:, N:], *fu, 1, "factor of dU")
    d = dH.double()
    dY, guard4 = _new(M, 2 * N)
    bl.tern_glu_bwd(dH, dY, saved=pair)
    assert torch.equal(dY[:, :N], (dH.float() * pair[:, :N].float()).bfloat16()) and torch.equal(dY[:, N:], (dH.float() * pair[:, N:].float()).bfloat16())
    bl.tern_glu_bwd(dH, pair, saved=pair)                         # in place
    assert torch.equal(dY, pair)
    bl.tern_glu_bwd(dH, dY, X=X, tiles=tiles, scale=scale, act=act)
    _near(dY[:, :N], fg[0] * d, fg[1] * d.abs(), 1, "dG")
    _near(dY[:, N:], fu[0] * d, fu[1] * d.abs(), 1, "dU")
    assert all(torch.all(t == 99.0) for t in (guard, guard2, guard3, guard4))
    assert bl.tern_device_status() == bl.TERN_OK


@pytest.mark.parametrize("M,K,N", [(1, 16, 16), (1, 8192, 48), (2, 528, 2064), (8, 512, 1360), (11, 4096, 1024), (16, 160, 4112), (17, 4096, 208), (33, 512, 144),
                                   (64, 1024, 400), (100, 48, 1360), (128, 2048, 16), (127, 80, 2064)])
def test_few_rows_from_either_weight(cuda_lib, M, K, N):
    """The codes alone, the bf16 plane alone, and both: each within the same bound, each the same every time."""
    bl = cuda_lib
    X, q, scale, _ = _inputs(M, K, N, K)
    H = _ref(X, q, scale, "silu")[0]
    for kw in (dict(t=False), dict(packed=False), {}):
        tiles = _tiles(bl, q, scale, **kw)
        out, guard = _new(M, N)
        bl.tern_glu_fwd(X, tiles, scale, out)
        _near(out, *H, 1, str(kw))
        again, _ = _new(M, N)
        bl.tern_glu_fwd(X, tiles, scale, again)
        assert torch.equal(out, again) and torch.all(guard == 99.0)


def test_outputs_at_16_bytes(cuda_lib):
    """Outputs that start between 32-byte words: the same bits."""
    bl = cuda_lib
    M, K, N = 150, 64, 80
    X, q, scale, dH = _inputs(M, K, N, 3)
    tiles = _tiles(bl, q, scale)
    outs = []
    for off in (0, 8):
        place = lambda k: torch.full((M * k + 16,), 9.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        bufs = [place(N), place(2 * N), place(2 * N)]
        H, pair, dY = (b[off:off + M * k].view(M, k) for b, k in zip(bufs, (N, 2 * N, 2 * N)))
        bl.tern_glu_fwd(X, tiles, scale, H, saved=pair)
        bl.tern_glu_bwd(dH, dY, X=X, tiles=tiles, scale=scale)
        assert all(torch.all(b[:off] == 9.0) and torch.all(b[off + M * k:] == 9.0) for b, k in zip(bufs, (N, 2 * N, 2 * N)))
        outs.append([t.clone() for t in (H, pair, dY)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_extreme_gates(cuda_lib):
    """Gates far out on both sides: no overflow, no NaN; a NaN row stays in its row."""
    bl = cuda_lib
    for M in (4, 40):
        K = N = 32
        X = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
        X[:, 0] = torch.linspace(-1, 1, M, device="cuda")
        X[:, 1] = 1.0
        X[2, 3] = float("nan")
        q = torch.zeros(K, 2 * N, dtype=torch.int8, device="cuda")
        q[0, :N] = 7
        q[1, N:] = 7
        q[3] = 7
        scale = torch.cat([torch.logspace(-2, 4, N, device="cuda"), torch.ones(N, device="cuda")])
        tiles = _tiles(bl, q, scale)
        dH = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
        rest = [i for i in range(M) if i != 2]
        for act in ACTS:
            H, fg, fu = _ref(X, q, scale, act)
            out, pair, dY = (torch.empty(M, k, dtype=torch.bfloat16, device="cuda") for k in (N, 2 * N, 2 * N))
            bl.tern_glu_fwd(X, tiles, scale, out, act=act)
            assert out[2].isnan().all()
            _near(out[rest], H[0][rest], H[1][rest], 1, act)
            bl.tern_glu_fwd(X, tiles, scale, out, saved=pair, act=act)
            bl.tern_glu_bwd(dH, dY, X=X, tiles=tiles, scale=scale, act=act)
            for got in (pair, dY):
                _near(got[rest, :N], fg[0][rest], fg[1][rest], 1, act)
                _near(got[rest, N:], fu[0][rest], fu[1][rest], 1, act)


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
def test_gates_of_any_size(cuda_lib, act):
    """Gates of +-1e5 to +-1e38, exact in fp32: act is 0 or g (sigmoid: 0 or 1), act' 0 or 1 (sigmoid: 0).
    One rounding, and 2^-20 for the reciprocal and its product."""
    bl, N = cuda_lib, 64
    for M in (4, 40):
        X = torch.zeros(M, 16, device="cuda", dtype=torch.bfloat16)
        X[0::2, 0], X[1::2, 0], X[:, 1] = 1.0, -1.0, 1.0
        q = torch.zeros(16, 2 * N, dtype=torch.int8, device="cuda")
        q[0, :N] = 7
        q[1, N:] = 7
        scale = torch.cat([torch.logspace(5, 38, N, device="cuda"), torch.ones(N, device="cuda")])
        tiles = _tiles(bl, q, scale)
        H, pair = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
        bl.tern_glu_fwd(X, tiles, scale, H, act=act)
        outs = [(H, None)]
        H2 = torch.empty_like(H)
        bl.tern_glu_fwd(X, tiles, scale, H2, saved=pair, act=act)
        outs.append((H2, pair))
        value = torch.ones(N, device="cuda").double() if act == "sigmoid" else scale[:N].double()
        slope = 0.0 if act == "sigmoid" else 1.0
        for h, f in outs:
            assert torch.all(h[1::2].double().abs() <= 1e-37)
            assert torch.all((h[0::2].double() - value).abs() <= value * (H8 + 2.0 ** -20) * (1 + H8))
            if f is not None:
                assert torch.all(f[1::2].double().abs() <= 1e-37)
                assert torch.all((f[0::2, :N].double() - slope).abs() <= H8 + 2.0 ** -20)
                assert torch.equal(f[0::2, N:], h[0::2])


def test_same_bits_streams_and_graphs(cuda_lib):
    bl = cuda_lib
    for M in (1, 16, 200):
        K, N = 512, 1360
        X, q, scale, dH = _inputs(M, K, N, 5)
        tiles = _tiles(bl, q, scale)
        bf = lambda k: torch.empty(M, k, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        H, pair, dY = bf(N), bf(2 * N), bf(2 * N)
        calls = [bl.GluForward(X, tiles, scale, H, saved=pair if M == 200 else None), bl.GluBackward(dH, dY, X=X, tiles=tiles, scale=scale)]

        def run():
            for c in calls:
                c()
            return [t.clone() for t in (H, dY)]
        want = run()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = run()
        side.synchronize()
        assert all(torch.equal(p, r) for p, r in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for c in calls:
                c()
        X2, _, _, dH2 = _inputs(M, K, N, 6)
        X.copy_(X2), dH.copy_(dH2)
        want = run()
        H.zero_(), dY.zero_()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(H, want[0]) and torch.equal(dY, want[1])
        assert bl.tern_device_status() == bl.TERN_OK


def test_refusals(cuda_lib):
    bl = cuda_lib
    X, q, scale, dH = _inputs(20, 32, 32, 1)
    tiles = _tiles(bl, q, scale)
    H, pair = torch.empty(20, 32, dtype=torch.bfloat16, device="cuda"), torch.empty(20, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        bl.tern_glu_fwd(X, tiles, scale, H, act="tanh")
    with pytest.raises(ValueError):
        bl.tern_glu_fwd(X[:, :16].contiguous(), tiles, scale, H)
    with pytest.raises(ValueError):
        bl.tern_glu_fwd(X, tiles, scale, pair)
    with pytest.raises(TypeError):
        bl.tern_glu_fwd(X.float(), tiles, scale, H)
    with pytest.raises(ValueError):
        bl.tern_glu_bwd(dH, pair, X=X)
    with pytest.raises(bl.TernError):                          # from 129 rows on the bf16 plane is read
        bl.tern_glu_fwd(X.repeat(7, 1), _tiles(bl, q, scale, t=False), scale, H.repeat(7, 1))
    with pytest.raises(bl.TernError):                          # and for the factors
        bl.tern_glu_fwd(X[:4], _tiles(bl, q, scale, t=False), scale, H[:4], saved=pair[:4])
