"""The embedding and the gradient of its table on the GPU: the forward bit for bit, the gradient
against fp64 sums within the bound of fp32 sums in any order."""
import numpy as np
import pytest
import torch

from _reference import check, embed_bwd

pytestmark = pytest.mark.gpu


def _tok(n, V, seed, dtype=torch.int64, pad=0.05):
    rng = np.random.default_rng(seed)
    t = np.minimum((V ** rng.random(n)).astype(np.int64) - 1, V - 1)
    t[rng.random(n) < pad] = -1
    t[rng.random(n) < pad] = V          # just past the table
    return torch.from_numpy(t).to(dtype).cuda()


def _bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (5, 3, 7), (33, 256, 8), (100, 1000, 64), (257, 31, 300), (64, 5000, 2056)])
@pytest.mark.parametrize("table", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tok", [torch.int32, torch.int64], ids=["i32", "i64"])
def test_embed_fwd_is_exact(cuda_lib, n, V, D, table, tok):
    t = _tok(n, V, n + D, tok)
    w = torch.randn(V, D, generator=torch.Generator().manual_seed(D)).to(table).cuda()
    out = torch.full((n, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    cuda_lib.tern_embed_fwd(t, w, out, scale=1.7)
    ok = ((t >= 0) & (t < V))[:, None]
    ref = torch.where(ok, w[t.long().clamp(0, V - 1)].float() * np.float32(1.7), torch.zeros((), device="cuda"))
    assert torch.equal(_bits(out), _bits(ref.to(torch.bfloat16)))


@pytest.mark.parametrize("n,D", [(2432, 2048), (2433, 2048), (5001, 2056), (7000, 263), (200001, 16), (160000, 7)])
@pytest.mark.parametrize("table", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_embed_fwd_of_more_rows_than_blocks(cuda_lib, n, D, table):
    """Blocks that loop over rows, the last of them uneven: every row once, and none past the last."""
    t = _tok(n, 900, n + D, torch.int32)
    w = torch.randn(900, D, generator=torch.Generator().manual_seed(D)).to(table).cuda()
    out = torch.full((n + 1, D), 5.0, dtype=torch.bfloat16, device="cuda")
    cuda_lib.tern_embed_fwd(t, w, out[:n], scale=0.3)
    ok = ((t >= 0) & (t < 900))[:, None]
    ref = torch.where(ok, w[t.long().clamp(0, 899)].float() * np.float32(0.3), torch.zeros((), device="cuda"))
    assert torch.equal(_bits(out[:n]), _bits(ref.to(torch.bfloat16))) and torch.all(out[n] == 5.0)


@pytest.mark.parametrize("D", [1, 5, 15, 16, 23, 247, 248, 249, 256, 263, 521])
@pytest.mark.parametrize("table", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_embed_rows_at_every_address(cuda_lib, D, table):
    """Tables, outputs and gradients that start at every element of a 16-byte word, with NaN on both
    sides of each and between strided rows: bit for bit the aligned call's, and nothing else written."""
    bl = cuda_lib
    n, V = 130, 40
    t = _tok(n, V, D, torch.int32)
    w = torch.randn(V, D, generator=torch.Generator().manual_seed(D)).to(table).cuda()
    ok = ((t >= 0) & (t < V))[:, None]
    ref = torch.where(ok, w[t.long().clamp(0, V - 1)].float() * np.float32(0.7), torch.zeros((), device="cuda")).bfloat16()
    ints = torch.randint(-9, 10, (n, D), device="cuda").bfloat16()
    gref = torch.zeros(V, D, device="cuda").index_add_(0, t.long().clamp(0, V - 1), torch.where(ok, ints.float(), torch.zeros((), device="cuda")))
    ws = torch.empty(bl.tern_embed_bwd_workspace(n, V, D), dtype=torch.uint8, device="cuda")
    for off in range(8):
        ld = D + (0, 3, 8)[off % 3]
        nan = lambda k, dt: torch.full((k,), float("nan"), dtype=dt, device="cuda")  # noqa: E731
        tbuf, obuf, dbuf, gbuf = nan(V * D + 9, table), nan(n * ld + 9, torch.bfloat16), nan(n * ld + 9, torch.bfloat16), nan(V * D + 9, torch.float32)
        tab, g = (b[off:off + V * D].view(V, D) for b in (tbuf, gbuf))
        out, dout = (b[off:off + n * ld].as_strided((n, D), (ld, 1), off) for b in (obuf, dbuf))
        tab.copy_(w), dout.copy_(ints)
        bl.tern_embed_fwd(t, tab, out, scale=0.7)
        assert torch.equal(_bits(out), _bits(ref)) and int(obuf.isnan().sum()) == obuf.numel() - n * D
        bl.tern_embed_bwd(t, dout, g, ws)
        assert torch.equal(g, gref) and int(gbuf.isnan().sum()) == 9
        bl.tern_embed_bwd(t, dout, g, ws, accumulate=True)
        assert torch.equal(g, 2 * gref) and int(gbuf.isnan().sum()) == 9


def test_embed_strided_rows_and_odd_addresses(cuda_lib):
    bl = cuda_lib
    for D in (64, 63):
        t = _tok(300, 50, D)
        w = torch.randn(50, D, device="cuda")
        wide = torch.full((300, 2 * D), 5.0, dtype=torch.bfloat16, device="cuda")
        odd = torch.full((300 * D + 1,), 5.0, dtype=torch.bfloat16, device="cuda")[1:].view(300, D)
        ref = torch.empty(300, D, dtype=torch.bfloat16, device="cuda")
        bl.tern_embed_fwd(t, w, ref)
        bl.tern_embed_fwd(t, w, wide[:, D:])
        bl.tern_embed_fwd(t, w, odd)
        assert torch.equal(wide[:, D:], ref) and torch.all(wide[:, :D] == 5.0) and torch.equal(odd, ref)
        ws = torch.empty(bl.tern_embed_bwd_workspace(300, 50, D), dtype=torch.uint8, device="cuda")
        d = [torch.full((50, D), float("nan"), device="cuda") for _ in range(3)]
        wide[:, :D] = float("nan")
        for x, g in zip((ref, wide[:, D:], odd), d):
            bl.tern_embed_bwd(t, x, g, ws)
        assert torch.equal(d[0], d[1]) and torch.equal(d[0], d[2])


SIZES = [(1, 1, 1), (1, 256, 8), (31, 2, 7), (256, 1, 64), (257, 255, 256), (2048, 256, 264), (2049, 2047, 33),
         (5000, 2048, 40), (5000, 70000, 16), (9000, 5, 520), (3000, 300000, 3)]


@pytest.mark.parametrize("n,V,D", SIZES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_bwd(cuda_lib, n, V, D, accumulate):
    bl = cuda_lib
    t = _tok(n, V, n + V, torch.int32 if accumulate else torch.int64)
    rng = np.random.default_rng(n)
    dout = torch.from_numpy(rng.normal(size=(n, D)).astype(np.float32)).cuda().bfloat16()
    g = torch.full((V, D), 0.5 if accumulate else float("nan"), device="cuda")
    ws = torch.full((bl.tern_embed_bwd_workspace(n, V, D),), 0xAB, dtype=torch.uint8, device="cuda")
    bl.tern_embed_bwd(t, dout, g, ws, scale=1.7, accumulate=accumulate)
    ref, bound = embed_bwd(t.cpu().numpy().astype(np.int64), dout.float().cpu().numpy(), V, 1.7)
    if accumulate:
        ref, bound = ref + 0.5, bound + (np.abs(ref) + 0.5) * 2.0 ** -23
    check("dtable", g.cpu().numpy(), ref, bound)
    if not accumulate:   # the same bits again, over a used workspace
        g2 = torch.full_like(g, float("nan"))
        bl.tern_embed_bwd(t, dout, g2, ws, scale=1.7)
        assert torch.equal(g, g2)


@pytest.mark.parametrize("n,V", [(32768, 300), (32769, 5000), (65537, 3), (100000, 2047), (131072, 2048), (140000, 9000), (131073, 2)])
def test_embed_bwd_many_positions(cuda_lib, n, V):
    """Each of the ways to sort: one cluster with tiles of three sizes, and three launches a pass."""
    bl = cuda_lib
    D = 3
    t = _tok(n, V, n)
    dout = torch.randint(-8, 9, (n, D), device="cuda").bfloat16()      # integers: the sums are exact
    g = torch.full((V, D), float("nan"), device="cuda")
    ws = torch.full((bl.tern_embed_bwd_workspace(n, V, D),), 0xAB, dtype=torch.uint8, device="cuda")
    bl.tern_embed_bwd(t, dout, g, ws)
    ok = (t >= 0) & (t < V)
    ref = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, t[ok], dout[ok].double())
    assert torch.equal(g.double(), ref)


@pytest.mark.parametrize("n", [255, 256, 257, 512, 4096, 5001])
def test_embed_bwd_long_runs(cuda_lib, n):
    """One token for all positions, and three whose runs end at, before and past the tiles' edges."""
    bl = cuda_lib
    D = 40
    dout = torch.randn(n, D, device="cuda").bfloat16()
    ws = torch.empty(bl.tern_embed_bwd_workspace(n, 9, D), dtype=torch.uint8, device="cuda")
    cuts = [np.full(n, 4), np.where(np.arange(n) < 256, 2, 7), np.where(np.arange(n) < 31, 0, np.where(np.arange(n) < 255, 3, 8)),
            np.where(np.arange(n) < n - 1, 5, 6)]
    for c in cuts:
        t = torch.from_numpy(np.random.default_rng(n).permutation(c)).cuda()
        g = torch.full((9, D), float("nan"), device="cuda")
        bl.tern_embed_bwd(t, dout, g, ws)
        ref, bound = embed_bwd(t.cpu().numpy(), dout.float().cpu().numpy(), 9, 1.0)
        check("dtable", g.cpu().numpy(), ref, bound)


def test_embed_padding_only_empty_and_masked_values(cuda_lib):
    bl = cuda_lib
    n, V, D = 70, 20, 24
    ws = torch.empty(bl.tern_embed_bwd_workspace(n, V, D), dtype=torch.uint8, device="cuda")
    t = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    t[1], t[2], t[3] = V, 2 ** 40, -2 ** 40           # ids that wrap in 32 bits are still outside
    dout = torch.full((n, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    g = torch.full((V, D), float("nan"), device="cuda")
    bl.tern_embed_bwd(t, dout, g, ws)
    assert torch.all(g == 0)
    out = torch.full((n, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    bl.tern_embed_fwd(t, torch.full((V, D), float("nan"), device="cuda"), out)
    assert torch.all(out == 0)
    t[5] = 3                                          # one live position among NaN ones
    dout[5] = 2.0
    bl.tern_embed_bwd(t, dout, g, ws)
    assert torch.all(g[3] == 2.0) and g.sum().item() == 2.0 * D
    g.fill_(float("nan"))                             # no positions at all: zeros; with accumulate nothing
    bl.tern_embed_bwd(t[:0], dout[:0], g, ws)
    assert torch.all(g == 0)
    g.fill_(7.0)
    bl.tern_embed_bwd(t[:0], dout[:0], g, ws, accumulate=True)
    assert torch.all(g == 7.0)
    bl.tern_embed_fwd(t[:0], g, out[:0])
    torch.cuda.synchronize()


def test_embed_graph_and_stream(cuda_lib):
    bl = cuda_lib
    n, V, D = 5000, 3000, 64
    t, dout = _tok(n, V, 1), torch.randn(n, D, device="cuda").bfloat16()
    ws = torch.empty(bl.tern_embed_bwd_workspace(n, V, D), dtype=torch.uint8, device="cuda")
    w = torch.randn(V, D, device="cuda")
    out, g = torch.empty(n, D, dtype=torch.bfloat16, device="cuda"), torch.empty(V, D, device="cuda")
    f, b = bl.EmbedForward(t, w, out), bl.EmbedBackward(t, dout, g, ws)
    f(), b()
    torch.cuda.synchronize()
    o1, g1 = out.clone(), g.clone()
    out.fill_(float("nan")), g.fill_(float("nan"))
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        f(), b()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o1) and torch.equal(g, g1)


def test_embed_tables_and_rows_past_32_bits(cuda_lib):
    """A table of more than 2^31 elements, and output rows that far apart."""
    bl = cuda_lib
    V, D = 70000, 32768
    t = torch.tensor([V - 1, 3, V - 1, 0, V], device="cuda")
    dout = torch.randint(-8, 9, (5, D), device="cuda").bfloat16()
    g = torch.full((V, D), 7.0, device="cuda")
    ws = torch.empty(bl.tern_embed_bwd_workspace(5, V, D), dtype=torch.uint8, device="cuda")
    bl.tern_embed_bwd(t, dout, g, ws)
    assert torch.equal(g[V - 1], dout[0].float() + dout[2].float())
    assert torch.equal(g[3], dout[1].float()) and torch.equal(g[0], dout[3].float())
    assert torch.count_nonzero(g) == sum(torch.count_nonzero(g[k]) for k in (0, 3, V - 1))
    n, ld = 2200, 1 << 20
    out = torch.zeros(n * ld, dtype=torch.bfloat16, device="cuda").as_strided((n, 8), (ld, 1))
    w = g[:, :8].contiguous()
    tok = torch.full((n,), 1, device="cuda")
    tok[-1] = V - 1
    bl.tern_embed_fwd(tok, w, out)
    assert torch.equal(out[-1].float(), w[V - 1].bfloat16().float()) and torch.count_nonzero(out[:-1]) == 0


def test_embed_gradient_against_differences(cuda_lib):
    """The forward is linear in the table: <dout, embed(U)> = <dtable, U>, in fp64 sums."""
    bl = cuda_lib
    n, V, D = 400, 60, 32
    t, dout = _tok(n, V, 3), torch.randn(n, D, device="cuda").bfloat16()
    u = torch.randint(-3, 4, (V, D), device="cuda").float()        # exact in bf16
    out, g = torch.empty(n, D, dtype=torch.bfloat16, device="cuda"), torch.empty(V, D, device="cuda")
    ws = torch.empty(bl.tern_embed_bwd_workspace(n, V, D), dtype=torch.uint8, device="cuda")
    bl.tern_embed_fwd(t, u, out, scale=2.0)
    bl.tern_embed_bwd(t, dout, g, ws, scale=2.0)
    left, right = (out.double() * dout.double()).sum(), (g.double() * u.double()).sum()
    size = (out.double() * dout.double()).abs().sum()
    assert abs(left - right) <= 400 * 2.0 ** -24 * size


def test_embed_refusals(cuda_lib):
    bl = cuda_lib
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    w, out = torch.zeros(5, 8, device="cuda"), torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        bl.tern_embed_fwd(t.short(), w, out)
    with pytest.raises(TypeError):
        bl.tern_embed_fwd(t, w.half(), out)
    with pytest.raises(TypeError):
        bl.tern_embed_fwd(t, w, out.float())
    with pytest.raises(ValueError):
        bl.tern_embed_fwd(t, w, out[:3])
    with pytest.raises(ValueError):
        bl.tern_embed_fwd(t, w.t().contiguous().t(), out)
    with pytest.raises(ValueError):
        bl.tern_embed_fwd(t, w, out.t().contiguous().t())
    small = torch.zeros(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(bl.TernError) as e:
        bl.tern_embed_bwd(t, out, w, small)
    assert e.value.status == bl.TERN_ERR_WORKSPACE
    with pytest.raises(bl.TernError) as e:
        bl.tern_embed_bwd(t, out, w, None)
    assert e.value.status == bl.TERN_ERR_WORKSPACE
