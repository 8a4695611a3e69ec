"""The gated linear recurrence on the GPU against the fp64 reference: forward, gradient and
single tokens over odd sizes, strides, padding, packed documents and non-finite masked values."""
import numpy as np
import pytest
import torch

from _reference import check, scan

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # of 8 and 24 significand bits


def _np(t):
    return t.detach().float().cpu().numpy()


class Case:
    """Inputs, poisoned outputs and the calls of one problem; fused: f, v, r are views of one [B, T, 3D]."""

    def __init__(self, bl, B, T, D, dtype=torch.float32, seed=0, lengths=None, starts=None, layout="dense"):
        self.bl, self.shape, self.dtype = bl, (B, T, D), dtype
        rng = np.random.default_rng(seed)

        def act(scale=1.0):
            x = torch.from_numpy((rng.normal(size=(B, T, D)) * scale).astype(np.float32)).cuda().to(dtype)
            return self.place(x, layout)
        self.layout = layout
        self.f, self.v, self.r, self.dy = act(), act(), act(), act(0.1)
        if layout == "fused":
            buf = torch.empty(B, T, 3 * D, dtype=dtype, device="cuda")
            for i, x in enumerate((self.f, self.v, self.r)):
                buf[..., i * D:(i + 1) * D] = x
            self.f, self.v, self.r = (buf[..., i * D:(i + 1) * D] for i in range(3))
        f32 = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).cuda()  # noqa: E731
        self.bias = torch.from_numpy(np.linspace(0.5, 6.0, D).astype(np.float32)).cuda()
        self.h0, self.dhT = f32(B, D), f32(B, D)
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.starts = None if starts is None else torch.from_numpy(starts.astype(np.uint8)).cuda()
        nan = float("nan")
        self.y, self.df, self.dv, self.dr = (self.place(torch.full((B, T, D), nan, dtype=dtype, device="cuda"), layout)
                                             for _ in range(4))
        self.hT, self.dh0 = (torch.full((B, D), nan, device="cuda") for _ in range(2))
        self.dbias = torch.full((D,), nan, device="cuda")
        self.saved = torch.full((max(4, bl.tern_scan_saved(B, T, D) // 4),), nan, device="cuda")
        self.ws = torch.full((max(4, bl.tern_scan_bwd_workspace(B, T, D) // 4),), nan, device="cuda")

    @staticmethod
    def place(x, layout):
        B, T, D = x.shape
        if layout == "time_major":      # [T, B, D] in memory
            return x.transpose(0, 1).contiguous().transpose(0, 1)
        if layout == "offset":          # one element past an aligned address, padded rows
            buf = torch.zeros(B * T * (D + 1) + 1, dtype=x.dtype, device="cuda")[1:].view(B, T, D + 1)[..., :D]
            buf.copy_(x)
            return buf
        return x.contiguous()

    def run(self, stream=None):
        kw = dict(f_bias=self.bias, lengths=self.lengths, starts=self.starts, stream=stream)
        self.bl.tern_scan_fwd(self.f, self.v, self.r, self.y, h0=self.h0, hT=self.hT, saved=self.saved, **kw)
        self.bl.tern_scan_bwd(self.f, self.v, self.r, self.dy, self.saved, self.ws, self.df, self.dv, self.dr,
                              dhT=self.dhT, dbias=self.dbias, dh0=self.dh0, **kw)
        return self

    def outputs(self):
        return {k: getattr(self, k) for k in ("y", "hT", "df", "dv", "dr", "dbias", "dh0")}

    def check(self, f=None, v=None, r=None, dy=None, h0=None):
        """Against the reference, on other inputs where given (what stands for masked values)."""
        pick = lambda x, own: _np(own) if x is None else x  # noqa: E731
        ref = scan(pick(f, self.f), pick(v, self.v), pick(r, self.r), _np(self.bias), pick(h0, self.h0),
                   None if self.lengths is None else self.lengths.cpu().numpy(),
                   None if self.starts is None else self.starts.cpu().numpy(), pick(dy, self.dy), _np(self.dhT))
        for name, got in self.outputs().items():
            val, err = ref[name]
            own = HALF_ULP[self.dtype] if got.dtype == self.dtype and name not in ("hT", "dh0", "dbias") else 2.0 ** -24
            check(name, _np(got), val, err * (1 + own) + np.abs(val) * own * 1.01 + 1e-37)
        return self


SIZES = [(1, 1, 1), (1, 2, 2), (2, 15, 31), (2, 16, 64), (3, 17, 65), (1, 63, 130), (2, 64, 66), (1, 65, 33),
         (2, 127, 64), (1, 128, 40), (1, 129, 7), (1, 1100, 70), (1, 2500, 64), (5, 300, 129)]


@pytest.mark.parametrize("B,T,D", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_scan_sizes(cuda_lib, B, T, D, dtype):
    Case(cuda_lib, B, T, D, dtype, seed=T + D).run().check()


@pytest.mark.parametrize("B,T,D", [(320, 200, 64), (160, 260, 64), (80, 520, 33), (320, 65, 8)])
def test_scan_clusters_and_single_blocks(cuda_lib, B, T, D):
    """From one block per sequence and channel tile up to clusters of eight."""
    Case(cuda_lib, B, T, D, torch.bfloat16, seed=B).run().check()


@pytest.mark.parametrize("layout", ["fused", "time_major", "offset"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_scan_strides(cuda_lib, layout, dtype):
    for D in (64, 35):
        Case(cuda_lib, 3, 150, D, dtype, seed=D, layout=layout).run().check()


def _starts(B, T, seed, p=0.05):
    rng = np.random.default_rng(seed)
    s = rng.random((B, T)) < p
    for t in (0, 15, 16, 63, 64, 127, 128):
        if t < T:
            s[t % B, t] = True
    return s


@pytest.mark.parametrize("T", [1, 16, 130, 1200])
def test_scan_padding_and_documents(cuda_lib, T):
    B = 5
    lengths = [0, 1, T // 2, T - 1, T]
    Case(cuda_lib, B, T, 66, torch.float32, 3, lengths=lengths).run().check()
    Case(cuda_lib, B, T, 66, torch.bfloat16, 4, starts=_starts(B, T, T)).run().check()
    Case(cuda_lib, B, T, 33, torch.float32, 5, lengths=lengths, starts=_starts(B, T, T + 1)).run().check()
    Case(cuda_lib, 2, T, 32, torch.float32, 6, lengths=[-3, T + 9]).run().check()      # clamped to 0..T


@pytest.mark.parametrize("B,T,D", [(330, 140, 32), (40, 700, 64), (2, 3000, 64), (5, 300, 129)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_scan_masks_in_every_block_shape(cuda_lib, B, T, D, dtype):
    """Uneven lengths and packed documents with many blocks, eight-warp clusters and narrow tiles."""
    rng = np.random.default_rng(T)
    lengths = rng.integers(0, T + 1, B)
    lengths[:2] = 0, T
    Case(cuda_lib, B, T, D, dtype, 3, lengths=lengths.tolist(), starts=_starts(B, T, D, 0.01)).run().check()


def test_scan_sequences_more_than_32_bits_apart(cuda_lib):
    """Sequences 2^31 elements apart (the offsets pass 32 bits in elements and in bytes)."""
    B, T, D = 2, 100, 64
    far = 1 << 31
    buf = torch.empty(far + 16 * T * D, dtype=torch.bfloat16, device="cuda")
    c = Case(cuda_lib, B, T, D, torch.bfloat16, 11)
    for i, name in enumerate(("f", "v", "r", "dy", "y", "df", "dv", "dr")):
        x = buf.as_strided((B, T, D), (far, D, 1), i * T * D)
        x.copy_(getattr(c, name))
        setattr(c, name, x)
    c.run().check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min])
def test_scan_masked_values_do_not_leak(cuda_lib, bad):
    """Whatever lies in padding, and whatever state an earlier document left, stays out."""
    B, T, D = 4, 200, 64
    lengths = [0, 1, 70, 199]
    c = Case(cuda_lib, B, T, D, torch.float32, 8, lengths=lengths, starts=_starts(B, T, 9))
    keep = [x.clone() for x in (c.f, c.v, c.r, c.dy)]
    for b, L in enumerate(lengths):
        for x in (c.f, c.v, c.r, c.dy):
            x[b, L:] = bad
    c.run().check(*[_np(x) for x in keep])
    # the first document's state is poison; the second starts at row 33
    starts = np.zeros((1, T), bool)
    starts[0, 33] = True
    c = Case(cuda_lib, 1, T, D, torch.float32, 10, starts=starts)
    c.h0.fill_(bad)
    c.run()
    ref = Case(cuda_lib, 1, T, D, torch.float32, 10, starts=starts).run()
    for k in ("y", "df", "dv", "dr"):
        assert torch.equal(getattr(c, k)[:, 33:], getattr(ref, k)[:, 33:]), k
    assert torch.equal(c.hT, ref.hT)


def test_scan_saturated_gates(cuda_lib):
    """Gates of +-infinity and of the type's extremes: keep the state, or take the value, exactly."""
    B, T, D = 2, 70, 8
    inf = float("inf")
    for big in (inf, 3e38, 100.0):
        c = Case(cuda_lib, B, T, D, torch.float32, 1)
        c.f.fill_(big)
        c.r.fill_(big)
        c.run()
        assert torch.equal(c.hT, c.h0) and torch.equal(c.y, c.h0[:, None].expand(B, T, D))
        c.f.fill_(-big)
        c.run()
        assert torch.allclose(c.y, c.v, rtol=2 ** -22, atol=1e-30) and torch.all(c.dh0.abs() <= 1e-30)
        c.r.fill_(-big)
        c.run()
        assert torch.all(c.y.abs() <= 1e-30)


def test_scan_a_nan_spreads_only_where_it_is_used(cuda_lib):
    c = Case(cuda_lib, 2, 40, 6, torch.float32, 2)
    c.f[1, 20, 3] = float("nan")
    c.run()
    assert torch.isnan(c.y[1, 20:, 3]).all() and not torch.isnan(c.y[1, :20]).any()
    y = c.y.clone()
    y[1, 20:, 3] = 0
    assert not torch.isnan(y).any()


@pytest.mark.parametrize("B,T,D", [(0, 5, 8), (2, 0, 8), (2, 5, 0)])
def test_scan_empty(cuda_lib, B, T, D):
    c = Case(cuda_lib, B, T, D, torch.bfloat16)
    if B == 0:   # no sequence: dbias has nothing to sum over and is refused
        cuda_lib.tern_scan_fwd(c.f, c.v, c.r, c.y, hT=c.hT, saved=c.saved)
        with pytest.raises(cuda_lib.TernError):
            c.run()
        return
    c.run()
    torch.cuda.synchronize()
    if T == 0:
        assert torch.equal(c.hT, c.h0) and torch.equal(c.dh0, c.dhT) and torch.all(c.dbias == 0)


def test_scan_optional_arguments(cuda_lib):
    """No bias, no initial state, no final state, no saved states: the same as zeros."""
    bl = cuda_lib
    c = Case(bl, 2, 100, 40, torch.float32, 3)
    c.bias.zero_(), c.h0.zero_(), c.dhT.zero_()
    c.run()
    y, df, dv, dr = (torch.empty_like(c.y) for _ in range(4))
    bl.tern_scan_fwd(c.f, c.v, c.r, y)
    bl.tern_scan_bwd(c.f, c.v, c.r, c.dy, c.saved, None, df, dv, dr)
    for a, b in ((y, c.y), (df, c.df), (dv, c.dv), (dr, c.dr)):
        assert torch.equal(a, b)


def test_scan_same_bits_on_another_stream_and_from_a_graph(cuda_lib):
    starts = _starts(2, 1500, 1)
    c = Case(cuda_lib, 2, 1500, 96, torch.bfloat16, 5, starts=starts).run()
    torch.cuda.synchronize()
    first = {k: x.clone() for k, x in c.outputs().items()}
    s = torch.cuda.Stream()
    for x in (c.saved, *c.outputs().values()):
        x.fill_(float("nan"))
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    for k, x in c.outputs().items():
        assert torch.equal(x, first[k]), k
        x.fill_(float("nan"))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        c.run()
    graph.replay()
    torch.cuda.synchronize()
    for k, x in c.outputs().items():
        assert torch.equal(x, first[k]), k


def test_scan_split_in_two_continues_the_state(cuda_lib):
    """Two calls, the second from the first's hT, against one call."""
    bl = cuda_lib
    c = Case(bl, 2, 300, 64, torch.float32, 6).run()
    y = torch.full_like(c.y, float("nan"))
    h = torch.empty_like(c.h0)
    for lo, hi in ((0, 129), (129, 300)):
        bl.tern_scan_fwd(c.f[:, lo:hi], c.v[:, lo:hi], c.r[:, lo:hi], y[:, lo:hi], f_bias=c.bias,
                         h0=c.h0 if lo == 0 else h, hT=h)
    c.y, c.hT = y, h
    c.check()


@pytest.mark.parametrize("B,D", [(1, 1), (1, 512), (7, 33), (64, 130), (300, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_step_matches_the_scan(cuda_lib, B, D, dtype):
    bl = cuda_lib
    c = Case(bl, B, 3, D, dtype, 7).run()
    h = c.h0.clone()
    y = torch.full_like(c.y, float("nan"))
    for t in range(3):   # in place, on strided views of the sequence
        bl.tern_scan_step(c.f[:, t], c.v[:, t], c.r[:, t], h, y[:, t], f_bias=c.bias)
    c.y, c.hT = y, h
    c.check()
    out = torch.full_like(c.h0, float("nan"))
    bl.tern_scan_step(c.f[:, 0], c.v[:, 0], c.r[:, 0], c.h0, y[:, 0], h_out=out, f_bias=c.bias)
    h1 = c.h0.clone()
    bl.tern_scan_step(c.f[:, 0], c.v[:, 0], c.r[:, 0], h1, y[:, 1], f_bias=c.bias)
    assert torch.equal(out, h1) and torch.equal(y[:, 0], y[:, 1])


def test_scan_gradient_against_differences_of_the_forward(cuda_lib):
    """The kernel's gradient along a random direction against central differences of the fp64 forward."""
    c = Case(cuda_lib, 2, 90, 20, torch.float32, 12, lengths=[60, 90], starts=_starts(2, 90, 2)).run()
    x = [_np(t).astype(np.float64) for t in (c.f, c.v, c.r, c.bias, c.h0)]
    rng = np.random.default_rng(0)
    u = [rng.normal(size=t.shape) for t in x]
    L, S = c.lengths.cpu().numpy(), c.starts.cpu().numpy()

    def loss(eps):
        o = scan(*[a + eps * b for a, b in zip(x, u)], L, S)
        return (o["y"][0] * _np(c.dy)).sum() + (o["hT"][0] * _np(c.dhT)).sum()
    num = (loss(1e-5) - loss(-1e-5)) / 2e-5
    parts = [(_np(g).astype(np.float64) * b) for g, b in zip((c.df, c.dv, c.dr, c.dbias, c.dh0), u)]
    got, size = sum(p.sum() for p in parts), sum(np.abs(p).sum() for p in parts)
    assert abs(num - got) <= 1e-5 * size     # fp32 gradients: about 1e-6 of each term; differences: 1e-9


def test_scan_refusals(cuda_lib):
    bl = cuda_lib
    c = Case(bl, 2, 10, 8, torch.float32)
    with pytest.raises(TypeError):
        bl.tern_scan_fwd(c.f.half(), c.v, c.r, c.y)
    with pytest.raises(TypeError):
        bl.tern_scan_fwd(c.f, c.v.bfloat16(), c.r, c.y)
    with pytest.raises(TypeError):
        bl.tern_scan_fwd(c.f.cpu(), c.v, c.r, c.y)
    with pytest.raises(ValueError):
        bl.tern_scan_fwd(c.f, c.v[:, :9], c.r, c.y)
    with pytest.raises(ValueError):
        bl.tern_scan_fwd(c.f, c.v, c.r, c.y.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        bl.tern_scan_fwd(c.f, c.v, c.r, c.y, h0=c.h0[:, :4])
    with pytest.raises(TypeError):
        bl.tern_scan_fwd(c.f, c.v, c.r, c.y, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(bl.TernError) as e:
        bl.tern_scan_fwd(c.f, c.v, c.r, c.y, saved=c.saved[:1])
    assert e.value.status == bl.TERN_ERR_WORKSPACE
    with pytest.raises(ValueError):
        bl.tern_scan_bwd(c.f, c.v, c.r, c.dy, c.saved[:1], c.ws, c.df, c.dv, c.dr)
    with pytest.raises(bl.TernError) as e:
        bl.tern_scan_bwd(c.f, c.v, c.r, c.dy, c.saved, c.ws[:1], c.df, c.dv, c.dr, dbias=c.dbias)
    assert e.value.status == bl.TERN_ERR_WORKSPACE
    with pytest.raises(ValueError):
        bl.tern_scan_step(c.f, c.v, c.r, c.h0, c.y)


class Guarded(Case):
    """Rows that start `off` elements past an aligned address and lie `pad` apart, NaN around them."""

    @staticmethod
    def place(x, layout):
        off, pad = layout
        B, T, D = x.shape
        buf = torch.full((B * T * (D + pad) + 16,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf.as_strided((B, T, D), (T * (D + pad), D + pad, 1), off)
        view.copy_(x)
        return view

    def outside(self):
        """The elements around the outputs that a call wrote."""
        n = 0
        for t in (self.y, self.df, self.dv, self.dr):
            whole = torch.empty(0, dtype=t.dtype, device="cuda").set_(t.untyped_storage())
            n += int((~whole.isnan()).sum()) - t.numel()
        return n


@pytest.mark.parametrize("B,T,D", [(2, 130, 33), (3, 70, 34), (1, 600, 36), (320, 64, 35), (1, 2500, 71)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_scan_rows_at_every_address(cuda_lib, B, T, D, dtype):
    """Whatever words the rows' addresses allow: right, the same bits, and nothing else read or written."""
    first = None
    for off, pad in ((0, 0), (1, 0), (2, 0), (3, 1), (5, 2), (0, 1), (4, 4)):
        case = Guarded(cuda_lib, B, T, D, dtype, seed=D, layout=(off, pad)).run()
        if first is None:
            first = case.check().outputs()
        for name, got in case.outputs().items():
            assert torch.equal(got, first[name]), (name, off, pad)
        assert case.outside() == 0, (off, pad)
