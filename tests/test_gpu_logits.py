"""Scores of logits and distillation on the GPU against the formulas in fp64.

Bounds, u = 2^-24: exp(z) is off by 2^-22 relative from the special function and by u |z| from its scaled argument;
a thread adds at most V / 128 terms (V / 512 from 16 KB rows on), rescales a sum by 2^-22 each time its
maximum moves (at most 20 times here) and joins in 5 + 4 + 16 steps.  So S is off by
E = u (V / 128 + 4 (20 + 25) + sum p |z|) relative, and what is formed from it by that and its own roundings."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]


def _gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, device="cuda", generator=g), lambda *s: torch.rand(*s, device="cuda", generator=g)


def _stats(x, T=1.0):
    """m, z = (x - m) / T, log S, p, A = sum p |z| and E, rows of fp64."""
    m = x.amax(1, keepdim=True)
    z = (x - m) / T
    e = z.exp()
    S = e.sum(1, keepdim=True)
    p = e / S
    A = torch.where(p > 0, p * z.abs(), torch.zeros_like(p)).sum(1, keepdim=True)
    return m, z, S.log(), p, A, U * (x.shape[1] / 128 + 180 + A)


def _close(got, ref, tol, name):
    # equal, or equal once rounded: a value past the type's range (log probabilities down to -6.8e38) is infinite
    same = (got.double() == ref) | (got == ref.to(got.dtype)) | (got.isnan() & ref.isnan())
    err = torch.where(same, torch.zeros_like(ref), (got.double() - ref).abs())
    bound = torch.where(same, torch.zeros_like(ref), tol + HALF[got.dtype] * (ref.abs() + tol))
    assert not (err.isnan() & ~same).any() and torch.all(err <= bound), (name, float((err - bound).max()))


def _top(x, k):
    return torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)


def _score(bl, x, tok, k):
    n = x.shape[0]
    new = lambda *s: torch.full(s, 77.0, device="cuda")  # noqa: E731
    logp, ent, lse = new(n), new(n), new(n)
    ids, top = (torch.full((n, k), -7, dtype=torch.int32, device="cuda"), new(n, k)) if k else (None, None)
    bl.tern_score(x, tok, logp, ent, lse, ids, top)
    return logp, ent, lse, ids, top


def _check_score(bl, x, tok, k, ties=True):
    n, V = x.shape
    logp, ent, lse, ids, top = _score(bl, x, tok, k)
    x = x.double()
    m, z, logS, p, A, E = _stats(x)
    dead = m == -math.inf            # rows of nothing else: -inf, and entropy 0, exactly
    zero = torch.zeros_like(m)
    lp = torch.where(dead, -math.inf, z - logS)
    tol = torch.where(dead, zero, E + 2 * U * logS.abs() + 2 * U * torch.where(z > -math.inf, z.abs(), torch.zeros_like(z)))
    _close(lse, torch.where(dead, -math.inf, m + logS)[:, 0], torch.where(dead, zero, E + 2 * U * (m.abs() + logS.abs()))[:, 0], "lse")
    _close(ent, torch.where(dead, zero, logS + A)[:, 0], torch.where(dead, zero, E * (1 + 2 * A) + 4 * U * (logS.abs() + A))[:, 0], "entropy")
    inside = (tok >= 0) & (tok < V)
    at = tok.long().clamp(0, V - 1)[:, None]
    zero = torch.zeros(n, dtype=torch.float64, device="cuda")
    _close(logp, torch.where(inside, lp.gather(1, at)[:, 0], zero), torch.where(inside, tol.gather(1, at)[:, 0], zero), "logp")
    if k:
        want = _top(x, k)
        assert torch.equal(ids, want)
        _close(top, lp.gather(1, want.long()), tol.gather(1, want.long()), "top")


def _tokens(n, V, dtype=torch.int64):
    t = torch.arange(n, device="cuda") * 7919 % V
    t[::5] = -1
    t[1::7] = V
    return t.to(dtype)


@pytest.mark.parametrize("n,V", [(1, 1), (3, 5), (9, 64), (70, 256), (6, 257), (5, 1000), (4, 1024), (700, 1025), (2500, 700), (2500, 3001), (1300, 9001), (3, 2050), (400, 4099), (33, 8192),
                                 (2, 8193), (350, 16411), (1, 50000), (3, 100003), (330, 33000), (1, 262145)])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_score(cuda_lib, n, V, dtype):
    randn, _ = _gen(n + V)
    x = (randn(n, V) * 3 + randn(V)).to(dtype)
    for k in sorted({0, 1, min(5, V), min(64, V)}):
        _check_score(cuda_lib, x, _tokens(n, V, torch.int32 if k == 1 else torch.int64), k)


@pytest.mark.parametrize("V", [40, 300, 1500, 9000, 70000])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_score_masks_and_ties(cuda_lib, V, dtype):
    """Masked rows down to one entry, constant rows, few distinct values, ascending, descending and periodic
    rows, the largest entries in one thread's words; equal logits in the order of their ids."""
    randn, rand = _gen(V)
    k, i = min(64, V), torch.arange(V, device="cuda")
    rows = [randn(V).masked_fill(rand(V) < s, -math.inf) for s in (0.3, 0.9, 0.99)]
    lone = torch.full((V,), -math.inf, device="cuda")
    lone[V // 2] = 1.5
    few = torch.full((V,), -math.inf, device="cuda")
    few[V - 3:], few[1] = 2.0, -4.0
    rows += [lone, few, torch.full((V,), -2.5, device="cuda"), torch.zeros(V, device="cuda") * torch.where(i % 2 == 0, 1.0, -1.0)]
    rows += [(i % 3).float(), -(i % 3).float(), (i / V * 8).float(), (-i / V * 8).float(), (i % 4096).float() / 512, (i // 8 % 128).float() / 16,
             torch.where(i // 8 % 128 < 4, 5.0 + rand(V), randn(V)), torch.where(i // 4 % 512 < 3, 5.0 + rand(V), -5.0 - rand(V))]
    rows += [torch.round(randn(V) * 2) / 2 + (V - i) * 0.0, torch.cat([randn(V - 1), torch.tensor([9.0], device="cuda")])]
    x = torch.stack(rows).to(dtype)
    for kk in {1, k // 2, k}:
        _check_score(cuda_lib, x, _tokens(len(rows), V), kk)
        _check_score(cuda_lib, x[:1], _tokens(1, V) + 3, kk)     # a row that blocks share
        for r in (3, 4, 5, 6, 7, 13):
            _check_score(cuda_lib, x[r:r + 1], _tokens(1, V) + 3, kk)


@pytest.mark.parametrize("V", [200, 3000, 40000])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_masks_of_the_lowest_value(cuda_lib, V, dtype):
    """Entries masked by the type's lowest value in place of -inf, rows of nothing else, and values near both ends."""
    randn, rand = _gen(V)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = torch.stack([randn(V).masked_fill(rand(V) < 0.5, low), torch.full((V,), low, device="cuda"),
                     torch.where(rand(V) < 0.5, low, high), torch.where(torch.arange(V, device="cuda") == 7, 1.0, low)]).to(dtype)
    _check_score(cuda_lib, x, torch.full((4,), 7, device="cuda"), 20)
    for r in range(4):
        _check_score(cuda_lib, x[r:r + 1], torch.full((1,), 7, device="cuda"), 20)
    # the teacher's entries where the student has probability
    ids = x.float().argmax(1, keepdim=True).int().repeat(1, 2)
    _check_distill(cuda_lib, x[[0, 1, 3]], ids[[0, 1, 3]], torch.zeros(3, 2, device="cuda"), torch.ones(3, device="cuda"), 1.0)


@pytest.mark.parametrize("V", [900, 8000, 70000])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_score_large_entries_in_few_places(cuda_lib, V, dtype):
    """Thousands of large entries, all in the words of fewer threads than k (of blocks of 128 or 256, or the
    lanes of a warp), largest last, and with many equal ones at the k-th place."""
    randn, rand = _gen(V + 1)
    i = torch.arange(V, device="cuda")
    words = i // (8 if dtype == torch.bfloat16 else 4)
    rows = []
    for T, few in ((256, 8), (128, 24), (512, 20), (32, 5)):
        big = words % T < few
        rows += [torch.where(big, 5 + 3 * i / V, randn(V)), torch.where(big, 5 + 3 * rand(V), randn(V)), torch.where(big, 7.0, randn(V)),
                 torch.where(big, 5 + torch.round(2 * rand(V)), randn(V)), torch.where(big, -1.0, -math.inf), torch.where(big, randn(V), -math.inf)]
    x = torch.stack(rows).to(dtype)
    for k in (1, 9, 40, 64):
        _check_score(cuda_lib, x, _tokens(len(rows), V), k)
        _check_score(cuda_lib, x[6:7], _tokens(1, V) + 3, k)


@pytest.mark.parametrize("V", [40, 900, 3000, 40000])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_score_rows_without_a_distribution(cuda_lib, V, dtype):
    """Nothing but -inf: -inf and 0, ids in order.  NaN and +inf: NaN, in their rows alone, and the largest
    entries in the documented order."""
    randn, _ = _gen(V)
    x = randn(7, V).to(dtype)
    x[1] = -math.inf
    x[2, 5] = math.nan
    x[3, 7], x[3, 30] = math.inf, math.inf
    x[4] = math.nan
    x[5, 3], x[5, 11], x[5, 20] = -math.inf, math.nan, math.inf
    keep = [0, 6]
    k = 32
    for rows in (slice(0, 7), slice(1, 2), slice(2, 3), slice(3, 4), slice(4, 5), slice(5, 6)):
        sub, tok = x[rows], torch.full((x[rows].shape[0],), 9, device="cuda")
        logp, ent, lse, ids, top = _score(cuda_lib, sub, tok, k)
        for j, r in enumerate(range(7)[rows]):
            key = torch.where(x[r].isnan(), torch.full((), 4e38, dtype=torch.float64, device="cuda"), x[r].double().clamp(max=3.9e38))
            assert torch.equal(ids[j], _top(key[None], k)[0]), r
            if r == 1:
                assert lse[j] == -math.inf and logp[j] == -math.inf and ent[j] == 0 and torch.all(top[j] == -math.inf)
            elif r in (2, 3, 4, 5):
                assert all(t[j].isnan().all() for t in (lse, logp, ent, top))
    _check_score(cuda_lib, x[keep], _tokens(2, V), k)
    pad = _score(cuda_lib, x, torch.full((7,), -1, device="cuda"), 0)[0]
    assert torch.all(pad == 0)


@pytest.mark.parametrize("V", [3, 100, 1023, 1030, 8195, 20001])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_at_every_address(cuda_lib, V, dtype):
    """Rows that start at every element of a 16-byte word, strided, between NaN: nothing else read or written."""
    bl = cuda_lib
    randn, _ = _gen(V)
    n, k = 5, min(V, 9)
    x0 = randn(n, V).to(dtype)
    ids, top, w = _teacher(n, V, 4, V)
    for off in range(8):
        ld = V + (0, 3, 8)[off % 3]
        buf, dbuf = (torch.full((n * ld + 17,), math.nan, dtype=dtype, device="cuda") for _ in range(2))
        x = buf[off:off + n * ld].as_strided((n, V), (ld, 1), off)
        x.copy_(x0)
        _check_score(bl, x, _tokens(n, V), k)
        for doff, dld in ((off, ld), ((off * 3 + 1) % 8, ld + 1)):
            dbuf = torch.full((n * dld + 17,), math.nan, dtype=dtype, device="cuda")
            d = dbuf[doff:].as_strided((n, V), (dld, 1), doff)
            _check_distill(bl, x, ids, top, w, 1.5, d=d)
            assert int(dbuf.isnan().sum()) == dbuf.numel() - n * V
        assert int(buf.isnan().sum()) == buf.numel() - n * V


def _teacher(n, V, k, seed, repeat=False):
    randn, rand = _gen(seed + 1)
    ids = torch.argsort(rand(n, V), 1)[:, :k] if n * V < 1 << 22 else (torch.arange(n, device="cuda")[:, None] * 31 + torch.arange(k, device="cuda") * (V // k)) % V
    if ids.shape[1] < k:
        ids = ids.repeat(1, -(-k // ids.shape[1]))[:, :k]
    if repeat and k > 3:
        ids[:, 2] = ids[:, 0]
        ids[:, k - 1] = ids[:, 0]
    return ids.to(torch.int32).contiguous(), randn(n, k) * 2, rand(n) + 0.1


def _distill_ref(x, ids, top, w, T):
    """loss, lse, dlogits in fp64 with their bounds, and what the gradient's bound has from its own lse."""
    x, ids, top, w = x.double(), ids.long(), top.double(), w.double()[:, None]
    n, V = x.shape
    ok = (ids >= 0) & (ids < V) & (top != -math.inf)
    live = ok.any(1, keepdim=True) & (w != 0)
    t = torch.where(ok, top / T, -math.inf)
    tm = t.amax(1, keepdim=True)
    p = torch.where(ok & live, torch.softmax(t, 1), torch.zeros_like(t))
    rp = 2.0 ** -20 + 4 * U * torch.where(ok, (tm - t).abs() + tm.abs(), torch.zeros_like(t)).nan_to_num(0)   # of each p, relative
    m, z, logS, q, A, E = _stats(x, T)
    at = ids.clamp(0, V - 1)
    lq = z.gather(1, at) - logS
    logp = torch.where(p > 0, p, torch.ones_like(p)).log()
    zero = torch.zeros_like(p)
    terms = torch.where(p > 0, p * (logp - lq), zero)
    tol = torch.where(p > 0, p * ((rp + 4 * U) * (logp.abs() + lq.abs() + 1) + E + 4 * U * (logS.abs() + z.gather(1, at).abs())), zero)
    c = w * T * T
    d0 = torch.zeros_like(x)
    loss = torch.where(live, c * terms.sum(1, keepdim=True), d0[:, :1])[:, 0]
    loss_tol = torch.where(live, c * (tol.sum(1, keepdim=True) + 40 * U * terms.abs().sum(1, keepdim=True)), d0[:, :1])[:, 0]
    lse = torch.where(live, m / T + logS, d0[:, :1])[:, 0]
    lse_tol = torch.where(live, E + 3 * U * ((m / T).abs() + logS.abs()), d0[:, :1])[:, 0]
    dense, dtol = d0.scatter_add(1, at, p), d0.scatter_add(1, at, p * (rp + U))
    qt = torch.where(q > 0, q * (E + 2.0 ** -21 + 4 * U * z.abs()), d0) + 2.0 ** -125
    d = torch.where(live, w * T * (q - dense), d0)
    d_tol = torch.where(live, w * T * (qt + dtol) + 3 * U * w * T * (q + dense), d0)
    return loss, loss_tol, lse, lse_tol, d, d_tol, live


def _check_distill(bl, x, ids, top, w, T, d=None, place=False):
    n = x.shape[0]
    ref = _distill_ref(x, ids, top, w, T)
    loss, lse = torch.full((n,), 77.0, device="cuda"), torch.full((n,), 77.0, device="cuda")
    keep = x.clone()
    bl.tern_distill(x, ids, top, loss, lse=lse, weight=w, temperature=T)
    _close(loss, ref[0], ref[1], "loss")
    _close(lse, ref[2], ref[3], "lse")
    d = torch.full_like(x, 5.0) if d is None else d
    loss2 = torch.empty_like(loss)
    bl.tern_distill(x, ids, top, loss2, dlogits=d, weight=w, temperature=T)
    _close(loss2, ref[0], ref[1], "loss with the gradient")
    _close(d, ref[4], ref[5], "dlogits")
    # from lse: its rounding and x / T's are in the exponent
    xa = torch.where(x > -math.inf, x.double().abs() / T, torch.zeros((), dtype=torch.float64, device="cuda"))
    live = ref[6]
    q = torch.where(live, (x.double() / T - ref[2][:, None]).exp(), torch.zeros_like(xa))
    extra = w.double()[:, None] * T * q * (4 * U * (xa + ref[2].abs()[:, None]) + ref[3][:, None])
    d2 = torch.full_like(x, 5.0)
    bl.tern_distill_bwd(x, ids, top, lse, d2, weight=w, temperature=T)
    _close(d2, ref[4], ref[5] + extra, "dlogits from lse")
    if place:
        y, again = x.clone(), torch.empty_like(loss)
        bl.tern_distill(y, ids, top, again, dlogits=y, weight=w, temperature=T)
        assert torch.equal(again, loss2) and torch.equal(y, d)
        y = x.clone()
        bl.tern_distill_bwd(y, ids, top, lse, y, weight=w, temperature=T)
        assert torch.equal(y, d2)
    assert torch.equal(x, keep)


@pytest.mark.parametrize("n,V,k", [(1, 1, 1), (3, 5, 3), (9, 64, 64), (70, 256, 16), (6, 257, 1), (5, 1000, 256), (4, 1024, 8), (700, 1025, 7), (2500, 1300, 40), (1300, 9001, 12), (700, 50001, 6), (3, 2050, 33),
                                   (33, 8192, 20), (2, 8193, 64), (350, 16411, 5), (1, 50000, 200), (3, 100003, 64), (1, 262145, 3)])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_distillation(cuda_lib, n, V, k, dtype):
    randn, _ = _gen(n + V)
    x = (randn(n, V) * 3 + randn(V)).to(dtype)
    ids, top, w = _teacher(n, V, k, V + k, repeat=True)
    for T in (1.0, 2.5):
        _check_distill(cuda_lib, x, ids, top, w, T, place=True)


@pytest.mark.parametrize("V", [50, 700, 5000, 30000])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_distillation_of_uneven_rows(cuda_lib, V, dtype):
    """Entries left out, rows without any, rows of weight 0 that hold NaN, ids of both kinds, masked students."""
    bl = cuda_lib
    randn, rand = _gen(V)
    n, k = 12, 6
    x = (randn(n, V) * 2).to(dtype)
    ids, top, w = _teacher(n, V, k, V)
    x[8] = x[8].masked_fill(rand(V) < 0.5, -math.inf)
    ids[8] = x[8].float().argmax().int()                      # one id, all of the probability
    ids[0, 1], ids[1, 0], ids[2] = -1, V, -1
    top[3, 2], top[4] = -math.inf, -math.inf
    w[5] = 0.0
    x[2], x[4], x[5] = math.nan, math.inf, math.nan           # rows that do not count
    good = torch.ones(n, dtype=torch.bool)
    good[[2, 4, 5]] = False
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    for kind in (torch.int32, torch.int64):
        d, d2 = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
        bl.tern_distill(x, ids.to(kind), top, loss, lse=lse, dlogits=d, weight=w, temperature=1.3)
        bl.tern_distill_bwd(x, ids.to(kind), top, lse, d2, weight=w, temperature=1.3)
        for r in (2, 4, 5):
            assert loss[r] == 0 and lse[r] == 0 and not d[r].any() and not d2[r].any()
        _check_distill(bl, x[good], ids[good].to(kind), top[good], w[good], 1.3)
        ref = _distill_ref(x[good], ids[good], top[good], w[good], 1.3)
        _close(d[good], ref[4], ref[5], "dlogits")
    # a student that gives a teacher's entry no probability, and rows with NaN
    x[0, ids[0, 0].long()] = -math.inf
    x[1, 3] = math.nan
    bl.tern_distill(x, ids, top, loss, dlogits=d, weight=w)
    assert loss[0] == math.inf and d[0].isfinite().all() and loss[1].isnan() and d[1].isnan().all() and loss[3].isfinite()


@pytest.mark.parametrize("n,V", [(20, 256), (7, 1500), (3, 20000)])
def test_cross_entropy(cuda_lib, n, V):
    """One entry a row: cross entropy, with or without a logit of it."""
    bl = cuda_lib
    randn, _ = _gen(V)
    x = randn(n, V)
    tok = torch.arange(n, device="cuda") * 13 % V
    loss, d = torch.empty(n, device="cuda"), torch.empty_like(x)
    bl.tern_distill(x, tok[:, None], None, loss, dlogits=d)
    other, d2 = torch.empty_like(loss), torch.empty_like(x)
    bl.tern_distill(x, tok[:, None], randn(n, 1), other, dlogits=d2, weight=torch.ones(n, device="cuda"))
    assert torch.equal(loss, other) and torch.equal(d, d2)
    ref = _distill_ref(x, tok[:, None], torch.zeros(n, 1, device="cuda"), torch.ones(n, device="cuda"), 1.0)
    _close(loss, ref[0], ref[1], "loss")
    _close(d, ref[4], ref[5], "dlogits")
    logp = torch.empty(n, device="cuda")
    bl.tern_score(x, tok, logp)
    assert (loss + logp).abs().max() <= 2 * float(ref[1].max()) + 4 * U * float(ref[0].max())


def test_gradient_against_differences(cuda_lib):
    """dlogits against differences of the losses' definition in fp64."""
    randn, _ = _gen(4)
    x = randn(3, 40)
    ids, top, w = _teacher(3, 40, 5, 9, repeat=True)
    loss, d = torch.empty(3, device="cuda"), torch.empty_like(x)
    cuda_lib.tern_distill(x, ids, top, loss, dlogits=d, weight=w, temperature=1.7)
    total = lambda x: float(_distill_ref(x, ids, top, w, 1.7)[0].sum())  # noqa: E731
    for s in range(6):
        v = torch.randn(3, 40, generator=torch.Generator().manual_seed(s), dtype=torch.float64).cuda()
        diff = (total(x.double() + 1e-4 * v) - total(x.double() - 1e-4 * v)) / 2e-4
        # third-order term at steps of 1e-4, and fp32's roundings of d
        assert abs(diff - float((v * d.double()).sum())) <= 1e-5 * float((v * d.double()).abs().sum())


def test_far_logits(cuda_lib):
    """Logits around 1000 and -1000, and a spread of 300: only differences count."""
    randn, _ = _gen(2)
    for V in (200, 3000, 20000):
        x = torch.stack([randn(V) + 1000, randn(V) - 1000, randn(V) * 100])
        _check_score(cuda_lib, x, _tokens(3, V), 8)
        ids, top, w = _teacher(3, V, 4, V)
        _check_distill(cuda_lib, x, ids, top, w, 1.0)


def test_same_bits_streams_and_graphs(cuda_lib):
    bl = cuda_lib
    for n, V in ((40, 256), (300, 3000), (2, 100003)):
        randn, _ = _gen(V)
        x, x2 = (randn(n, V) * 2).bfloat16(), (randn(n, V) * 2).bfloat16()
        tok = _tokens(n, V)
        ids, top, w = _teacher(n, V, 8, V)
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        outs = [f32(n), f32(n), f32(n), torch.empty(n, 9, dtype=torch.int32, device="cuda"), f32(n, 9), f32(n), torch.empty_like(x)]
        score = bl.Score(x, tok, outs[0], outs[1], outs[2], outs[3], outs[4])
        train = bl.Distill(x, ids, top, outs[5], dlogits=outs[6], weight=w, temperature=2.0)

        def run():
            score()
            train()
            return [t.clone() for t in outs]
        want = run()
        for _ in range(3):
            assert all(torch.equal(p, q) for p, q in zip(want, run()))
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = run()
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            score()
            train()
        x.copy_(x2)
        want = run()
        for t in outs:
            t.zero_()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, outs))


def test_offsets_past_32_bits(cuda_lib):
    """Rows behind 2^32 bytes: 22000 rows of 100003 in bf16, the last ones against the formulas."""
    bl = cuda_lib
    n, V, k = 22000, 100003, 4
    x = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    for i, part in enumerate(x.split(2000)):
        part.normal_(generator=torch.Generator(device="cuda").manual_seed(i))
    tok = _tokens(n, V)
    ids = (torch.arange(n, device="cuda")[:, None] * 17 + torch.arange(k, device="cuda") * 20000).to(torch.int32) % V
    top, w = torch.ones(n, k, device="cuda"), torch.ones(n, device="cuda")
    logp, _, lse, tids, tlogp = _score(bl, x, tok, k)
    loss, d = torch.empty(n, device="cuda"), torch.empty_like(x)
    bl.tern_distill(x, ids, top, loss, dlogits=d, weight=w)
    for r in (slice(0, 3), slice(n - 3, n)):
        m, z, logS, _, _, E = _stats(x[r].double())
        _close(lse[r], (m + logS)[:, 0], (E + 2 * U * (m.abs() + logS.abs()))[:, 0], "lse")
        assert torch.equal(tids[r], _top(x[r].double(), k))
        ref = _distill_ref(x[r], ids[r], top[r], w[r], 1.0)
        _close(loss[r], ref[0], ref[1], "loss")
        _close(d[r], ref[4], ref[5], "dlogits")


def test_refusals(cuda_lib):
    bl = cuda_lib
    x, v = torch.zeros(4, 80, device="cuda"), torch.zeros(4, device="cuda")
    ids, top = torch.zeros(4, 3, dtype=torch.int32, device="cuda"), torch.zeros(4, 3, device="cuda")
    with pytest.raises(ValueError):
        bl.tern_score(x, logp=v)                               # no tokens
    with pytest.raises(ValueError):
        bl.tern_score(x, top_ids=ids)                          # ids without log probabilities
    with pytest.raises(TypeError):
        bl.tern_score(x.half(), entropy=v)
    with pytest.raises(TypeError):
        bl.tern_score(x, torch.zeros(4, device="cuda"), logp=v)
    with pytest.raises(ValueError):
        bl.tern_score(x, entropy=v[:3])
    for k in (65, 81):
        with pytest.raises(bl.TernError):
            bl.tern_score(x, top_ids=torch.zeros(4, k, dtype=torch.int32, device="cuda"), top_logp=torch.zeros(4, k, device="cuda"))
    with pytest.raises(ValueError):
        bl.tern_distill(x, ids, top[:, :2].contiguous(), v)
    with pytest.raises(TypeError):
        bl.tern_distill(x, ids, top, v, dlogits=torch.zeros(4, 80, dtype=torch.bfloat16, device="cuda"))
    for T in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(bl.TernError):
            bl.tern_distill(x, ids, top, v, temperature=T)
    with pytest.raises(bl.TernError):
        bl.tern_distill(x, ids, None, v)                       # three entries without logits
    with pytest.raises(bl.TernError):
        bl.tern_distill(x, torch.zeros(4, 257, dtype=torch.int32, device="cuda"), torch.zeros(4, 257, device="cuda"), v)
    with pytest.raises(bl.TernError):
        bl.tern_distill(x, ids, top, v, dlogits=torch.zeros(1, 80, device="cuda").expand(4, 80))
    with pytest.raises(bl.TernError):
        bl.tern_distill(torch.zeros(8, 40, device="cuda").as_strided((4, 40), (80, 1)), ids, top, v, dlogits=torch.zeros(1, 40, device="cuda").expand(4, 40))
