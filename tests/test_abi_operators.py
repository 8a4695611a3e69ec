"""Sizes and argument checks of the embedding, recurrence and orthogonalise calls, without a GPU:
each returns its status before touching the device."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._builder().build()
    import bit_linear_gb300 as bl
    return bl


def test_sizes(lib):
    assert lib.tern_scan_saved(3, 65, 10) == 3 * 2 * 10 * 4          # a state every 64 rows
    assert lib.tern_scan_saved(3, 64, 10) == 3 * 1 * 10 * 4
    assert lib.tern_scan_saved(3, 0, 10) == 0 and lib.tern_scan_saved(-1, 5, 5) == 0
    assert lib.tern_scan_bwd_workspace(2, 100, 7) == 2 * 16 * 7 * 4  # up to 16 blocks a sequence
    for n, V, D in ((0, 1, 1), (1, 256, 8), (200000, 100003, 64)):
        assert lib.tern_embed_bwd_workspace(n, V, D) >= 16 * n + V
    assert lib.tern_embed_bwd_workspace(-1, 5, 5) == 0 and lib.tern_embed_bwd_workspace(5, 0, 5) == 0
    assert lib.tern_embed_bwd_workspace(5, 5, 1 << 23) == 0
    K, N = 100, 37
    planes = 4 * (K * 40 * 2) + 4 * (37 * 40 * 2)                    # two X, A and M, rows rounded up to eight
    assert planes <= lib.tern_orthogonalize_workspace(K, N) <= planes + 8192
    assert lib.tern_orthogonalize_workspace(0, 5) == 0 and lib.tern_orthogonalize_workspace(1 << 30, 5) == 0
    # from 1024 rows and 1.5 times as many columns two more matrices, for steps two at a time
    small, large = lib.tern_orthogonalize_workspace(1024, 1528), lib.tern_orthogonalize_workspace(1024, 1536)
    assert large - small > 4 * 1024 * 1024 * 2


def test_embed_argument_checks(lib):
    f = lib.lib.tern_embed_fwd
    tok, tab, out = P(0x10000), P(0x20000), P(0x30000)
    ok = lambda n=4, V=5, D=8, ld=8, tk=lib.TERN_I64, tb=lib.TERN_F32, t=tok, w=tab, o=out: f(t, tk, w, tb, n, V, D, 1.0, o, ld, None)  # noqa: E731
    assert ok(n=0) == lib.TERN_OK and ok(D=0, ld=0) == lib.TERN_OK   # nothing to do
    for kw in (dict(n=-1), dict(V=0), dict(D=-1), dict(ld=7), dict(tk=lib.TERN_BF16), dict(tb=lib.TERN_I32), dict(t=None), dict(w=None),
               dict(o=None), dict(n=1 << 31), dict(V=1 << 31), dict(D=1 << 23, ld=1 << 23)):
        assert ok(**kw) == lib.TERN_ERR_ARG, kw
    for kw in (dict(t=P(0x10004)), dict(w=P(0x20002)), dict(o=P(0x30001))):
        assert ok(**kw) == lib.TERN_ERR_ALIGN, kw
    g = lib.lib.tern_embed_bwd
    need = lib.tern_embed_bwd_workspace(4, 5, 8)
    back = lambda n=4, ld=8, acc=0, t=tok, d=out, dt=tab, ws=P(0x40000), nb=need, tk=lib.TERN_I32: g(  # noqa: E731
        t, tk, d, ld, n, 5, 8, 1.0, acc, dt, ws, nb, None)
    assert back(n=0, acc=1) == lib.TERN_OK
    for kw in (dict(ld=7), dict(tk=9), dict(t=None), dict(d=None), dict(dt=None)):
        assert back(**kw) == lib.TERN_ERR_ARG, kw
    assert back(nb=need - 1) == lib.TERN_ERR_WORKSPACE and back(ws=None) == lib.TERN_ERR_WORKSPACE
    for kw in (dict(ws=P(0x40008)), dict(t=P(0x10002)), dict(dt=P(0x20002)), dict(d=P(0x30001))):
        assert back(**kw) == lib.TERN_ERR_ALIGN, kw


def _scan(lib, B=2, T=10, D=8, dtype=None, f=0x10000, bias=0x20000, lengths=None, stride=80):
    act = lambda p: lib._Act(P(p), stride, 8)  # noqa: E731
    return lib._Scan(act(f), act(0x11000), act(0x12000), P(bias), P(lengths) if lengths else None, None, B, T, D,
                     lib.TERN_F32 if dtype is None else dtype)


def test_scan_argument_checks(lib):
    f, g = lib.lib.tern_scan_fwd, lib.lib.tern_scan_bwd
    y = lib._Act(P(0x30000), 80, 8)
    big = 1 << 20
    fwd = lambda s, y=y, saved=P(0x50000), nb=big, h0=None: f(  # noqa: E731
        None if s is None else ctypes.byref(s), h0, None if y is None else ctypes.byref(y), None, saved, nb, None)
    assert fwd(_scan(lib, B=0)) == lib.TERN_OK and fwd(_scan(lib, D=0)) == lib.TERN_OK
    for s in (None, _scan(lib, B=-1), _scan(lib, T=-1), _scan(lib, D=-1), _scan(lib, dtype=lib.TERN_I32), _scan(lib, T=1 << 31), _scan(lib, f=0),
              _scan(lib, stride=-1), _scan(lib, stride=1 << 62)):
        assert fwd(s) == lib.TERN_ERR_ARG
    assert fwd(_scan(lib), y=None) == lib.TERN_ERR_ARG
    assert fwd(_scan(lib), nb=lib.tern_scan_saved(2, 10, 8) - 1) == lib.TERN_ERR_WORKSPACE
    for s in (_scan(lib, f=0x10002), _scan(lib, bias=0x20002), _scan(lib, lengths=0x20001)):
        assert fwd(s) == lib.TERN_ERR_ALIGN
    assert fwd(_scan(lib), h0=P(0x60002)) == lib.TERN_ERR_ALIGN
    a = [ctypes.byref(lib._Act(P(0x70000 + 0x1000 * i), 80, 8)) for i in range(4)]
    bwd = lambda s, saved=P(0x50000), acts=a, dbias=P(0x80000), ws=P(0x90000), nb=big: g(  # noqa: E731
        ctypes.byref(s), saved, acts[0], None, *acts[1:], dbias, None, ws, nb, None)
    assert bwd(_scan(lib), saved=None) == lib.TERN_ERR_ARG
    assert bwd(_scan(lib), acts=[a[0], a[1], None, a[3]]) == lib.TERN_ERR_ARG
    assert bwd(_scan(lib, B=0)) == lib.TERN_ERR_ARG                  # dbias of no sequences
    assert bwd(_scan(lib, B=0), dbias=None) == lib.TERN_OK
    assert bwd(_scan(lib), ws=None) == lib.TERN_ERR_WORKSPACE
    assert bwd(_scan(lib), nb=lib.tern_scan_bwd_workspace(2, 10, 8) - 1) == lib.TERN_ERR_WORKSPACE
    assert bwd(_scan(lib), dbias=P(0x80002)) == lib.TERN_ERR_ALIGN
    st = lib.lib.tern_scan_step
    step = lambda s, h=P(0x60000), o=P(0x60000), y=y: st(ctypes.byref(s), h, o, ctypes.byref(y) if y else None, None)  # noqa: E731
    assert step(_scan(lib)) == lib.TERN_ERR_ARG                      # T is not 1
    assert step(_scan(lib, T=1, lengths=0x20000)) == lib.TERN_ERR_ARG
    assert step(_scan(lib, T=1), h=None) == lib.TERN_ERR_ARG and step(_scan(lib, T=1), y=None) == lib.TERN_ERR_ARG
    assert step(_scan(lib, T=1), o=P(0x60001)) == lib.TERN_ERR_ALIGN
    assert step(_scan(lib, T=1, B=0)) == lib.TERN_OK


def test_orthogonalize_argument_checks(lib):
    f = lib.lib.tern_orthogonalize
    need = lib.tern_orthogonalize_workspace(16, 24)
    call = lambda G=P(0x10000), K=16, N=24, steps=5, eps=1e-7, out=P(0x20000), ws=P(0x30000), nb=need: f(  # noqa: E731
        G, K, N, steps, eps, 1.0, out, ws, nb, None)
    assert call(K=0) == lib.TERN_OK and call(N=0) == lib.TERN_OK
    for kw in (dict(G=None), dict(out=None), dict(K=-1), dict(steps=0), dict(steps=65), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(N=1 << 30)):
        assert call(**kw) == lib.TERN_ERR_ARG, kw
    assert call(ws=None) == lib.TERN_ERR_WORKSPACE and call(nb=need - 1) == lib.TERN_ERR_WORKSPACE
    for kw in (dict(G=P(0x10002)), dict(out=P(0x20001)), dict(ws=P(0x30040))):
        assert call(**kw) == lib.TERN_ERR_ALIGN, kw
