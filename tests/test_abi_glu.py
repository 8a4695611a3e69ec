"""Argument checks of the gated feed-forward calls, without a GPU: each returns its status before
touching the device."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._builder().build()
    import bit_linear_gb300 as bl
    return bl


def _tiles(lib, packed=0x50000, t=0x60000):
    return ctypes.byref(lib._Tiles(P(packed) if packed else None, P(t) if t else None, None, None, None, None))


def test_forward_checks(lib):
    f = lib.lib.tern_glu_fwd
    both = _tiles(lib)

    def call(X=P(0x10000), W=both, scale=P(0x20000), act=0, H=P(0x30000), saved=None, M=140, K=32, N=48):
        return f(X, W, scale, act, H, saved, M, K, N, None)

    assert call(M=0) == lib.TERN_OK
    for kw in (dict(X=None), dict(W=None), dict(scale=None), dict(H=None), dict(act=-1), dict(act=4), dict(M=-1), dict(K=0), dict(N=0),
               dict(M=1 << 31), dict(N=1 << 30), dict(W=_tiles(lib, t=0)), dict(M=1, W=_tiles(lib, packed=0, t=0)),
               dict(M=1, saved=P(0x40000), W=_tiles(lib, t=0))):
        assert call(**kw) == lib.TERN_ERR_ARG, kw
    for kw in (dict(K=24), dict(N=40), dict(X=P(0x10008)), dict(scale=P(0x20004)), dict(H=P(0x30008)), dict(saved=P(0x40008)),
               dict(W=_tiles(lib, t=0x60008)), dict(M=1, W=_tiles(lib, packed=0x50004))):
        assert call(**kw) == lib.TERN_ERR_ALIGN, kw


def test_gradient_checks(lib):
    f = lib.lib.tern_glu_bwd
    both = _tiles(lib)

    def call(dH=P(0x10000), saved=None, X=P(0x70000), W=both, scale=P(0x20000), act=0, dY=P(0x30000), M=40, K=32, N=48):
        return f(dH, saved, X, W, scale, act, dY, M, K, N, None)

    kept = dict(saved=P(0x40000), X=None, W=None, scale=None, K=0)
    assert call(M=0) == lib.TERN_OK and call(M=0, **kept) == lib.TERN_OK
    for kw in (dict(dH=None), dict(dY=None), dict(X=None), dict(W=None), dict(scale=None), dict(W=_tiles(lib, t=0)), dict(act=9), dict(K=0),
               dict(kept, dH=None), dict(kept, dY=None), dict(kept, N=0), dict(kept, M=-1)):
        assert call(**kw) == lib.TERN_ERR_ARG, kw
    for kw in (dict(K=40), dict(N=24), dict(dH=P(0x10002)), dict(dY=P(0x30008)), dict(X=P(0x70008)), dict(kept, saved=P(0x40004)), dict(kept, N=24)):
        assert call(**kw) == lib.TERN_ERR_ALIGN, kw
