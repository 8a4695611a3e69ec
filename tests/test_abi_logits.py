"""Argument checks of the score and distillation calls, without a GPU: each returns its status before
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


def test_score_checks(lib):
    f = lib.lib.tern_score

    def call(x=P(0x10000), dt=lib.TERN_BF16, ld=100, n=4, V=100, tok=P(0x20000), tk=lib.TERN_I64, logp=P(0x30000), ent=None, lse=None, k=5,
             ids=P(0x40000), top=P(0x50000)):
        return f(x, dt, ld, n, V, tok, tk, logp, ent, lse, k, ids, top, None)

    assert call(n=0) == lib.TERN_OK
    for kw in (dict(x=None), dict(dt=lib.TERN_I32), dict(ld=99), dict(n=-1), dict(n=1 << 27), dict(V=0), dict(V=1 << 31, ld=1 << 31), dict(tok=None),
               dict(tk=lib.TERN_F32), dict(k=-1), dict(k=65), dict(V=4, k=5), dict(ids=None), dict(top=None), dict(ld=1 << 41)):
        assert call(**kw) == lib.TERN_ERR_ARG, kw
    for kw in (dict(x=P(0x10001)), dict(dt=lib.TERN_F32, x=P(0x10002)), dict(tok=P(0x20004)), dict(logp=P(0x30002)), dict(ent=P(0x30001)),
               dict(lse=P(0x30002)), dict(ids=P(0x40002)), dict(top=P(0x50002))):
        assert call(**kw) == lib.TERN_ERR_ALIGN, kw


def test_distillation_checks(lib):
    fwd, bwd = lib.lib.tern_distill, lib.lib.tern_distill_bwd

    def make(x=P(0x10000), ld=100, n=4, V=100, dt=lib.TERN_F32, tk=lib.TERN_I32, ids=P(0x20000), top=P(0x30000), k=5, T=1.0, w=None):
        return ctypes.byref(lib._Distillation(x, ld, n, V, dt, tk, ids, top, k, T, w))

    def call(loss=P(0x40000), lse=None, d=None, ldd=100, **kw):
        return fwd(make(**kw), loss, lse, d, ldd, None)

    def back(lse=P(0x50000), d=P(0x60000), ldd=100, **kw):
        return bwd(make(**kw), lse, d, ldd, None)

    assert call(n=0) == lib.TERN_OK and back(n=0) == lib.TERN_OK and call(n=0, loss=None) == lib.TERN_OK
    assert fwd(None, P(0x40000), None, None, 0, None) == lib.TERN_ERR_ARG and bwd(None, P(0x40000), P(0x50000), 100, None) == lib.TERN_ERR_ARG
    assert call(loss=None) == lib.TERN_ERR_ARG and back(lse=None) == lib.TERN_ERR_ARG and back(d=None) == lib.TERN_ERR_ARG
    nan = float("nan")
    for kw in (dict(x=None), dict(ld=99), dict(n=-1), dict(n=1 << 27), dict(V=0), dict(dt=lib.TERN_I32), dict(tk=lib.TERN_F32), dict(ids=None),
               dict(top=None), dict(k=0), dict(k=257), dict(T=0.0), dict(T=-1.0), dict(T=nan), dict(T=float("inf")), dict(T=1e-7)):
        assert call(**kw) == lib.TERN_ERR_ARG, kw
        assert back(**kw) == lib.TERN_ERR_ARG, kw
    assert call(d=P(0x60000), ldd=99) == lib.TERN_ERR_ARG and back(ldd=99) == lib.TERN_ERR_ARG
    assert call(d=P(0x10000), ldd=101) == lib.TERN_ERR_ARG                # in place, at another stride
    for kw in (dict(x=P(0x10002)), dict(ids=P(0x20002)), dict(tk=lib.TERN_I64, ids=P(0x20004)), dict(top=P(0x30001)), dict(w=P(0x70002))):
        assert call(**kw) == lib.TERN_ERR_ALIGN, kw
        assert back(**kw) == lib.TERN_ERR_ALIGN, kw
    assert call(loss=P(0x40001)) == lib.TERN_ERR_ALIGN and call(lse=P(0x40002)) == lib.TERN_ERR_ALIGN and back(d=P(0x60002)) == lib.TERN_ERR_ALIGN
