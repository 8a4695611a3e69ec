"""Sizes and argument checks of the layer norm calls, without a GPU: each returns its status before
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


def test_sizes(lib):
    f = lib.tern_norm_bwd_workspace
    assert f(1, 512) == 2 * 512 * 4 and f(9, 513) == 2 * 9 * 513 * 4      # the sums of at most a block a row
    assert f(1 << 20, 4096) == 2 * 608 * 4096 * 4                         # at most 608 blocks
    assert f(77, 16385) == 77 * 4
    assert f(0, 512) == 0 and f(-1, 5) == 0 and f(5, (1 << 22) + 1) == 0


def test_forward_checks(lib):
    f = lib.lib.tern_norm_fwd
    B, F = lib.TERN_BF16, lib.TERN_F32

    def call(x=P(0x10000), tx=F, ldx=8, w=None, b=None, n=4, D=8, eps=1e-5, y=P(0x20000), ty=B, ldy=8, mean=None, rstd=None):
        return f(x, tx, ldx, w, b, n, D, eps, y, ty, ldy, mean, rstd, None)

    assert call(n=0) == lib.TERN_OK and call(D=0, ldx=0, ldy=0) == lib.TERN_OK
    for kw in (dict(x=None), dict(y=None), dict(n=-1), dict(D=-1), dict(n=1 << 31), dict(D=(1 << 22) + 1, ldx=1 << 23, ldy=1 << 23),
               dict(ldx=7), dict(ldy=7), dict(ldx=1 << 41), dict(tx=lib.TERN_I32), dict(ty=9), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**kw) == lib.TERN_ERR_ARG, kw
    for kw in (dict(x=P(0x10002)), dict(y=P(0x20001)), dict(w=P(0x30002)), dict(b=P(0x30001)), dict(mean=P(0x30002)), dict(rstd=P(0x30002))):
        assert call(**kw) == lib.TERN_ERR_ALIGN, kw


def test_gradient_checks(lib):
    f = lib.lib.tern_norm_bwd
    B, F = lib.TERN_BF16, lib.TERN_F32
    need = lib.tern_norm_bwd_workspace(4, 8)

    def call(x=P(0x10000), tx=F, ldx=8, w=None, mean=P(0x30000), rstd=P(0x31000), dy=P(0x20000), ty=B, ldy=8, n=4, D=8, dx=P(0x40000),
             lddx=8, dw=P(0x50000), db=None, ws=P(0x60000), nb=need):
        return f(x, tx, ldx, w, mean, rstd, dy, ty, ldy, n, D, dx, lddx, dw, db, ws, nb, None)

    assert call(D=0, ldx=0, ldy=0, lddx=0) == lib.TERN_OK
    for kw in (dict(x=None), dict(dy=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(ldx=7), dict(ldy=7), dict(lddx=7),
               dict(tx=3), dict(ty=2), dict(n=-1)):
        assert call(**kw) == lib.TERN_ERR_ARG, kw
    assert call(ws=None) == lib.TERN_ERR_WORKSPACE and call(nb=need - 1) == lib.TERN_ERR_WORKSPACE
    for kw in (dict(x=P(0x10002)), dict(dy=P(0x20001)), dict(dx=P(0x40002)), dict(dw=P(0x50002)), dict(ws=P(0x60008)), dict(mean=P(0x30001))):
        assert call(**kw) == lib.TERN_ERR_ALIGN, kw
