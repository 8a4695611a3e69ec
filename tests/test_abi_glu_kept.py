"""The gated layer's gradient from kept factors reads neither the activation nor K, without a GPU: no value of
either is refused."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._builder().build()
    import bit_linear_gb300 as bl
    return bl


def test_activation_and_width_are_not_read(lib):
    f = lib.lib.tern_glu_bwd

    def call(saved, act=0, K=32, M=0):
        return f(P(0x10000), saved, None, None, None, act, P(0x30000), M, K, 48, None)

    kept = P(0x40000)
    for kw in (dict(act=-1), dict(act=4), dict(act=1 << 30), dict(K=0), dict(K=-5), dict(K=1 << 40), dict(act=99, K=7)):
        assert call(kept, **kw) == lib.TERN_OK, kw
        assert call(None, **kw) in (lib.TERN_ERR_ARG, lib.TERN_ERR_ALIGN), kw
    assert call(kept, M=-1) == lib.TERN_ERR_ARG
