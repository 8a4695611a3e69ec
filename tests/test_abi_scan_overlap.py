"""Outputs of the recurrence whose rows overlap one another are refused, whatever their strides, and no
others; on the host, before the device is touched."""
import ctypes
import itertools

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._builder().build()
    import bit_linear_gb300 as bl
    return bl


def _overlap(B, T, D, sb, st):
    """The definition: two rows of D elements that share one."""
    at = sorted(b * sb + t * st for b in range(B) for t in range(T))
    return any(y - x < D for x, y in zip(at, at[1:]))


def _scan(lib, B, T, D):
    act = lambda p: lib._Act(P(p), T * D, D)  # noqa: E731
    return lib._Scan(act(0x100000), act(0x200000), act(0x300000), None, None, None, B, T, D, lib.TERN_BF16)


def _fwd(lib, B, T, D, sb, st):
    # `saved` too small: a call whose strides are accepted ends there, still on the host
    y = lib._Act(P(0x400000), sb, st)
    return lib.lib.tern_scan_fwd(ctypes.byref(_scan(lib, B, T, D)), None, ctypes.byref(y), None, P(0x500000), 0, None)


def test_every_pair_of_small_strides(lib):
    for B, T, D in itertools.product((1, 2, 3, 5), (1, 2, 4, 7), (1, 3, 8)):
        for sb, st in itertools.product(range(0, 5 * D + 2), range(0, 8 * D + 2, max(1, D // 3))):
            want = lib.TERN_ERR_ARG if _overlap(B, T, D, sb, st) else lib.TERN_ERR_WORKSPACE
            assert _fwd(lib, B, T, D, sb, st) == want, (B, T, D, sb, st)


def test_large_strides_and_sizes(lib):
    big = 1 << 40
    assert _fwd(lib, 2, 3, 8, big, 8) == _fwd(lib, 2, 3, 8, 8, big) == lib.TERN_ERR_WORKSPACE
    assert _fwd(lib, 4096, 65536, 512, 512, 4096 * 512) == lib.TERN_ERR_WORKSPACE            # [T, B, D] in memory
    assert _fwd(lib, 4096, 65536, 512, 65536 * 1536, 1536) == lib.TERN_ERR_WORKSPACE         # a part of a wider row
    assert _fwd(lib, 4096, 65536, 512, 65536 * 512 - 1, 512) == lib.TERN_ERR_ARG             # one element of the next sequence
    assert _fwd(lib, 1 << 30, 1 << 30, 8, 0, 0) == lib.TERN_ERR_ARG
    assert _fwd(lib, 1 << 30, 1 << 30, 8, 1 << 58, 8) == lib.TERN_ERR_WORKSPACE


def test_every_output_and_no_input(lib):
    B, T, D = 2, 10, 8
    ok, bad = lib._Act(P(0x400000), 80, 8), lib._Act(P(0x400000), 0, 8)      # bad: one tensor for all sequences
    s = _scan(lib, B, T, D)
    ref = ctypes.byref
    for at in range(3):
        outs = [ref(bad if i == at else ok) for i in range(3)]
        assert lib.lib.tern_scan_bwd(ref(s), P(0x500000), ref(ok), None, *outs, P(0x600000), None, None, 0, None) == lib.TERN_ERR_ARG
    # the gradient that comes in may be one for all sequences (the sum of outputs' gradient)
    assert lib.lib.tern_scan_bwd(ref(s), P(0x500000), ref(bad), None, *[ref(ok)] * 3, P(0x600000), None, None, 0,
                                 None) == lib.TERN_ERR_WORKSPACE
    step = _scan(lib, B, 1, D)
    assert lib.lib.tern_scan_step(ref(step), P(0x500000), P(0x500000), ref(bad), None) == lib.TERN_ERR_ARG
    assert lib.lib.tern_scan_step(ref(step), P(0x500000), P(0x500002), ref(ok), None) == lib.TERN_ERR_ALIGN
