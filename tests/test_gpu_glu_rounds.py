"""The gated layer's GEMM with several tiles a block (or pair of blocks): both accumulators in turn, their
release by the epilogue while the next tile's products run, and stages carried over from tile to tile; in
each of its four tile forms, forward with and without factors and the recomputed gradient.  The bounds are
those of tests/test_gpu_glu.py."""
import pytest
import torch

from test_gpu_glu import ACTS, _inputs, _near, _new, _ref, _tiles

pytestmark = pytest.mark.gpu


def _form(M, N, sms):
    """(blocks, outputs) of a tile and the tiles of the busiest, as the launch chooses them."""
    cg = 2 if M > 128 else 1
    units = sms // cg
    wide, narrow = (-(-(-(-M // (128 * cg)) * -(-N // hn)) // units) for hn in (128, 64))
    return ((cg, 64), narrow) if narrow * 5 < wide * 9 else ((cg, 128), wide)


@pytest.mark.parametrize("M,K,N,form", [(8192, 80, 1360, (2, 128)), (4100, 528, 2064, (2, 128)), (20000, 16, 512, (2, 128)),
                                        (80000, 80, 64, (2, 64)), (40000, 144, 192, (2, 64)), (60001, 1040, 48, (2, 64)),
                                        (40, 64, 58000, (1, 128)), (128, 272, 57920, (1, 128)), (40, 64, 40976, (1, 64)), (100, 336, 40960, (1, 64))])
def test_several_tiles_a_block(cuda_lib, M, K, N, form):
    bl = cuda_lib
    got, rounds = _form(M, N, torch.cuda.get_device_properties(0).multi_processor_count)
    assert got == form and rounds > 2
    X, q, scale, dH = _inputs(M, K, N, M + K + N)
    tiles = _tiles(bl, q, scale, packed=False)
    d = dH.double()
    for act in ACTS if K == 80 else ACTS[:2]:
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
        dY, guard4 = _new(M, 2 * N)
        bl.tern_glu_bwd(dH, dY, X=X, tiles=tiles, scale=scale, act=act)
        _near(dY[:, :N], fg[0] * d, fg[1] * d.abs(), 1, "dG")
        _near(dY[:, N:], fu[0] * d, fu[1] * d.abs(), 1, "dU")
        again, _ = _new(M, 2 * N)
        bl.tern_glu_bwd(dH, again, X=X, tiles=tiles, scale=scale, act=act)
        assert torch.equal(again, dY)
        assert all(torch.all(t == 99.0) for t in (guard, guard2, guard3, guard4))
    assert bl.tern_device_status() == bl.TERN_OK
