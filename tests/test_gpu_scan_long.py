"""Long runs of the recurrence: clusters that take many steps each, so that the two buffers of the
exchange, their phases and the ring of copies are used again and again; against the fp64 reference,
and the same bits from every repeat."""
import numpy as np
import pytest
import torch

from test_gpu_scan import Case, _starts

pytestmark = pytest.mark.gpu


def _repeats(case, times=3):
    first = {k: x.clone() for k, x in case.outputs().items()}
    for _ in range(times):
        for x in (case.saved, case.ws, *case.outputs().values()):
            x.fill_(float("nan"))
        case.run()
        for k, x in case.outputs().items():
            assert torch.equal(x, first[k]), k


# tiles of half the channels in clusters of 16: seven and thirteen steps a block; clusters of two
# eight-warp blocks: six and twelve; eight-warp blocks of odd widths
@pytest.mark.parametrize("B,T,D,dtype", [(1, 25000, 64, torch.bfloat16), (1, 25000, 33, torch.float32), (40, 3000, 64, torch.bfloat16),
                                         (20, 3000, 64, torch.float32), (7, 5000, 131, torch.bfloat16)])
def test_many_steps_of_a_cluster(cuda_lib, B, T, D, dtype):
    c = Case(cuda_lib, B, T, D, dtype, seed=D + B).run().check()
    _repeats(c)
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


@pytest.mark.parametrize("B,T,D,dtype", [(2, 25000, 64, torch.float32), (2, 25000, 33, torch.bfloat16), (40, 3000, 64, torch.bfloat16),
                                         (20, 3000, 64, torch.float32)])
def test_many_steps_with_padding_and_documents(cuda_lib, B, T, D, dtype):
    """Sequences that end early leave whole steps of their clusters without a live row."""
    lengths = np.random.default_rng(B).integers(0, T + 1, B)
    lengths[:2] = 9001 if T > 10000 else 0, T
    c = Case(cuda_lib, B, T, D, dtype, seed=D, lengths=lengths.tolist(), starts=_starts(B, T, D, 0.002)).run().check()
    _repeats(c)
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK
