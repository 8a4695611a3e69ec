"""Calls from two host threads at once, each on its own stream and buffers: kernels whose shared memory depends
on the sizes are asked for it per call, and neither thread's request may undo the other's."""
import threading

import pytest
import torch

from test_gpu_glu import _inputs, _tiles

pytestmark = pytest.mark.gpu


def test_few_rows_of_different_counts_from_two_threads(cuda_lib):
    """The gated layer's codes with 9 and with 16 rows (77 and 84 KB of shared memory a block)."""
    bl = cuda_lib
    K, N = 512, 2048
    X, q, scale, _ = _inputs(16, K, N, 1)
    tiles = _tiles(bl, q, scale)
    wants, outs = [], [torch.empty(m, N, dtype=torch.bfloat16, device="cuda") for m in (9, 16)]
    for out in outs:
        bl.tern_glu_fwd(X[:len(out)], tiles, scale, out)
        wants.append(out.clone())
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2)

    def work(out, stream):
        call = bl.GluForward(X[:len(out)], tiles, scale, out)
        start.wait(timeout=60)
        try:
            for _ in range(20000):
                call(stream)
        except bl.TernError as e:
            failed.append(e)
    streams = [torch.cuda.Stream() for _ in outs]
    threads = [threading.Thread(target=work, args=a) for a in zip(outs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
    assert all(torch.equal(a, b) for a, b in zip(outs, wants))
