"""The norm, feed-forward, score and distillation calls side by side: sizes first met inside a capture, and
two streams at once."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _calls(bl, seed, size):
    """Prepared calls of one size of each operator, and their outputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    e = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    n, D, F, V = size
    x, dy, y, dx = r(n, D).to(bf), r(n, D).to(bf), e(n, D, dt=bf), e(n, D, dt=bf)
    mean, rstd, dw, db, w = e(n), e(n), e(D), e(D), r(D)
    calls = [bl.NormForward(x, y, w, None, mean=mean, rstd=rstd),
             bl.NormBackward(x, dy, mean, rstd, dx, e(max(16, bl.tern_norm_bwd_workspace(n, D)), dt=torch.uint8), w, dw, db)]
    K = D // 16 * 16
    q, scale = torch.randint(-7, 8, (K, 2 * F), dtype=torch.int8, device="cuda", generator=g), torch.full((2 * F,), K ** -0.5, device="cuda")
    tiles = bl.Tiles.empty(K, 2 * F, hi_lo=False)
    bl.tern_materialize(q, scale, tiles, 2, 7)
    X, H, pair, dH, dY = r(n, K).to(bf), e(n, F, dt=bf), e(n, 2 * F, dt=bf), r(n, F).to(bf), e(n, 2 * F, dt=bf)
    calls += [bl.GluForward(X, tiles, scale, H), bl.GluForward(X, tiles, scale, H, saved=pair, act="gelu"), bl.GluBackward(dH, dY, saved=pair),
              bl.GluBackward(dH, pair, X=X, tiles=tiles, scale=scale, act="relu2")]
    x2, tok = r(n, V).to(bf), torch.randint(0, V, (n,), device="cuda", generator=g)
    logp, ent, ids, top, loss, d = e(n), e(n), e(n, 8, dt=torch.int32), e(n, 8), e(n), e(n, V, dt=bf)
    calls += [bl.Score(x2, tok, logp, ent, None, ids, top), bl.Distill(x2, ids, top, loss, dlogits=d, temperature=2.0)]
    return calls, [y, mean, rstd, dx, dw, db, H, pair, dY, logp, ent, ids, top, loss, d]


SIZES = [(3, 64, 48, 200), (700, 520, 144, 3000), (33, 2050, 400, 50000), (3000, 256, 64, 900)]


def _capture_unseen():
    """Each operator called once at one size, then other sizes captured without a call before."""
    sys.path.insert(0, ROOT)
    import bit_linear_gb300 as bl
    for c in _calls(bl, 0, SIZES[0])[0]:
        c()
    torch.cuda.synchronize()
    for size in SIZES[1:]:
        calls, outs = _calls(bl, 1, size)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for c in calls:
                c()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        for c in calls:
            c()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), size
    assert bl.tern_device_status() == bl.TERN_OK
    print("captured")


def test_sizes_first_met_in_a_capture(cuda_lib):
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_two_streams_at_once(cuda_lib):
    bl = cuda_lib
    both = [_calls(bl, 10 + i, SIZES[1 + i]) for i in range(2)]
    want = []
    for calls, outs in both:
        for c in calls:
            c()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(len(both[0][0])):
            for (calls, _), s in zip(both, streams):
                calls[i](s)
    torch.cuda.synchronize()
    for (_, outs), w in zip(both, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
    assert bl.tern_device_status() == bl.TERN_OK


if __name__ == "__main__":
    _capture_unseen()
