"""The gradient of the embedding where its other kernels run: 256 positions a block in 16-byte rows
and several channel tiles, two and three passes of either sort.  Integer rows, so the sums are exact."""
import pytest
import torch

from test_gpu_embed import _tok

pytestmark = pytest.mark.gpu

# one cluster sorts up to 32768 positions (in smaller tiles up to 8192), three launches a pass more; keys
# of more than 11 bits take two passes, of more than 22 three
SIZES = [(32768, 100003, 512), (20000, 3000, 520), (65537, 5000, 264), (40000, 3000, 521), (40000, 300, 1032), (20000, 5000000, 2),
         (50000, 5000000, 1), (8192, 3000, 64), (8193, 3000, 64), (32768, 3000, 65), (32769, 3000, 64), (8192, 5000000, 1)]


@pytest.mark.parametrize("n,V,D", SIZES)
@pytest.mark.parametrize("tok", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("long_run", [False, True], ids=["text", "long_run"])
def test_gradient_is_exact(cuda_lib, n, V, D, tok, long_run):
    bl = cuda_lib
    t = _tok(n, V, n + D, tok)
    if long_run:      # one token's positions fill many of a block's 256
        t[n // 5:4 * n // 5] = V // 2
    dout = torch.randint(-8, 9, (n, D), device="cuda").bfloat16()
    ok = (t >= 0) & (t < V)
    ref = torch.zeros(V, D, device="cuda", dtype=torch.float64).index_add_(0, t[ok].long(), dout[ok].double())
    ws = torch.full((bl.tern_embed_bwd_workspace(n, V, D),), 0xAB, dtype=torch.uint8, device="cuda")
    g = torch.full((V, D), float("nan"), device="cuda")
    bl.tern_embed_bwd(t, dout, g, ws)
    assert torch.equal(g.double(), ref)
    bl.tern_embed_bwd(t, dout, g, ws, accumulate=True, scale=2.0)
    assert torch.equal(g.double(), 3 * ref)
