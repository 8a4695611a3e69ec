"""The example model with its feed-forward layer, its scores and distillation: gradients against autograd
over the same formulas in fp64, single bytes against whole sequences, the same bits every time."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def bm(cuda_lib):
    import byte_model
    return byte_model


@pytest.fixture(scope="module", name="cuda_lib")
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_linear_gb300 as bl
    return bl


PARAMS = ("table", "bias", "head", "norm_w", "norm_b")
GRADS = ("dtable", "dbias", "dhead", "dnorm_w", "dnorm_b")


def _logits(m, tokens):
    """The model's logits in fp64 and its continuous parameters, with gradients."""
    par = {k: getattr(m, k).double().clone().requires_grad_() for k in PARAMS}
    scale = {k: v.double().clone().requires_grad_() for k, v in m.scale.items()}

    def weight(k):
        q = m.q[k].double()
        return torch.where(q.abs() >= 2, torch.sign(q), torch.zeros_like(q)) * scale[k]
    x = par["table"][tokens]
    f, v, r = (x @ weight(k) for k in "fvr")
    a = torch.sigmoid(f + par["bias"])
    h, ys = torch.zeros(m.B, m.D, dtype=torch.float64, device="cuda"), []
    for t in range(m.T):
        h = a[:, t] * h + (1 - a[:, t]) * v[:, t]
        ys.append(torch.sigmoid(r[:, t]) * h)
    z = x + torch.stack(ys, 1) @ weight("o")
    n = torch.nn.functional.layer_norm(z, (m.D,), par["norm_w"], par["norm_b"], 1e-5)
    g, u = (n @ weight("u")).chunk(2, -1)
    z = z + (torch.nn.functional.silu(g) * u) @ weight("d")
    return z @ par["head"], par, scale


def _check(m, par, scale):
    # bf16 activations and gradients: 2^-9 rms in each of a dozen roundings on the way
    for k, d in zip(PARAMS, GRADS):
        ref = par[k].grad
        assert (getattr(m, d).double() - ref).norm() <= 0.03 * ref.norm(), k
    for k, s in scale.items():
        assert (m.sgrad[k].double() - s.grad).norm() <= 0.03 * s.grad.norm(), k


def test_gradients_agree_with_autograd(bm, cuda_lib):
    m = bm.ByteModel(width=64, batch=4, length=40, ffn=176)
    tokens, targets = next(bm.batches(m))
    logits, par, scale = _logits(m, tokens)
    torch.nn.functional.cross_entropy(logits.reshape(-1, 256), targets.reshape(-1)).backward()
    assert (m.forward(tokens).double() - logits).norm() <= 0.02 * logits.norm()
    m.train_step(tokens, targets, lr=0.0, target_step=0.0)
    _check(m, par, scale)
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


def test_distillation_agrees_with_autograd(bm, cuda_lib):
    teacher = bm.ByteModel(width=128, batch=4, length=40, seed=3)
    m = bm.ByteModel(width=64, batch=4, length=40, ffn=48)
    tokens, _ = next(bm.batches(m, seed=2))
    _, _, ids, top = teacher.score(tokens, top=12)
    logits, par, scale = _logits(m, tokens)
    p = torch.softmax(top.double() / 2, -1)
    logq = torch.log_softmax(logits / 2, -1).gather(-1, ids.long())
    loss = 4 * (p * (p.log() - logq)).sum(-1).mean()
    loss.backward()
    got = m.distill_step(tokens, ids, top, temperature=2.0, lr=0.0, target_step=0.0)
    assert abs(got.item() - loss.item()) <= 0.02 * loss.item()
    _check(m, par, scale)
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


def test_scores(bm):
    m = bm.ByteModel(width=64, batch=3, length=20, ffn=64)
    tokens, targets = next(bm.batches(m))
    logp, entropy, ids, top = m.score(tokens, targets, top=6)
    want = torch.log_softmax(m.forward(tokens).double(), -1)
    # fp32 sums of 256 terms: 2^-15 covers them at these sizes
    assert (logp - want.gather(-1, targets[..., None])[..., 0]).abs().max() <= 2 ** -15
    assert (entropy + (want.exp() * want).sum(-1)).abs().max() <= 2 ** -15
    values, order = torch.sort(want, dim=-1, descending=True, stable=True)
    assert torch.equal(ids.long(), order[..., :6]) and (top - values[..., :6]).abs().max() <= 2 ** -15


def test_training_repeats(bm):
    runs = []
    for _ in range(2):
        m = bm.ByteModel(width=64, batch=4, length=32, ffn=176)
        teacher = bm.ByteModel(width=64, batch=4, length=32, seed=5)
        losses = []
        for _, (x, y) in zip(range(10), bm.batches(m)):
            losses.append(m.train_step(x, y).item())
            _, _, ids, top = teacher.score(x, top=4)
            losses.append(m.distill_step(x, ids, top).item())
        runs.append((losses, [t.clone() for t in (*m.q.values(), m.head, m.norm_w)]))
    assert runs[0][0] == runs[1][0] and all(torch.equal(a, b) for a, b in zip(runs[0][1], runs[1][1]))


def test_generation_matches_the_sequence(bm):
    m = bm.ByteModel(width=128, batch=3, length=30, ffn=352)
    tokens, _ = next(bm.batches(m, seed=3))
    whole = m.forward(tokens).clone()
    following = m.generator(batch=3)
    for t in range(m.T):
        logits = following(tokens[:, t])
        # activations may round to a neighbouring bf16 value, and the codes sum in another order
        assert (logits - whole[:, t]).norm() <= 0.01 * whole[:, t].norm(), t


def test_feed_forward_in_a_graph(bm, cuda_lib):
    """The feed-forward layer's calls and the loss, captured and replayed on new inputs."""
    m = bm.ByteModel(width=64, batch=4, length=32, ffn=176)
    (x, y), (x2, y2) = (b for _, b in zip(range(2), bm.batches(m)))

    def step():
        for call in m._feed:
            call()
        torch.mm(m.z1 + m.ff, m.head, out=m.logits)
        m._cross_entropy()
        m.dff.copy_(m.dlogits @ m.head.t())
        for call in m._feed_back:
            call()

    def outputs():
        return [t.clone() for t in (m.loss, m.dlogits, m.dz1, m.gq["u"], m.gq["d"], m.sgrad["u"], m.dnorm_w)]
    m.forward(x)
    m.targets.copy_(y.reshape(-1, 1))
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    m.forward(x2)
    m.targets.copy_(y2.reshape(-1, 1))
    step()
    want = outputs()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, outputs()))
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK
