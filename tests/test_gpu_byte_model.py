"""The example model: its training step learns, its gradients agree with autograd over the same
formulas, and single-byte generation gives the logits of the whole sequence."""
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


def _weight(m, k):
    """scale * ternary(q), theta = 2, in fp64."""
    q = m.q[k].double()
    return torch.where(q.abs() >= 2, torch.sign(q), torch.zeros_like(q)) * m.scale[k].double()


def _autograd_loss(m, tokens, targets):
    """The model's loss in fp64, with gradients on the table, the bias and the head."""
    par = {k: getattr(m, k).double().clone().requires_grad_() for k in ("table", "bias", "head")}
    x = par["table"][tokens]
    f, v, r = (x @ _weight(m, k) for k in "fvr")
    a = torch.sigmoid(f + par["bias"])
    h, ys = torch.zeros(m.B, m.D, dtype=torch.float64, device="cuda"), []
    for t in range(m.T):
        h = a[:, t] * h + (1 - a[:, t]) * v[:, t]
        ys.append(torch.sigmoid(r[:, t]) * h)
    logits = (x + torch.stack(ys, 1) @ _weight(m, "o")) @ par["head"]
    loss = torch.nn.functional.cross_entropy(logits.reshape(-1, 256), targets.reshape(-1))
    loss.backward()
    return loss.detach(), logits.detach(), par


def test_gradients_agree_with_autograd(bm, cuda_lib):
    m = bm.ByteModel(width=64, batch=4, length=40)
    tokens, targets = next(bm.batches(m))
    loss, logits, par = _autograd_loss(m, tokens, targets)
    before = {k: getattr(m, k).clone() for k in ("table", "bias", "head")}
    ours = m.forward(tokens)
    # bf16 activations: 2^-9 rms in each of five roundings on the way
    assert (ours.double() - logits).norm() <= 0.02 * logits.norm()
    got = m.train_step(tokens, targets, lr=0.0, target_step=0.0)
    assert abs(got.item() - loss.item()) <= 0.02 * loss.item()
    for k, d in (("table", m.dtable), ("bias", m.dbias), ("head", m.dhead)):
        ref = par[k].grad
        assert (d.double() - ref).norm() <= 0.03 * ref.norm(), k
        assert torch.equal(getattr(m, k), before[k])      # lr = 0 moves nothing
    assert cuda_lib.tern_device_status() == cuda_lib.TERN_OK


def test_training_learns_and_repeats(bm):
    losses = []
    for _ in range(2):
        m = bm.ByteModel(width=128, batch=8, length=64)
        losses.append([m.train_step(x, y).item() for _, (x, y) in zip(range(120), bm.batches(m))])
    assert losses[0] == losses[1]                          # the same bits every time
    assert sum(losses[0][-10:]) / 10 < 0.5 * losses[0][0]


def test_generation_matches_the_sequence(bm):
    m = bm.ByteModel(width=128, batch=3, length=50)
    tokens, _ = next(bm.batches(m, seed=3))
    whole = m.forward(tokens)
    following = m.generator(batch=3)
    for t in range(m.T):
        logits = following(tokens[:, t])
        # the state is fp32 either way; activations may round to a neighbouring bf16 value
        assert (logits - whole[:, t]).norm() <= 0.01 * whole[:, t].norm(), t
