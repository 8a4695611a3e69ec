"""A small recurrent byte model on the library's calls: training, and generation one byte at a time.

    x = embedding(bytes); f, v, r = x W_f, x W_v, x W_r (ternary); y = gated recurrence(f, v, r);
    z = x + y W_o (ternary); logits = z head

Training runs the embedding, the grouped ternary projections and the recurrence forward and back,
then moves the ternary accumulators by their orthogonalised gradients (tern_orthogonalize, then
tern_sr4_step) and everything continuous (scales, table, gate bias, head) by AdamW.  PyTorch
supplies memory, the small dense head and the loss.

    python examples/byte_model.py [steps]
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_linear_gb300 as bl  # noqa: E402

NAMES = ("f", "v", "r", "o")


def _bytes(n):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device="cuda")


class ByteModel:
    def __init__(self, width=128, batch=8, length=64, seed=0):
        self.D, self.B, self.T = D, B, T = width, batch, length
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.q = {k: torch.randint(-3, 4, (D, D), dtype=torch.int8, device="cuda", generator=g) for k in NAMES}
        self.scale = {k: torch.full((D,), 0.5 / math.sqrt(D), device="cuda") for k in NAMES}
        self.tiles = {k: bl.Tiles.empty(D, D) for k in NAMES}
        self.table, self.head = rnd(256, D) * 0.5, rnd(D, 256) / math.sqrt(D)
        self.bias = torch.linspace(0.0, 4.0, D, device="cuda")     # memories from two bytes to about fifty
        self._materialize = bl.MaterializeGrouped([dict(q=self.q[k], scale=self.scale[k], tiles=self.tiles[k]) for k in NAMES])
        self._materialize()
        self._buffers()
        self.step_count = 0

    def _buffers(self):
        D, B, T, M = self.D, self.B, self.T, self.B * self.T
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.tokens = torch.zeros(M, dtype=torch.int64, device="cuda")
        self.x, self.out, self.y, self.dy, self.dout, self.dx = (bf(M, D) for _ in range(6))
        self.act = {k: bf(M, D) for k in "fvr"}
        self.dact = {k: bf(M, D) for k in "fvr"}
        self.dxs = {k: f32(M, D) for k in "fvr"}
        self.gq = {k: f32(D, D) for k in NAMES}
        self.sgrad = {k: f32(D) for k in NAMES}
        self.dtable, self.dhead, self.dbias = f32(256, D), f32(D, 256), f32(D)
        self.saved, scan_ws = _bytes(bl.tern_scan_saved(B, T, D)), _bytes(bl.tern_scan_bwd_workspace(B, T, D))
        rows = lambda t: t.view(B, T, D)  # noqa: E731
        a, da = [rows(self.act[k]) for k in "fvr"], [rows(self.dact[k]) for k in "fvr"]

        def layer(k, X, **kw):
            return dict(X=X, tiles=self.tiles[k], scale=self.scale[k], **kw)
        self._embed = bl.EmbedForward(self.tokens, self.table, self.x)
        self._project = bl.GroupedForward([layer(k, self.x, Y_bf16=self.act[k]) for k in "fvr"])
        self._scan = bl.ScanForward(*a, rows(self.y), f_bias=self.bias, saved=self.saved)
        self._output = bl.GroupedForward([layer("o", self.y, Y_bf16=self.out)])
        ws = _bytes(bl.tern_linear_bwd_grouped_workspace([(M, D, D)] * 3))
        self._output_back = bl.GroupedBackward(
            [layer("o", self.y, dY=self.dout, dX_bf16=self.dy, gq=self.gq["o"], sgrad=self.sgrad["o"])], ws)
        self._scan_back = bl.ScanBackward(*a, rows(self.dy), self.saved, scan_ws, *da, f_bias=self.bias, dbias=self.dbias)
        self._project_back = bl.GroupedBackward(
            [layer(k, self.x, dY=self.dact[k], dX=self.dxs[k], gq=self.gq[k], sgrad=self.sgrad[k]) for k in "fvr"], ws)
        self._embed_back = bl.EmbedBackward(self.tokens, self.dx, self.dtable, _bytes(bl.tern_embed_bwd_workspace(M, 256, D)))
        # updates
        self.update = {k: torch.empty(D, D, dtype=torch.bfloat16, device="cuda") for k in NAMES}
        ortho_ws = _bytes(bl.tern_orthogonalize_workspace(D, D))
        self._ortho = {k: bl.Orthogonalize(self.gq[k], self.update[k], ortho_ws) for k in NAMES}
        self.sr4_ws = _bytes(bl.tern_sr4_workspace(D * D))
        ws_, gs = [*self.scale.values(), self.table, self.head, self.bias], [*self.sgrad.values(), self.dtable, self.dhead, self.dbias]
        m, v = [torch.zeros_like(w) for w in ws_], [torch.zeros_like(w) for w in ws_]
        self.hyper = torch.empty(4, device="cuda")
        self._adamw = bl.MultiAdamW(ws_, gs, m, v, self.hyper, 0.9, 0.95, 1e-8, 0.0)

    def forward(self, tokens):
        """Logits [B, T, 256] of the bytes after each of tokens [B, T]."""
        self.tokens.copy_(tokens.reshape(-1))
        self._embed()
        self._project()
        self._scan()
        self._output()
        self.z = self.x.float() + self.out.float()
        return (self.z @ self.head).view(self.B, self.T, 256)

    def train_step(self, tokens, targets, lr=3e-3, target_step=0.02):
        """One step; returns the mean cross entropy (a device scalar)."""
        logits = self.forward(tokens).view(-1, 256)
        logp = torch.log_softmax(logits, 1)
        loss = -logp.gather(1, targets.reshape(-1, 1)).mean()
        dlogits = torch.exp(logp)
        dlogits.scatter_add_(1, targets.reshape(-1, 1), torch.full_like(logp[:, :1], -1.0))
        dlogits /= logits.shape[0]
        torch.mm(self.z.t(), dlogits, out=self.dhead)
        dz = dlogits @ self.head.t()
        self.dout.copy_(dz)
        self._output_back()
        self._scan_back()
        self._project_back()
        self.dx.copy_(dz + self.dxs["f"] + self.dxs["v"] + self.dxs["r"])
        self._embed_back()
        t = self.step_count = self.step_count + 1
        for i, k in enumerate(NAMES):
            self._ortho[k]()
            bl.tern_sr4_step(self.q[k], self.update[k].float(), self.sr4_ws, target_step=target_step, idx_base=i * self.D * self.D,
                             counter=t)
        self.hyper.copy_(torch.tensor([lr, 1 - 0.9 ** t, 1 - 0.95 ** t, 1.0]))
        self._adamw()
        self._materialize()
        return loss

    def generator(self, batch=1):
        """A function from one byte per sequence [batch] to the next byte's logits [batch, 256]; the
        state is carried in place by single-token steps."""
        D = self.D
        bf = lambda: torch.empty(batch, D, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        tok, x, y, out, act = torch.zeros(batch, dtype=torch.int64, device="cuda"), bf(), bf(), bf(), {k: bf() for k in "fvr"}
        h = torch.zeros(batch, D, device="cuda")
        embed = bl.EmbedForward(tok, self.table, x)
        project = bl.GroupedForward([dict(X=x, tiles=self.tiles[k], scale=self.scale[k], Y_bf16=act[k]) for k in "fvr"])
        step = bl.ScanStep(act["f"], act["v"], act["r"], h, y, f_bias=self.bias)
        output = bl.GroupedForward([dict(X=y, tiles=self.tiles["o"], scale=self.scale["o"], Y_bf16=out)])

        def next_logits(tokens):
            tok.copy_(tokens)
            embed()
            project()
            step()
            output()
            return (x.float() + out.float()) @ self.head
        return next_logits


TEXT = b"the quick brown fox jumps over the lazy dog while seven wizards quietly mix black jugs of zinc. "


def batches(model, seed=0):
    """Endless (tokens, targets) from random places of a repeated sentence."""
    data = torch.tensor(list(TEXT * 8), device="cuda")
    g = torch.Generator().manual_seed(seed)
    while True:
        at = torch.randint(0, len(data) - model.T - 1, (model.B,), generator=g).tolist()
        rows = torch.stack([data[i:i + model.T + 1] for i in at])
        yield rows[:, :-1], rows[:, 1:]


def main(steps=200):
    model = ByteModel()
    for i, (tokens, targets) in zip(range(steps), batches(model)):
        loss = model.train_step(tokens, targets)
        if i % 20 == 0 or i + 1 == steps:
            print(f"step {i}: loss {loss.item():.3f}")
    if bl.tern_device_status() != bl.TERN_OK:
        raise RuntimeError("a bounded wait gave up")
    following = model.generator()
    text = list(b"the quick ")
    for b in text:
        logits = following(torch.tensor([b], device="cuda"))
    for _ in range(80):
        text.append(int(logits.argmax()))
        logits = following(torch.tensor([text[-1]], device="cuda"))
    print(bytes(text).decode(errors="replace"))


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
