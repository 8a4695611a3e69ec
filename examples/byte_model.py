"""A small recurrent byte model on the library's calls: training, and generation one byte at a time.

    x = embedding(bytes); f, v, r = x W_f, x W_v, x W_r (ternary); y = gated recurrence(f, v, r);
    z = x + y W_o (ternary); with a feed-forward layer z = z + (silu(g) * u) W_d, g | u = norm(z) W_u
    (ternary); logits = z head

Training runs the embedding, the grouped ternary projections, the recurrence, the feed-forward layer
and the loss forward and back, then moves the ternary accumulators by their orthogonalised gradients
(tern_orthogonalize, then tern_sr4_step) and everything continuous (scales, table, gate bias, norm,
head) by AdamW.  The loss is cross entropy of the next byte, or distillation from another model's most
likely bytes.  PyTorch supplies memory and the small dense head.

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
    def __init__(self, width=128, batch=8, length=64, seed=0, ffn=0):
        """ffn: width of the feed-forward layer (a multiple of 16), 0 for none."""
        self.D, self.B, self.T, self.F = D, B, T, F = width, batch, length, ffn
        self.shapes = {k: (D, D) for k in NAMES}
        if F:
            self.shapes |= {"u": (D, 2 * F), "d": (F, D)}
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.q = {k: torch.randint(-3, 4, self.shapes[k], dtype=torch.int8, device="cuda", generator=g) for k in NAMES}
        self.scale = {k: torch.full((n,), 0.5 / math.sqrt(m), device="cuda") for k, (m, n) in self.shapes.items()}
        self.tiles = {k: bl.Tiles.empty(*s) for k, s in self.shapes.items()}
        self.table, self.head = rnd(256, D) * 0.5, rnd(D, 256) / math.sqrt(D)
        self.bias = torch.linspace(0.0, 4.0, D, device="cuda")     # memories from two bytes to about fifty
        if F:
            self.q |= {k: torch.randint(-3, 4, self.shapes[k], dtype=torch.int8, device="cuda", generator=g) for k in "ud"}
            self.norm_w, self.norm_b = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
        self._materialize = bl.MaterializeGrouped([dict(q=self.q[k], scale=self.scale[k], tiles=self.tiles[k]) for k in self.shapes])
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
        self.gq = {k: f32(*s) for k, s in self.shapes.items()}
        self.sgrad = {k: f32(s[1]) for k, s in self.shapes.items()}
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
        if self.F:
            self._feed_forward_buffers(layer)
        # the loss and its gradient, mean over the positions
        self.logits, self.dlogits, self.loss, self.mean = f32(M, 256), f32(M, 256), f32(M), torch.full((M,), 1.0 / M, device="cuda")
        self.targets = torch.zeros(M, 1, dtype=torch.int64, device="cuda")
        self._cross_entropy = bl.Distill(self.logits, self.targets, None, self.loss, dlogits=self.dlogits, weight=self.mean)
        # updates
        self.update = {k: torch.empty(s, dtype=torch.bfloat16, device="cuda") for k, s in self.shapes.items()}
        ortho_ws = _bytes(max(bl.tern_orthogonalize_workspace(*s) for s in self.shapes.values()))
        self._ortho = {k: bl.Orthogonalize(self.gq[k], self.update[k], ortho_ws) for k in self.shapes}
        self.sr4_ws = _bytes(max(bl.tern_sr4_workspace(m * n) for m, n in self.shapes.values()))
        ws_, gs = [*self.scale.values(), self.table, self.head, self.bias], [*self.sgrad.values(), self.dtable, self.dhead, self.dbias]
        if self.F:
            ws_, gs = ws_ + [self.norm_w, self.norm_b], gs + [self.dnorm_w, self.dnorm_b]
        m, v = [torch.zeros_like(w) for w in ws_], [torch.zeros_like(w) for w in ws_]
        self.hyper = torch.empty(4, device="cuda")
        self._adamw = bl.MultiAdamW(ws_, gs, m, v, self.hyper, 0.9, 0.95, 1e-8, 0.0)

    def _feed_forward_buffers(self, layer):
        D, F, M = self.D, self.F, self.B * self.T
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.z1, self.ff, self.dz1 = f32(M, D), f32(M, D), f32(M, D)
        xn, dxn, H, dH, dff, pair = bf(M, D), bf(M, D), bf(M, F), bf(M, F), bf(M, D), bf(M, 2 * F)
        mean, rstd, self.dnorm_w, self.dnorm_b, self.dff = f32(M), f32(M), f32(D), f32(D), dff
        ws = _bytes(bl.tern_linear_bwd_grouped_workspace([(M, F, D), (M, D, 2 * F)]))
        # forward: the gate's and the value's factors of the gradient are kept in `pair`, which the
        # gradient turns into dY in place
        self._feed = [bl.NormForward(self.z1, xn, self.norm_w, self.norm_b, mean=mean, rstd=rstd),
                      bl.GluForward(xn, self.tiles["u"], self.scale["u"], H, saved=pair),
                      bl.GroupedForward([layer("d", H, Y=self.ff)])]
        self._feed_back = [bl.GroupedBackward([layer("d", H, dY=dff, dX_bf16=dH, gq=self.gq["d"], sgrad=self.sgrad["d"])], ws),
                           bl.GluBackward(dH, pair, saved=pair),
                           bl.GroupedBackward([layer("u", xn, dY=pair, dX_bf16=dxn, gq=self.gq["u"], sgrad=self.sgrad["u"])], ws),
                           bl.NormBackward(self.z1, dxn, mean, rstd, self.dz1, _bytes(bl.tern_norm_bwd_workspace(M, D)), self.norm_w,
                                           self.dnorm_w, self.dnorm_b)]

    def forward(self, tokens):
        """Logits [B, T, 256] of the bytes after each of tokens [B, T]."""
        self._run(tokens)
        return self.logits.view(self.B, self.T, 256).clone()

    def _run(self, tokens):
        self.tokens.copy_(tokens.reshape(-1))
        self._embed()
        self._project()
        self._scan()
        self._output()
        self.z = self.x.float() + self.out.float()
        if self.F:
            self.z1.copy_(self.z)
            for call in self._feed:
                call()
            self.z = self.z1 + self.ff
        torch.mm(self.z, self.head, out=self.logits)

    def score(self, tokens, targets=None, top=0):
        """Of the bytes after each of tokens [B, T]: the log probability of targets [B, T] (None without),
        the entropy, and the `top` most likely bytes with their log probabilities [B, T, top]."""
        self._run(tokens)
        M, f32 = self.B * self.T, lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        logp, entropy = None if targets is None else f32(M), f32(M)
        ids, values = (torch.empty(M, top, dtype=torch.int32, device="cuda"), f32(M, top)) if top else (None, None)
        bl.tern_score(self.logits, None if targets is None else targets.reshape(-1).contiguous(), logp, entropy, top_ids=ids, top_logp=values)
        rows = lambda t: None if t is None else t.view(self.B, self.T, *t.shape[1:])  # noqa: E731
        return rows(logp), rows(entropy), rows(ids), rows(values)

    def train_step(self, tokens, targets, lr=3e-3, target_step=0.02):
        """One step; returns the mean cross entropy (a device scalar)."""
        self._run(tokens)
        self.targets.copy_(targets.reshape(-1, 1))
        self._cross_entropy()
        return self._learn(lr, target_step)

    def distill_step(self, tokens, ids, top, temperature=2.0, lr=3e-3, target_step=0.02):
        """One step towards a teacher's most likely bytes, as its score() gives them; returns the mean loss."""
        self._run(tokens)
        M = self.B * self.T
        bl.tern_distill(self.logits, ids.reshape(M, -1), top.reshape(M, -1), self.loss, dlogits=self.dlogits, weight=self.mean,
                        temperature=temperature)
        return self._learn(lr, target_step)

    def _learn(self, lr, target_step):
        loss = self.loss.sum()
        torch.mm(self.z.t(), self.dlogits, out=self.dhead)
        dz = self.dlogits @ self.head.t()
        if self.F:
            self.dff.copy_(dz)
            for call in self._feed_back:
                call()
            dz = dz + self.dz1
        self.dout.copy_(dz)
        self._output_back()
        self._scan_back()
        self._project_back()
        self.dx.copy_(dz + self.dxs["f"] + self.dxs["v"] + self.dxs["r"])
        self._embed_back()
        t = self.step_count = self.step_count + 1
        at = 0
        for k, (m, n) in self.shapes.items():
            self._ortho[k]()
            bl.tern_sr4_step(self.q[k], self.update[k].float(), self.sr4_ws, target_step=target_step, idx_base=at, counter=t)
            at += m * n
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
        if self.F:
            z, ff, xn = torch.empty(batch, D, device="cuda"), torch.empty(batch, D, device="cuda"), bf()
            H = torch.empty(batch, self.F, dtype=torch.bfloat16, device="cuda")
            feed = [bl.NormForward(z, xn, self.norm_w, self.norm_b), bl.GluForward(xn, self.tiles["u"], self.scale["u"], H),
                    bl.GroupedForward([dict(X=H, tiles=self.tiles["d"], scale=self.scale["d"], Y=ff)])]

        def next_logits(tokens):
            tok.copy_(tokens)
            embed()
            project()
            step()
            output()
            if not self.F:
                return (x.float() + out.float()) @ self.head
            torch.add(x.float(), out.float(), out=z)
            for call in feed:
                call()
            return (z + ff) @ self.head
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
    model = ByteModel(ffn=352)
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
    # a smaller model learns from its eight most likely bytes
    student = ByteModel(width=64, seed=1)
    for i, (tokens, targets) in zip(range(steps), batches(model, seed=1)):
        _, _, ids, top = model.score(tokens, top=8)
        loss = student.distill_step(tokens, ids, top)
        if i % 20 == 0 or i + 1 == steps:
            logp, entropy, _, _ = student.score(tokens, targets)
            print(f"student step {i}: distillation {loss.item():.3f}, cross entropy {-logp.mean().item():.3f}, entropy {entropy.mean().item():.3f}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
