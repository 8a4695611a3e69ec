"""Workloads of the operators between and behind the ternary projections: layer norm with its gradient, the
gated feed-forward layer with its gradient, log probabilities of tokens with entropy and the most
likely alternatives, and distillation from a teacher's top logits with its gradient.

Each case runs one pass either through the package's calls (``own`` true) or in a plain form of
elementary torch operations in fp32, and ``exact`` gives the same outputs from the definitions in
fp64.  Definitions, for rows i, channels c, vocabulary entries j:

    norm     y = (x - mean) * rstd * weight + bias, rstd = 1 / sqrt(var + eps); its gradients in x,
             weight and bias
    glu      g | u = scale * (X T) for a ternary T of 2 N columns, the gate's first; H = act(g) * u;
             gradient dY = dH * u * act'(g) | dH * act(g), the dY of the projection's own backward
    score    lse = log sum exp(x), logp = x[token] - lse (0 for an id outside the row), entropy of
             softmax(x), the k largest logits' ids (the lower id first where equal) and x - lse there
    distill  p = softmax(top / T) over the teacher's k entries (ids outside the row and -inf left out),
             q = softmax(x / T); loss = w T^2 sum p (log p - log q[id]), its gradient w T (q - p);
             rows without an entry or with w = 0: 0
"""
import math

import torch

own = False

EPS = 1e-5                         # of the norm

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # generation: the norm of one token
        {"name": "norm token", "op": "norm_fwd", "n": 1, "D": 512, "x": "bf16", "y": "bf16"},
        # the byte model's block: 16 sequences of 512 bytes, an fp32 residual stream into bf16 projections
        {"name": "norm train block", "op": "norm_train", "n": 8192, "D": 512, "x": "f32", "y": "bf16"},
        # the large projection's input
        {"name": "norm train wide", "op": "norm_train", "n": 32768, "D": 4096, "x": "bf16", "y": "bf16"},
        # generation: one token's row of a large vocabulary, with the alternatives that a server reports
        {"name": "score token", "op": "score", "n": 1, "V": 100003, "k": 20, "dtype": "bf16", "masked": False},
        # the byte model's evaluation
        {"name": "score bytes", "op": "score", "n": 8192, "V": 256, "k": 5, "dtype": "f32", "masked": False},
        # a teacher's pass over sequences of a large vocabulary: what distillation learns from
        {"name": "score vocabulary", "op": "score", "n": 4096, "V": 100003, "k": 64, "dtype": "bf16", "masked": False},
        # the byte model's loss and gradient
        {"name": "distill bytes", "op": "distill", "mode": "train", "n": 8192, "V": 256, "k": 16, "dtype": "f32"},
        # a large vocabulary's loss and gradient
        {"name": "distill vocabulary", "op": "distill", "mode": "train", "n": 4096, "V": 100003, "k": 64, "dtype": "bf16"},
        # generation: one token through the byte model's feed-forward layer
        {"name": "glu token", "op": "glu_fwd", "M": 1, "K": 512, "N": 2048, "act": "silu"},
        # generation for a batch at the large projection's sizes (its 12288 columns are gate and value)
        {"name": "glu batch", "op": "glu_fwd", "M": 16, "K": 4096, "N": 6144, "act": "silu"},
        # the byte model's training block, a width between tiles, forward recomputed in the backward pass
        {"name": "glu train block", "op": "glu_train", "M": 8192, "K": 512, "N": 1360, "act": "gelu", "saved": False},
        # training at the large projection's sizes
        {"name": "glu train large", "op": "glu_train", "M": 32768, "K": 4096, "N": 6144, "act": "silu", "saved": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_train", "score", "score", "distill", "distill", "glu_fwd", "glu_train"])
    if op in ("norm_fwd", "norm_train"):
        D = _log(rng, 48, 8192)
        n = _log(rng, 1, min(131072, (1 << 27) // D))
        return {"op": op, "n": n, "D": D, "x": rng.choice(["bf16", "f32"]), "y": rng.choice(["bf16", "bf16", "f32"])}
    if op in ("score", "distill"):
        V = _log(rng, 200, 131072)
        dtype = rng.choice(["bf16", "f32"])
        n = _log(rng, 1, min(32768, (400000000 if dtype == "bf16" else 200000000) // V))
        if op == "score":
            return {"op": op, "n": n, "V": V, "k": rng.randint(0, 64), "dtype": dtype, "masked": rng.random() < 0.3}
        return {"op": op, "mode": rng.choice(["train", "train", "fwd", "bwd"]), "n": n, "V": V, "k": _log(rng, 1, 128), "dtype": dtype}
    K, N = 16 * _log(rng, 4, 256), 16 * _log(rng, 4, 512)
    act = rng.choice(["silu", "gelu", "relu2", "sigmoid"])
    most = 32768 * 4096 * 6144 // (K * N)
    if op == "glu_fwd":
        return {"op": op, "M": _log(rng, 1, min(32768, most)), "K": K, "N": N, "act": act}
    return {"op": op, "M": _log(rng, 32, min(32768, most)), "K": K, "N": N, "act": act, "saved": rng.random() < 0.5}


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _logits(n, V, dtype, randn):
    """Logits of a language model: a frequency bias over the vocabulary, noise per row, in `dtype`."""
    x = randn(n, V).mul_(2.0)
    x += randn(V).mul_(2.0)
    return x.to(_DT[dtype])


def _inputs(case, seed):
    g = _gen(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def rand(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    op = case["op"]
    if op in ("norm_fwd", "norm_train"):
        n, D = case["n"], case["D"]
        # a residual stream: rows of different size, channels with offsets of their own
        s = {"x": (randn(n, D) * (0.5 + 2.0 * rand(n, 1)) + randn(D)).to(_DT[case["x"]]),
             "weight": 1.0 + 0.1 * randn(D), "bias": 0.1 * randn(D)}
        if op == "norm_train":
            s["dy"] = randn(n, D).mul_(0.01).to(_DT[case["y"]])
        return s
    if op in ("glu_fwd", "glu_train"):
        M, K, N = case["M"], case["K"], case["N"]
        # accumulators in -7..7, ternarised at 2; scales that keep the products near 1
        s = {"q": torch.randint(-7, 8, (K, 2 * N), dtype=torch.int8, device="cuda", generator=g),
             "scale": (0.5 + rand(2 * N)) * math.sqrt(1.25 / K), "X": randn(M, K).to(torch.bfloat16)}
        if op == "glu_train":
            s["dH"] = randn(M, N).mul_(0.01).to(torch.bfloat16)
        return s
    n, V, k = case["n"], case["V"], case["k"]
    s = {"logits": _logits(n, V, case["dtype"], randn)}
    if op == "score":
        s["tokens"] = torch.where(rand(n) < 1.0 / 32, -1, torch.randint(0, V, (n,), device="cuda", generator=g))
        if case["masked"]:      # rows under a grammar: a share of their own masked, the last row of several all of it
            share = rand(n, 1)
            if n > 1:
                share[-1] = 2.0
            s["logits"].masked_fill_(rand(n, V) < share, -math.inf)
        return s
    # the teacher's entries: places of their own in each row, logits near the student's range, largest first
    first = torch.randint(0, V, (n, 1), device="cuda", generator=g)
    stride = 1 + torch.randint(0, max(1, V // k), (n, 1), device="cuda", generator=g)
    s["ids"] = ((first + stride * torch.arange(k, device="cuda")) % V).to(torch.int32)
    s["top"] = randn(n, k).mul_(2.0).sort(1, descending=True).values.contiguous()
    s["ids"][rand(n, k) < 1.0 / 64] = -1
    # the rows' weights: the mean over rows, with padding rows of weight 0
    s["weight"] = torch.where(rand(n) < 1.0 / 32, 0.0, 1.0 / n)
    s["T"] = 2.0
    return s


def _ternary(q):
    return (q >= 2).float() - (q <= -2).float()


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "distill" and case["mode"] == "bwd":   # what the forward pass left
        s["lse"] = torch.cat([torch.logsumexp(rows.double() / s["T"], 1) for rows in s["logits"].split(256)]).float()
    if own:
        s["call"], s["out"] = _own_call(case, s)
    elif "q" in s:
        s["W"] = _ternary(s["q"])                            # the weight as a program without codes keeps it
    return s


def _own_call(case, s):
    """The prepared call on this state's buffers and the outputs that it writes."""
    import bit_linear_gb300 as bl
    op = case["op"]

    def new(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def both(fwd, bwd):
        def call():
            fwd()
            bwd()
        return call

    if op in ("norm_fwd", "norm_train"):
        n, D = case["n"], case["D"]
        y = new(n, D, dtype=_DT[case["y"]])
        if op == "norm_fwd":
            return bl.NormForward(s["x"], y, weight=s["weight"], bias=s["bias"], eps=EPS), y
        mean, rstd, dx, dw, db = new(n), new(n), torch.empty_like(s["x"]), new(D), new(D)
        ws = new(max(16, bl.tern_norm_bwd_workspace(n, D)), dtype=torch.uint8)
        fwd = bl.NormForward(s["x"], y, weight=s["weight"], bias=s["bias"], eps=EPS, mean=mean, rstd=rstd)
        bwd = bl.NormBackward(s["x"], s["dy"], mean, rstd, dx, ws, weight=s["weight"], dweight=dw, dbias=db)
        return both(fwd, bwd), (y, mean, rstd, dx, dw, db)
    if op in ("glu_fwd", "glu_train"):
        M, K, N = case["M"], case["K"], case["N"]
        tiles = bl.Tiles.empty(K, 2 * N, hi_lo=False)
        bl.tern_materialize(s["q"], s["scale"], tiles, 2, 7)
        H = new(M, N, dtype=torch.bfloat16)
        if op == "glu_fwd":
            return bl.GluForward(s["X"], tiles, s["scale"], H, act=case["act"]), H
        dY = new(M, 2 * N, dtype=torch.bfloat16)
        if case["saved"]:
            fwd = bl.GluForward(s["X"], tiles, s["scale"], H, act=case["act"], saved=dY)
            bwd = bl.GluBackward(s["dH"], dY, saved=dY)      # in place
        else:
            fwd = bl.GluForward(s["X"], tiles, s["scale"], H, act=case["act"])
            bwd = bl.GluBackward(s["dH"], dY, X=s["X"], tiles=tiles, scale=s["scale"], act=case["act"])
        return both(fwd, bwd), (H, dY)
    n, k = case["n"], case["k"]
    if op == "score":
        logp, entropy, lse = new(n), new(n), new(n)
        ids, top = (new(n, k, dtype=torch.int32), new(n, k)) if k else (None, None)
        call = bl.Score(s["logits"], tokens=s["tokens"], logp=logp, entropy=entropy, lse=lse, top_ids=ids, top_logp=top)
        return call, (logp, entropy, lse) + ((ids, top) if k else ())
    teacher = dict(weight=s["weight"], temperature=s["T"])
    dlogits = torch.empty_like(s["logits"]) if case["mode"] != "fwd" else None
    if case["mode"] == "bwd":
        return bl.DistillBackward(s["logits"], s["ids"], s["top"], s["lse"], dlogits, **teacher), dlogits
    loss, lse = new(n), new(n)
    call = bl.Distill(s["logits"], s["ids"], s["top"], loss, lse=lse, dlogits=dlogits, **teacher)
    return call, (loss, dlogits) if case["mode"] == "train" else (loss, lse)


def run(state):
    if own:
        state["call"]()
        return state["out"]
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- plain forms, fp32

def _plain_norm_fwd(s):
    x = s["x"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    return (d * rstd * s["weight"] + s["bias"]).to(_DT[s["case"]["y"]])


def _plain_norm_train(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    xhat = d * rstd
    y = (xhat * s["weight"] + s["bias"]).to(_DT[s["case"]["y"]])
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return y, mean[:, 0].clone(), rstd[:, 0].clone(), dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0)


_SQRT_HALF, _INV_SQRT_2PI = math.sqrt(0.5), 1.0 / math.sqrt(2.0 * math.pi)


def _act(g, name):
    """act(g) and act'(g)."""
    if name == "relu2":
        r = g.clamp(min=0)
        return r * r, 2 * r
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * _SQRT_HALF))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * _INV_SQRT_2PI
    sig = 1 / (1 + torch.exp(-g))
    d = sig / (1 + torch.exp(g))
    return (sig, d) if name == "sigmoid" else (g * sig, sig + g * d)


def _plain_glu_fwd(s):
    y = (s["X"].float() @ s["W"]) * s["scale"]
    g, u = y.chunk(2, 1)
    return (_act(g, s["case"]["act"])[0] * u).to(torch.bfloat16)


def _plain_glu_train(s):
    y = (s["X"].float() @ s["W"]) * s["scale"]
    g, u = y.chunk(2, 1)
    a, d = _act(g, s["case"]["act"])
    dH = s["dH"].float()
    return (a * u).to(torch.bfloat16), torch.cat([dH * u * d, dH * a], 1).to(torch.bfloat16)


def _zero_where(m, x):
    return torch.where(m, torch.zeros((), device="cuda"), x)


def _plain_score(s):
    x, k, V = s["logits"].float(), s["case"]["k"], s["case"]["V"]
    m = x.amax(1, keepdim=True)
    dead = m == -math.inf                                   # nothing but masked entries
    z = x - _zero_where(dead, m)
    e = torch.exp(z)
    S = e.sum(1, keepdim=True)
    logS = torch.log(S)
    entropy = _zero_where(dead, logS - _zero_where(e == 0, e * z).sum(1, keepdim=True) / S)[:, 0]
    lse = m + _zero_where(dead, logS)
    z = torch.where(dead, -math.inf, z - logS)
    tok = s["tokens"]
    inside = (tok >= 0) & (tok < V)
    logp = _zero_where(~inside, z.gather(1, tok.clamp(0, V - 1)[:, None])[:, 0])
    if not k:
        return logp, entropy, lse[:, 0]
    # one integer key an entry: larger for a larger logit, then for a lower id
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * V + (V - 1 - torch.arange(V, device="cuda"))
    ids = V - 1 - torch.topk(key, k, dim=1).values % V
    return logp, entropy, lse[:, 0], ids.to(torch.int32), z.gather(1, ids)


def _plain_teacher(s):
    """The teacher's probabilities [n, k] (0 for entries left out), the ids to read, and the rows that count."""
    ids, V = s["ids"].long(), s["case"]["V"]
    ok = (ids >= 0) & (ids < V) & (s["top"] != -math.inf)
    t = torch.where(ok, s["top"] / s["T"], -math.inf)
    live = ok.any(1, keepdim=True) & (s["weight"] != 0)[:, None]
    m = t.amax(1, keepdim=True)
    e = torch.exp(t - _zero_where(m == -math.inf, m))
    p = e / torch.where(live, e.sum(1, keepdim=True), torch.ones((), device="cuda"))
    return _zero_where(~(live & ok), p), ids.clamp(0, V - 1), live


def _plain_distill(s):
    mode, T, w = s["case"]["mode"], s["T"], s["weight"][:, None]
    p, at, live = _plain_teacher(s)
    x = s["logits"].float()
    if mode == "bwd":
        q = torch.exp(x / T - s["lse"][:, None])
    else:
        m = x.amax(1, keepdim=True)
        z = (x - m) / T
        q = torch.exp(z)
        S = q.sum(1, keepdim=True)
        logS = torch.log(S)
        q = q / S
        lp = torch.log(torch.where(p > 0, p, torch.ones((), device="cuda")))
        loss = _zero_where(~live, w * (T * T) * (p * (lp - z.gather(1, at) + logS)).sum(1, keepdim=True))[:, 0]
        if mode == "fwd":
            return loss, _zero_where(~live, m / T + logS)[:, 0]
    q.scatter_add_(1, at, -p)
    d = _zero_where(~live, q * (w * T)).to(s["logits"].dtype)
    return d if mode == "bwd" else (loss, d)


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_train": _plain_norm_train, "glu_fwd": _plain_glu_fwd,
          "glu_train": _plain_glu_train, "score": _plain_score, "distill": _plain_distill}


# ---------------------------------------------------------------------------- definitions, fp64

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("norm_fwd", "norm_train"):
        return _exact_norm(s, op == "norm_train")
    if op in ("glu_fwd", "glu_train"):
        return _exact_glu(case, s)
    # a few rows at a time
    parts = []
    for at in range(0, case["n"], 256):
        rows = {k: v[at:at + 256] if isinstance(v, torch.Tensor) else v for k, v in s.items()}
        parts.append(_exact_score(case, rows) if op == "score" else _exact_distill(case, rows))
    whole = tuple(torch.cat(p) for p in zip(*parts))
    return whole[0] if len(whole) == 1 else whole


def _exact_norm(s, train):
    x, w = s["x"].double(), s["weight"].double()
    D = x.shape[1]
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    sd = (var + EPS).sqrt()
    xhat = (x - mean) / sd
    y = torch.addcmul(s["bias"].double(), xhat, w)
    if not train:
        return y
    dy = s["dy"].double()
    # the projection of w dy off the constants and off xhat, divided by the deviation
    g = dy * w
    along = torch.einsum("nd,nd->n", g, xhat)[:, None] / D
    dx = (g - g.sum(1, keepdim=True) / D - along * xhat) / sd
    return y, mean.squeeze(1), sd.reciprocal().squeeze(1), dx, torch.einsum("nd,nd->d", dy, xhat), torch.einsum("nd->d", dy)


def _exact_glu(case, s):
    N = case["N"]
    q = s["q"]
    T = torch.where(q.abs() >= 2, torch.sign(q), torch.zeros_like(q)).double()
    parts = []
    for X, dH in zip(s["X"].split(4096), s.get("dH", s["X"]).split(4096)):
        y = torch.mm(X.double(), T).mul_(s["scale"].double())
        g, u = y[:, :N], y[:, N:]
        if case["act"] == "silu":
            a, d = g * torch.sigmoid(g), torch.sigmoid(g) * (1 + g * torch.sigmoid(-g))
        elif case["act"] == "sigmoid":
            a, d = torch.sigmoid(g), torch.sigmoid(g) * torch.sigmoid(-g)
        elif case["act"] == "gelu":
            cdf = torch.special.ndtr(g)
            a, d = g * cdf, cdf + g * torch.exp(g.square() / -2) / math.sqrt(2 * math.pi)
        else:
            a, d = torch.relu(g).square(), 2 * torch.relu(g)
        if case["op"] == "glu_fwd":
            parts.append((a * u,))
        else:
            dH = dH.double()
            parts.append((a * u, torch.cat([d * u * dH, a * dH], 1)))
    whole = tuple(torch.cat(p) for p in zip(*parts))
    return whole if len(whole) > 1 else whole[0]


def _exact_score(case, s):
    x, k, V, tok = s["logits"].double(), case["k"], case["V"], s["tokens"]
    lse = torch.logsumexp(x, 1)
    logp = x - lse[:, None]
    logp[lse == -math.inf] = -math.inf
    entropy = torch.special.entr(logp.exp()).sum(1)
    padded = torch.cat([logp, torch.zeros_like(logp[:, :1])], 1)
    given = padded.gather(1, torch.where((tok < 0) | (tok >= V), torch.full_like(tok, V), tok)[:, None])[:, 0]
    if not k:
        return given, entropy, lse
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    return given, entropy, lse, order.to(torch.int32), logp.gather(1, order)


def _exact_distill(case, s):
    T, V, ids = s["T"], case["V"], s["ids"].long()
    x = s["logits"].double() / T
    lse = torch.logsumexp(x, 1, keepdim=True)
    logq = x - lse
    out = (ids < 0) | (ids >= V)
    t = (s["top"].double() / T).masked_fill(out, -math.inf)
    live = ~torch.isinf(t).all(1, keepdim=True) & (s["weight"] != 0)[:, None]
    p = torch.softmax(t, 1).nan_to_num(0.0)
    w = s["weight"].double()[:, None]
    # sum p log p - sum p log q
    ce = (p * logq.gather(1, ids.clamp(0, V - 1))).sum(1, keepdim=True)
    loss = (w * T * T * (torch.xlogy(p, p).sum(1, keepdim=True) - ce)).masked_fill(~live, 0.0).squeeze(1)
    if case["mode"] == "fwd":
        return loss, lse.masked_fill(~live, 0.0).squeeze(1)
    dense = torch.zeros(x.shape[0], V + 1, device="cuda", dtype=torch.float64)
    dense.scatter_add_(1, ids.masked_fill(out, V), p)
    d = ((logq.exp() - dense[:, :V]) * (w * T)).masked_fill(~live, 0.0)
    return (d,) if case["mode"] == "bwd" else (loss, d)


# ---------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_train"):
        n, D = case["n"], case["D"]
        ex, ey = (2 if case[t] == "bf16" else 4 for t in "xy")
        if op == "norm_fwd":
            return {"bytes": n * D * (ex + ey) + 8 * D, "flops": 8 * n * D}
        # forward and backward each read x; y, dy, dx once
        return {"bytes": n * D * (3 * ex + 2 * ey) + 20 * D + 16 * n, "flops": 24 * n * D}
    if op in ("glu_fwd", "glu_train"):
        M, K, N = case["M"], case["K"], case["N"]
        b = 2 * M * K + K * N // 2 + 8 * N + 2 * M * N      # the weight at two bits each
        if op == "glu_train":
            b += 6 * M * N
        return {"bytes": b, "flops": 4 * M * K * N + (12 if op == "glu_train" else 6) * M * N}
    n, V, k, es = case["n"], case["V"], case["k"], 2 if case["dtype"] == "bf16" else 4
    if op == "score":
        return {"bytes": n * (V * es + 8 + 12 + 8 * k), "flops": 6 * n * V}
    passes = 1 if case["mode"] == "fwd" else 2
    return {"bytes": n * (passes * V * es + 8 * k + 16), "flops": (5 if passes == 1 else 8) * n * V}
