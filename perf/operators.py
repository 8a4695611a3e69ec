"""Workloads of the operators around the ternary projections: the embedding of tokens and its
gradient, the gated linear recurrence (whole sequences, training, one token at a time) and the
orthogonalised update of a weight's gradient.

Each case runs one pass either through the package's calls (``own`` true) or in a plain form of
elementary torch operations in fp32, and ``exact`` gives the same outputs from the definitions in
fp64.  Definitions, for tokens i, rows t, channels d:

    embedding    out[i] = scale * table[tok[i]]          (an id outside the table: a row of zeros)
                 dtable[k] = scale * sum over i with tok[i] = k of dout[i]
    recurrence   a = sigmoid(f + bias), h_t = a_t h_{t-1} + (1 - a_t) v_t, y_t = sigmoid(r_t) h_t,
                 h_{t-1} read as 0 where starts[t]; rows at or past lengths[b] are padding: the state
                 passes them unchanged, y and the gradients there are 0
    update       X = G / (|G|_F + eps), then `steps` times X <- a X + (b A + c A A) X with A = X X^T
                 (the smaller side), out = gain * X
"""
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)     # the odd quintic's coefficients
NS_EPS = 1e-7

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the byte model's input: 16 sequences of 512 bytes, width 512
        {"name": "embed fwd bytes", "op": "embed_fwd", "n": 8192, "V": 256, "D": 512, "table": "f32"},
        # a large vocabulary's input at the large projection's width, prime table height
        {"name": "embed fwd vocabulary", "op": "embed_fwd", "n": 32768, "V": 100003, "D": 4096, "table": "bf16"},
        # the byte model's table gradient: few rows, each the sum of many tokens
        {"name": "embed bwd bytes", "op": "embed_bwd", "n": 8192, "V": 256, "D": 512},
        # a large vocabulary's table gradient: many rows, most of them untouched
        {"name": "embed bwd vocabulary", "op": "embed_bwd", "n": 32768, "V": 100003, "D": 2048},
        # prompts of uneven length before generation, fp32 activations, odd sizes
        {"name": "scan fwd prompts", "op": "scan_fwd", "B": 3, "T": 1000, "D": 521, "dtype": "f32",
         "lengths": True, "starts": False},
        # one long document
        {"name": "scan fwd long", "op": "scan_fwd", "B": 1, "T": 65536, "D": 512, "dtype": "bf16",
         "lengths": False, "starts": False},
        # the byte model's training block
        {"name": "scan train block", "op": "scan_train", "B": 16, "T": 512, "D": 512, "dtype": "bf16",
         "lengths": False, "starts": False},
        # training at the wide layer's width and tokens, several documents packed in a row
        {"name": "scan train packed wide", "op": "scan_train", "B": 8, "T": 2048, "D": 2048, "dtype": "bf16",
         "lengths": False, "starts": True},
        # generation: one sequence, and a batch of them
        {"name": "scan step one", "op": "scan_step", "B": 1, "D": 512, "dtype": "bf16"},
        {"name": "scan step batch", "op": "scan_step", "B": 256, "D": 2048, "dtype": "bf16"},
        # the byte model's FFN matrix, and the large projection
        {"name": "orthogonalize ffn", "op": "orthogonalize", "K": 512, "N": 2048},
        {"name": "orthogonalize large", "op": "orthogonalize", "K": 4096, "N": 12288},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "scan_fwd", "scan_train", "scan_step", "orthogonalize"])
    if op in ("embed_fwd", "embed_bwd"):
        V, D = _log(rng, 200, 131072), _log(rng, 64, 4096)
        n = _log(rng, 1, min(131072, (1 << 26) // D))
        if op == "embed_fwd":
            return {"op": op, "n": n, "V": V, "D": D, "table": rng.choice(["f32", "bf16"])}
        V = max(200, min(V, (1 << 27) // D))
        return {"op": op, "n": n, "V": V, "D": D}
    if op == "scan_step":
        return {"op": op, "B": _log(rng, 1, 256), "D": _log(rng, 64, 4096), "dtype": rng.choice(["bf16", "f32"])}
    if op in ("scan_fwd", "scan_train"):
        B, D = _log(rng, 1, 32), _log(rng, 64, 4096)
        T = _log(rng, 1, min(65536 if op == "scan_fwd" else 16384, (1 << 24) // (B * D)))
        return {"op": op, "B": B, "T": T, "D": D, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "lengths": rng.random() < 0.4, "starts": rng.random() < 0.4}
    m = _log(rng, 32, 4096)
    n = _log(rng, m, 12288)
    K, N = rng.choice([(m, n), (n, m)])
    return {"op": op, "K": K, "N": N}


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tokens(n, V, g):
    """Ids with the long-tailed frequencies of text (rank-frequency exponent about 1), the ranks scattered
    over the table, one in 32 a padding id (-1)."""
    u = torch.rand(n, device="cuda", generator=g)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    tok = torch.randperm(V, device="cuda", generator=g)[rank]
    pad = torch.rand(n, device="cuda", generator=g) < 1.0 / 32
    return torch.where(pad, torch.full_like(tok, -1), tok)


def _inputs(case, seed):
    g = _gen(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    op = case["op"]
    if op in ("embed_fwd", "embed_bwd"):
        n, V, D = case["n"], case["V"], case["D"]
        s = {"tokens": _tokens(n, V, g), "scale": math.sqrt(D)}
        if op == "embed_fwd":
            s["table"] = randn(V, D).mul_(0.02).to(_DT[case["table"]])
        else:
            s["dout"] = randn(n, D).mul_(0.01).to(torch.bfloat16)
        return s
    if op == "orthogonalize":
        K, N = case["K"], case["N"]
        # a gradient: a few strong directions over a full-rank bulk
        r = max(1, min(K, N) // 16)
        w = torch.arange(1, r + 1, device="cuda", dtype=torch.float32).pow_(-0.5)
        G = (randn(K, r) * w) @ randn(r, N)
        return {"G": G.add_(randn(K, N), alpha=0.5).mul_(1e-3), "gain": 0.2 * math.sqrt(max(K, N))}
    B, T, D, dt = case["B"], case.get("T", 1), case["D"], _DT[case["dtype"]]
    shape = (B, D) if op == "scan_step" else (B, T, D)
    # memories from a few tokens to a few thousand: channel biases of the gates spread over [1, 7]
    s = {"f": randn(*shape).to(dt), "v": randn(*shape).to(dt), "r": randn(*shape).to(dt),
         "bias": torch.linspace(1.0, 7.0, D, device="cuda"), "h0": randn(B, D).mul_(0.3)}
    if op == "scan_step":
        return s
    s["lengths"] = s["starts"] = None
    if case["lengths"]:
        s["lengths"] = torch.randint(0, T + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    if case["starts"]:   # documents of about 400 tokens
        s["starts"] = torch.rand(B, T, device="cuda", generator=g).lt_(1.0 / 400).to(torch.uint8)
    if op == "scan_train":
        s["dy"] = randn(*shape).mul_(0.01).to(dt)
        s["dhT"] = randn(B, D).mul_(0.01)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        s["call"], s["out"] = _own_call(case, s)
    return s


def _own_call(case, s):
    """The prepared call on this state's buffers and the outputs that it writes."""
    import bit_linear_gb300 as bl
    op = case["op"]

    def new(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def scratch(nbytes):
        return new(max(16, nbytes), dtype=torch.uint8)

    if op == "embed_fwd":
        out = new(case["n"], case["D"], dtype=torch.bfloat16)
        return bl.EmbedForward(s["tokens"], s["table"], out, scale=s["scale"]), out
    if op == "embed_bwd":
        n, V, D = case["n"], case["V"], case["D"]
        dtable = new(V, D)
        ws = scratch(bl.tern_embed_bwd_workspace(n, V, D))
        return bl.EmbedBackward(s["tokens"], s["dout"], dtable, ws, scale=s["scale"]), dtable
    if op == "orthogonalize":
        K, N = case["K"], case["N"]
        out = new(K, N, dtype=torch.bfloat16)
        ws = scratch(bl.tern_orthogonalize_workspace(K, N))
        return bl.Orthogonalize(s["G"], out, ws, steps=5, eps=NS_EPS, gain=s["gain"]), out
    B, T, D = case["B"], case.get("T", 1), case["D"]
    y = torch.empty_like(s["f"])
    hT = new(B, D)
    if op == "scan_step":
        return bl.ScanStep(s["f"], s["v"], s["r"], s["h0"], y, h_out=hT, f_bias=s["bias"]), (y, hT)
    rows = dict(f_bias=s["bias"], lengths=s["lengths"], starts=s["starts"])
    if op == "scan_fwd":
        return bl.ScanForward(s["f"], s["v"], s["r"], y, h0=s["h0"], hT=hT, **rows), (y, hT)
    saved = scratch(bl.tern_scan_saved(B, T, D))
    ws = scratch(bl.tern_scan_bwd_workspace(B, T, D))
    df, dv, dr = (torch.empty_like(s["f"]) for _ in range(3))
    dbias, dh0 = new(D), new(B, D)
    fwd = bl.ScanForward(s["f"], s["v"], s["r"], y, h0=s["h0"], hT=hT, saved=saved, **rows)
    bwd = bl.ScanBackward(s["f"], s["v"], s["r"], s["dy"], saved, ws, df, dv, dr, dhT=s["dhT"], dh0=dh0,
                          dbias=dbias, **rows)

    def both():
        fwd()
        bwd()
    return both, (y, hT, df, dv, dr, dbias, dh0)


def run(state):
    if own:
        state["call"]()
        return state["out"]
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- plain forms, fp32

def _plain_embed_fwd(s):
    tok, V = s["tokens"], s["table"].shape[0]
    ok = (tok >= 0) & (tok < V)
    rows = s["table"][tok.clamp(0, V - 1)].float() * s["scale"]
    return torch.where(ok[:, None], rows, torch.zeros_like(rows)).to(torch.bfloat16)


def _plain_embed_bwd(s):
    tok, V = s["tokens"], s["case"]["V"]
    ok = (tok >= 0) & (tok < V)
    rows = torch.where(ok[:, None], s["dout"].float(), torch.zeros((), device="cuda"))
    d = torch.zeros(V, s["case"]["D"], device="cuda")
    d.index_add_(0, tok.clamp(0, V - 1), rows)
    return d * s["scale"]


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by log2(T) steps over the whole tensor."""
    T, k = a.shape[1], 1
    while k < T:
        b = torch.cat([b[:, :k], torch.addcmul(b[:, k:], a[:, k:], b[:, :-k])], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _gates(s):
    """fp32 gates with padding made neutral (a = 1, 1 - a = 0) and document starts (no state before)."""
    f, v, r = s["f"].float() + s["bias"], s["v"].float(), s["r"].float()
    a, na, o = torch.sigmoid(f), torch.sigmoid(-f), torch.sigmoid(r)
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(f.shape[1], device="cuda")[None, :] < s["lengths"][:, None])[..., None]
        a, na, v, o = (torch.where(live, x, torch.full((), z, device="cuda"))
                       for x, z in ((a, 1.0), (na, 0.0), (v, 0.0), (o, 0.0)))
    keep = a
    if s["starts"] is not None:
        st = s["starts"].bool()[..., None]
        if live is not None:
            st = st & live
        keep = torch.where(st, torch.zeros((), device="cuda"), a)
    return keep, a, na, v, o


def _plain_scan_fwd(s):
    keep, _, na, v, o = _gates(s)
    b = na * v
    b[:, 0] += keep[:, 0] * s["h0"]
    h = _doubling(keep, b)
    return (o * h).to(s["f"].dtype), h[:, -1].clone()


def _plain_scan_train(s):
    keep, a, na, v, o = _gates(s)
    b = na * v
    b[:, 0] += keep[:, 0] * s["h0"]
    h = _doubling(keep, b)
    prev = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
    if s["starts"] is not None:
        prev = torch.where(keep == 0, torch.zeros((), device="cuda"), prev)
    dy = s["dy"].float()
    if s["lengths"] is not None:
        live = (torch.arange(h.shape[1], device="cuda")[None, :] < s["lengths"][:, None])[..., None]
        dy = torch.where(live, dy, torch.zeros((), device="cuda"))
    # e_t = keep_t (g_t + e_{t+1}) from the end, e_T = dhT; dh_t = g_t + e_{t+1}
    g = o * dy
    e = keep * g
    e[:, -1] += keep[:, -1] * s["dhT"]
    e = _doubling(keep.flip(1), e.flip(1)).flip(1)
    dh = g + torch.cat([e[:, 1:], s["dhT"][:, None]], 1)
    df = dh * (prev - v) * a * na
    dt = s["f"].dtype
    return ((o * h).to(dt), h[:, -1].clone(), df.to(dt), (dh * na).to(dt), (dy * h * o * (1 - o)).to(dt),
            df.sum((0, 1)), e[:, 0].clone())


def _plain_scan_step(s):
    f, v, r = s["f"].float() + s["bias"], s["v"].float(), s["r"].float()
    h = torch.sigmoid(f) * s["h0"] + torch.sigmoid(-f) * v
    return (torch.sigmoid(r) * h).to(s["f"].dtype), h


def _plain_orthogonalize(s):
    G = s["G"]
    tall = G.shape[0] > G.shape[1]
    X = G.t() if tall else G
    X = X / (torch.sqrt((X * X).sum()) + NS_EPS)
    a, b, c = NS
    for _ in range(5):
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    X = X * s["gain"]
    return (X.t() if tall else X).to(torch.bfloat16).contiguous()


_PLAIN = {"embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd, "scan_fwd": _plain_scan_fwd,
          "scan_train": _plain_scan_train, "scan_step": _plain_scan_step, "orthogonalize": _plain_orthogonalize}


# ---------------------------------------------------------------------------- definitions, fp64

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        tok, V = s["tokens"], case["V"]
        padded = torch.cat([s["table"].double() * s["scale"], torch.zeros(1, case["D"], device="cuda", dtype=torch.float64)])
        return padded[torch.where((tok < 0) | (tok >= V), torch.full_like(tok, V), tok)]
    if op == "embed_bwd":
        tok = s["tokens"]
        at = torch.nonzero((tok >= 0) & (tok < case["V"])).flatten()
        d = torch.zeros(case["V"], case["D"], device="cuda", dtype=torch.float64)
        return d.index_put_((tok[at],), s["dout"][at].double(), accumulate=True).mul_(s["scale"])
    if op == "orthogonalize":
        return _exact_orthogonalize(s)
    if op == "scan_step":
        a = 1 / (1 + torch.exp(-(s["f"].double() + s["bias"].double())))
        h = s["h0"].double() * a + s["v"].double() * (1 - a)
        return h / (1 + torch.exp(-s["r"].double())), h
    return _exact_scan(case, s)


def _exact_orthogonalize(s):
    G = s["G"].double()
    flip = G.shape[0] > G.shape[1]
    X = (G.T if flip else G) / (torch.linalg.vector_norm(G) + NS_EPS)
    for _ in range(5):
        XXt = torch.mm(X, X.T)
        P = NS[0] * torch.eye(X.shape[0], device="cuda", dtype=torch.float64) + NS[1] * XXt + NS[2] * torch.mm(XXt, XXt)
        X = torch.mm(P, X)
    X = X * s["gain"]
    return (X.T if flip else X).contiguous()


def _exact_scan(case, s):
    """One row after the other, in both directions."""
    T, train = case["T"], case["op"] == "scan_train"
    f, v, r, bias = s["f"], s["v"], s["r"], s["bias"].double()
    lengths, starts = s["lengths"], s["starts"]

    def live(t):
        return None if lengths is None else (lengths > t)[:, None]

    def masked(m, x, other):
        return x if m is None else torch.where(m, x, other)

    def first(t):
        return None if starts is None else (starts[:, t] == 0)[:, None]

    h = s["h0"].double()
    zero = torch.zeros_like(h)
    ys, hs = [], [h]
    for t in range(T):
        a = 1 / (1 + torch.exp(-(f[:, t].double() + bias)))
        now = masked(first(t), h, zero) * a + (1 - a) * v[:, t].double()
        h = masked(live(t), now, h)
        ys.append(masked(live(t), h / (1 + torch.exp(-r[:, t].double())), zero))
        hs.append(h)
    y = torch.stack(ys, 1)
    if not train:
        return y, h
    e, sums = s["dhT"].double(), torch.zeros_like(bias)
    dfs, dvs, drs = [None] * T, [None] * T, [None] * T
    for t in reversed(range(T)):
        a = 1 / (1 + torch.exp(-(f[:, t].double() + bias)))
        o = 1 / (1 + torch.exp(-r[:, t].double()))
        dy = s["dy"][:, t].double()
        dh = e + o * dy
        df = dh * (masked(first(t), hs[t], zero) - v[:, t].double()) * a * (1 - a)
        dfs[t] = masked(live(t), df, zero)
        dvs[t] = masked(live(t), dh * (1 - a), zero)
        drs[t] = masked(live(t), dy * hs[t + 1] * o * (1 - o), zero)
        e = masked(live(t), masked(first(t), dh * a, zero), e)
        sums = sums + dfs[t].sum(0)
    return (y, h, torch.stack(dfs, 1), torch.stack(dvs, 1), torch.stack(drs, 1), sums, e)


# ---------------------------------------------------------------------------- work

def _distinct(n, V):
    """Expected number of different ids among n of _tokens."""
    k = torch.arange(1, V + 1, dtype=torch.float64)
    p = torch.log((k + 1) / k) / math.log(V + 1.0) * (31.0 / 32)
    return int((1 - torch.exp(n * torch.log1p(-p))).sum())


def work(case):
    op = case["op"]
    if op == "embed_fwd":
        n, V, D = case["n"], case["V"], case["D"]
        return {"bytes": 8 * n + _distinct(n, V) * D * (4 if case["table"] == "f32" else 2) + 2 * n * D, "flops": n * D}
    if op == "embed_bwd":
        n, V, D = case["n"], case["V"], case["D"]
        return {"bytes": 8 * n + 2 * n * D + 4 * V * D, "flops": 2 * n * D}
    if op == "orthogonalize":
        m, n = sorted((case["K"], case["N"]))
        # the Gram matrix and its square are symmetric: half of each product
        return {"bytes": 6 * m * n, "flops": 5 * (m * m * n + m * m * m + 2 * m * m * n)}
    B, T, D, es = case["B"], case.get("T", 1), case["D"], 2 if case["dtype"] == "bf16" else 4
    e = B * T * D
    if op == "scan_step":
        return {"bytes": 4 * es * e + 8 * e + 4 * D, "flops": 14 * e}
    if op == "scan_fwd":
        return {"bytes": 4 * es * e + 8 * B * D, "flops": 14 * e}
    return {"bytes": 11 * es * e + 16 * B * D, "flops": 40 * e}
