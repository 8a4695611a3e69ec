"""Plain fp64 references (numpy) of the operators around the ternary projections, with bounds
on what fp32 arithmetic may differ by, carried through the same formulas.

U is half an fp32 ulp at 1.  A gate sigmoid(x) is taken as good to (6 + 1.2 |x|) 2^-23
relative: CUDA documents __expf with 2 + 1.173 |x| ulp and __fdividef with 2 ulp."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def gate_err(x):
    return (6.0 + 1.2 * np.minimum(np.abs(x), 90.0)) * 2.0 * U


def scan(f, v, r, bias=None, h0=None, lengths=None, starts=None, dy=None, dhT=None):
    """Row by row.  Returns a dict of y, hT and, with dy, df, dv, dr, dbias, dh0, each as
    (value, error bound of fp32 arithmetic before the output's own rounding)."""
    B, T, D = f.shape
    f, v, r = (x.astype(np.float64) for x in (f, v, r))
    x = f + (0.0 if bias is None else bias.astype(np.float64))
    a, n, o, no = sigmoid(x), sigmoid(-x), sigmoid(r), sigmoid(-r)
    ea, eo = gate_err(x) + U * 4, gate_err(r) + U * 4      # + the addition of the bias and the products
    live = np.ones((B, T), bool) if lengths is None else np.arange(T)[None] < np.clip(lengths, 0, T)[:, None]
    st = np.zeros((B, T), bool) if starts is None else (starts != 0) & live
    h = np.zeros((B, D)) if h0 is None else h0.astype(np.float64)
    hA, E = np.abs(h), np.zeros((B, D))
    H, HA, HE, HP, HPA, HPE = (np.zeros((B, T, D)) for _ in range(6))
    y, ye = np.zeros((B, T, D)), np.zeros((B, T, D))
    for t in range(T):
        c = st[:, t, None]
        hp, hpA, hpE = (np.where(c, 0.0, z) for z in (h, hA, E))
        b = n[:, t] * v[:, t]
        hn = a[:, t] * hp + b
        hnA = a[:, t] * hpA + np.abs(b)
        hnE = a[:, t] * hpE + ea[:, t] * hnA
        L = live[:, t, None]
        h, hA, E = np.where(L, hn, h), np.where(L, hnA, hA), np.where(L, hnE, E)
        H[:, t], HA[:, t], HE[:, t], HP[:, t], HPA[:, t], HPE[:, t] = h, hA, E, hp, hpA, hpE
        y[:, t] = np.where(L, o[:, t] * h, 0.0)
        ye[:, t] = np.where(L, o[:, t] * (E + eo[:, t] * hA), 0.0)
    out = {"y": (y, ye), "hT": (h, E)}
    if dy is None:
        return out
    dy = dy.astype(np.float64)
    e = np.zeros((B, D)) if dhT is None else dhT.astype(np.float64)
    eA, eE = np.abs(e), np.zeros((B, D))
    g = {k: (np.zeros((B, T, D)), np.zeros((B, T, D))) for k in ("df", "dv", "dr")}
    sb, sbA, sbE = np.zeros(D), np.zeros(D), np.zeros(D)
    for t in reversed(range(T)):
        L, c = live[:, t, None], st[:, t, None]
        gt = np.where(L, o[:, t] * np.where(L, dy[:, t], 0.0), 0.0)
        dh, dhA = gt + e, np.abs(gt) + eA
        dhE = eE + eo[:, t] * dhA
        w = a[:, t] * n[:, t]
        diff, diffA = HP[:, t] - v[:, t], HPA[:, t] + np.abs(v[:, t])
        df = dh * w * diff
        dfE = w * (np.abs(diff) * dhE + dhA * HPE[:, t] + 4 * ea[:, t] * dhA * diffA)
        dyt = np.where(L, dy[:, t], 0.0)
        wr = o[:, t] * no[:, t]
        for k, val, err in (("df", df, dfE), ("dv", n[:, t] * dh, n[:, t] * (dhE + 2 * ea[:, t] * dhA)),
                            ("dr", dyt * H[:, t] * wr, np.abs(dyt) * wr * (HE[:, t] + 4 * eo[:, t] * HA[:, t]))):
            g[k][0][:, t], g[k][1][:, t] = np.where(L, val, 0.0), np.where(L, err, 0.0)
        sb += g["df"][0][:, t].sum(0)
        sbA += np.abs(g["df"][0][:, t]).sum(0)
        sbE += g["df"][1][:, t].sum(0)
        en, enA, enE = (np.where(c, 0.0, z) for z in (a[:, t] * dh, a[:, t] * dhA, a[:, t] * (dhE + ea[:, t] * dhA)))
        e, eA, eE = np.where(L, en, e), np.where(L, enA, eA), np.where(L, enE, eE)
    out.update(g)
    out["dbias"] = (sb, sbE + sbA * (B * T + 8) * U)
    out["dh0"] = (e, eE)
    return out


def embed_bwd(tok, dout, V, scale):
    """(gradient of the table, error bound of fp32 sums in any order)."""
    n, D = dout.shape
    d, ab, cnt = np.zeros((V, D)), np.zeros((V, D)), np.zeros(V)
    ok = (tok >= 0) & (tok < V)
    np.add.at(d, tok[ok], dout[ok].astype(np.float64))
    np.add.at(ab, tok[ok], np.abs(dout[ok].astype(np.float64)))
    np.add.at(cnt, tok[ok], 1)
    s = float(np.float32(scale))
    return d * s, ab * abs(s) * (cnt[:, None] + 3) * U


def bf16(x):
    """Round to bf16 (nearest even) and back, through torch."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def check(name, got, ref, bound):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{name}: non-finite output"
    err = np.abs(got - ref)
    bad = err > bound
    if bad.any():
        i = np.unravel_index(np.argmax(err - bound), err.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside the bound; worst at {i}: "
                             f"got {got[i]!r}, reference {ref[i]!r}, |err| {err[i]:.3e}, bound {bound[i]:.3e}")
