"""The references of the recurrence's gradient against central differences, in fp64 on the CPU."""
import numpy as np
import pytest

from _reference import scan


@pytest.mark.parametrize("B,T,D,masks", [(2, 7, 3, False), (3, 9, 2, True), (1, 1, 1, False)])
def test_scan_gradient_formulas_match_differences(B, T, D, masks):
    rng = np.random.default_rng(B * 100 + T)
    x = {k: rng.normal(size=(B, T, D)) for k in ("f", "v", "r")}
    x["bias"], x["h0"] = rng.normal(size=D), rng.normal(size=(B, D))
    lengths = np.array([0, T - 2, T][:B]) if masks else None
    starts = (rng.random((B, T)) < 0.3).astype(np.uint8) if masks else None
    dy, dhT = rng.normal(size=(B, T, D)), rng.normal(size=(B, D))

    def loss(z):
        o = scan(z["f"], z["v"], z["r"], z["bias"], z["h0"], lengths, starts)
        return (o["y"][0] * dy).sum() + (o["hT"][0] * dhT).sum()

    got = scan(x["f"], x["v"], x["r"], x["bias"], x["h0"], lengths, starts, dy, dhT)
    for k, name in (("f", "df"), ("v", "dv"), ("r", "dr"), ("bias", "dbias"), ("h0", "dh0")):
        g = got[name][0]
        for i in np.ndindex(*x[k].shape):
            step = 1e-5
            hi, lo = {**x, k: x[k].copy()}, {**x, k: x[k].copy()}
            hi[k][i] += step
            lo[k][i] -= step
            num = (loss(hi) - loss(lo)) / (2 * step)
            assert abs(num - g[i]) <= 1e-8 * (1 + abs(num)), (name, i, num, g[i])
