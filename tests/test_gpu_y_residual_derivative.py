"""The backward step between two blocks against the derivative of the forward pass itself, in 64
bits from r and f (and not from the stream and the statistics that the forward pass left).

The forward pass makes h from the sum before it rounds u to the stream's format; the backward
pass has the rounded u.  So its normalised row is off by delta, at most half a step of u over
the row's deviation, and by what the statistics are off.  The bounds carry delta through the
formulas: Sum |dh| delta for the pre norm's weight, and for G = du + rho (g - [mean g] -
z mean(g z)) rho (|z| c' + |c| delta + c' delta), c = mean(g z), c' = mean(|g| delta)."""
import numpy as np
import pytest
import torch

import block_plain as plain
import zero_sharded_mixed_shard_amd as zs
from test_gpu_y_residual import Case, DEV, F64

pytestmark = pytest.mark.gpu
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
ALL = ("w1", "b1", "gate", "w2", "b2")


def both_passes(c):
    """What the two calls give: the backward pass on what the forward pass left."""
    d = lambda t: t.to(DEV)
    told = c.told()
    r, f, dh, du = d(c.r), d(c.f), d(c.dh), d(c.du)
    u, h, stats = torch.zeros_like(r), torch.zeros_like(f), torch.zeros(c.rows, 4, device=DEV)
    zs.zero_residual_norm(u, h, stats, r, f, **told)
    df, dr = torch.zeros_like(f), torch.zeros_like(r)
    g = {k: None if c.par[k] is None else torch.zeros(c.cols, device=DEV) for k in ALL}
    ws = torch.empty(zs.zero_residual_norm_workspace(c.rows, c.cols), dtype=torch.uint8,
                     device=DEV)
    zs.zero_residual_norm_backward(
        df, dr, dh, du, f, u, stats, workspace=ws, d_post_weight=g["w1"], d_post_bias=g["b1"],
        d_gate=g["gate"], d_pre_weight=g["w2"], d_pre_bias=g["b2"], **told)
    return u, stats, dict(df=df, dr=dr, **g)


def moved(g, eg, z, dz, rho, rel, kind):
    """By how much a norm's Jacobian product changes where g, z and rho (relatively) do."""
    c = np.abs((g * z).mean(1, keepdims=True))
    dc = (np.abs(g) * dz + eg * (np.abs(z) + dz)).mean(1, keepdims=True)
    e = eg + (eg.mean(1, keepdims=True) if kind == "layer" else 0.0)
    e = e + np.abs(z) * dc + dz * c + dz * dc
    t = np.abs(g) + np.abs(z) * c + \
        (np.abs(g.mean(1, keepdims=True)) if kind == "layer" else 0.0)
    return rho * (e * (1 + rel) + t * rel)


def allowance(c, stats, exact_stats):
    """{name: how far each gradient may be from the forward pass's derivative} besides the
    backward pass's own rounding."""
    P = c.P
    one = lambda k, other: np.full(c.cols, other) if P[k] is None else P[k]
    u, eu, _, _, _ = plain.forward(F64(c.r), F64(c.f), P)
    got = F64(stats)
    shift = np.abs(got - exact_stats)
    out = {}
    mean, rho = exact_stats[:, 2:3], exact_stats[:, 3:4]
    rel = shift[:, 3:4] / rho
    z = (u - mean) * rho
    # The u in memory is the FP32 sum, off by eu (the norm, its weight, bias and gate, the mask's
    # factor and the sum round one after the other; the forward pass is held to the same bound),
    # rounded to the stream's format.  In FP32 eu is all there is: without it a stream in FP32 was
    # allowed one rounding of u for the six and more that make it.
    off = eu + (np.abs(u) + eu) * HALF_STEP[c.res] + plain.TINY + shift[:, 2:3]
    dz = off * rho * (1 + rel) + np.abs(z) * rel
    dh = F64(c.dh)
    g = one("w2", 1.0) * dh
    out["w2"], out["b2"] = (np.abs(dh) * dz).sum(0), np.zeros(c.cols)
    eG = moved(g, np.zeros_like(g), z, dz, rho, rel, P["pre"])
    out["dr"] = abs(P["scale"]) * eG
    back = g - z * (g * z).mean(1, keepdims=True)
    if P["pre"] == "layer":
        back = back - g.mean(1, keepdims=True)
    G = F64(c.du) + rho * back
    keep, k = plain.mask(c.rows, c.cols, P["p"], P["seed"], P["offset"])
    G, eG = np.where(keep, G * float(k), 0), np.where(keep, eG * float(k), 0)
    mean, rho = exact_stats[:, 0:1], exact_stats[:, 1:2]
    rel = shift[:, 1:2] / rho
    z = (F64(c.f) - mean) * rho
    dz = shift[:, 0:1] * rho * (1 + rel) + np.abs(z) * rel
    a, b = (np.abs(G) * dz + eG * (np.abs(z) + dz)).sum(0), eG.sum(0)
    w, bias, gate = one("w1", 1.0), one("b1", 0.0), one("gate", 1.0)
    out["w1"], out["b1"] = np.abs(gate) * a, np.abs(gate) * b
    out["gate"] = np.abs(w) * a + np.abs(bias) * b
    out["df"] = np.abs(gate) * eG if P["post"] == "none" else moved(
        w * gate * G, np.abs(w * gate) * eG, z, dz, rho, rel, P["post"])
    return out


@pytest.mark.parametrize("rows,cols", [(40, 300), (33, 4096), (5, 12288), (3, 17000)])
@pytest.mark.parametrize("dt,res", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                    ("f32", "f32")])
@pytest.mark.parametrize("post,pre,mean", [("rms", "layer", 0.0), ("rms", "layer", 20.0),
                                           ("none", "rms", 5.0), ("layer", "layer", 100.0)])
def test_against_the_forward_passes_derivative(rows, cols, dt, res, post, pre, mean):
    # (rows of u lie about 0.8 mean deviations from zero)
    c = Case(rows, cols, dt, res, post, pre, mean=mean, gate=True)
    _, stats, got = both_passes(c)
    u64, _, _, _, st = plain.forward(F64(c.r), F64(c.f), c.P)
    exact = plain.backward(F64(c.dh), F64(c.du), F64(c.f), u64, st, c.P)
    more = allowance(c, stats, st)
    for k, t in got.items():
        if t is None:
            continue
        v, e = exact[k]
        fmt = {"df": dt, "dr": res}.get(k, "f32")
        assert np.all(np.abs(F64(t) - v) <= plain.rounded(v, (e + more[k]) * 1.01, fmt)), k


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_a_norm_of_its_own_takes_the_stored_stream(dt):
    # rows a hundred deviations from zero on a 16-bit stream: with the norm in a call of its own
    # (no f, r the stored u) both passes see the same row, and the weight's gradient is that of
    # h = pre(u) within FP32's rounding
    c = Case(60, 2000, dt, dt, "none", "layer", mean=100.0, p=0.0, scale=1.0, gate=False)
    d = lambda t: t.to(DEV)
    told = c.told()
    r, f = d(c.r), d(c.f)
    u, h = torch.zeros_like(r), torch.zeros_like(f)
    stats = torch.zeros(60, 4, device=DEV)
    first = dict(told, pre=zs.NORM_NONE, pre_weight=None, pre_bias=None)
    zs.zero_residual_norm(u, None, None, r, f, **first)
    zs.zero_residual_norm(None, h, stats, u, **told)
    dr, g = torch.zeros_like(u), torch.zeros(2000, device=DEV)
    ws = torch.empty(zs.zero_residual_norm_workspace(60, 2000), dtype=torch.uint8, device=DEV)
    zs.zero_residual_norm_backward(None, dr, d(c.dh), d(c.du), None, u, stats, d_pre_weight=g,
                                   workspace=ws, **told)
    _, _, wh, eh, st = plain.forward(F64(u), None, c.P)
    assert np.all(np.abs(F64(h) - wh) <= plain.rounded(wh, eh, dt))
    exact = plain.backward(F64(c.dh), F64(c.du), None, F64(u), st, c.P)
    # besides: the statistics are FP32 (as found, a bound on them is checked elsewhere)
    shift = np.abs(F64(stats) - st)
    z = (F64(u) - st[:, 2:3]) * st[:, 3:4]
    rel = shift[:, 3:4] / st[:, 3:4]
    dz = shift[:, 2:3] * st[:, 3:4] * (1 + rel) + np.abs(z) * rel
    assert float(dz.max()) < 2.0 ** -12
    v, e = exact["w2"]
    more = (np.abs(F64(c.dh)) * dz).sum(0)
    assert np.all(np.abs(F64(g) - v) <= plain.rounded(v, (e + more) * 1.01, "f32"))
