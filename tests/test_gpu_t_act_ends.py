"""Activation functions at the ends of their range and to the last bits, on the GPU.

The error bounds count half steps (U = 2^-24 for FP32) of the evaluation by e = e^-|t|:

    q = e / (1 + e) = s(-|t|),  r = 1 / (1 + e) = s(|t|)
    act(x)  = x - x q  for t > 0,  x q  otherwise
    act'(x) = 1 + q (x t' r - 1)  for t > 0,  q (x t' r + 1)  otherwise

t is x for SiLU and takes seven roundings for GELU, the exponential two half steps more and
1 + e and the quotient one each: q is off by (7 |t| + 4) U relative, and one rounding more
where it is a product.  x t' takes five roundings (GELU), its product with r and the sum four
more with r's own.  So the errors are those of q, which is small wherever the result is
large, and one last rounding.  Below the normal range e is off by a step of the subnormals,
2^-149, and factors up to 320 (x t' where e is not zero) meet it: 2^-138 absolute.  Nothing
grows with |x|.

16-bit results may come from the hardware's 2^x and reciprocal, which take and give
subnormals as zero: where e^|t| is past 2^126 the result may be zero, and there |x| e^-|t|
and |x t'| e^-|t| are below 300 * 2^-126 < 2^-117.  Elsewhere (9 |t| + 8) U and
(18 |t| + 20) U relative to the terms, and 1 - s(t) is off by 4 U absolute while s(t) is not 1
(|t| < 20).
"""
import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs
from gpu_util import log
from test_gpu_o_act import ACTS

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = plain.U


def _parts(x, kind):
    """t, x t', q, r in FP64; x t' is held at +-1e6, where q is zero."""
    t, dt = plain._inner(x, kind)
    with np.errstate(over="ignore", under="ignore"):
        e = np.exp(-np.abs(t))
    return t, np.clip(x * dt, -1e6, 1e6), e / (1 + e), 1 / (1 + e)


def value(x, kind, dt):
    """(act(x), bound before the rounding to dt)."""
    t, _, q, _ = _parts(x, kind)
    y = np.where(t > 0, x - x * q, x * q)
    if dt == "f32":
        b = (np.abs(x * q) * (7 * np.abs(t) + 4) + np.where(t > 0, 0.0, np.abs(y))) * U * 1.01
        return y, np.where(q > 0, b, 0.0) + 2.0 ** -138
    live = np.abs(t) < 200
    return y, np.where(live, np.abs(y) * (9 * np.abs(t) + 8) * U, 0.0) + 2.0 ** -117


def slope(x, kind, dt):
    """(act'(x), bound before the product with dy and the rounding to dt)."""
    t, xt, q, r = _parts(x, kind)
    up = t > 0
    w = xt * r + np.where(up, -1.0, 1.0)
    s = np.where(up, 1.0, 0.0) + q * w
    if dt == "f32":
        b = np.abs(s) + q * (np.abs(xt) * r * (9 + 7 * np.abs(t) * q) +
                             np.abs(w) * (7 * np.abs(t) + 6))
        return s, np.where(q > 0, b, np.abs(s)) * U * 1.01 + 2.0 ** -138
    live = np.abs(t) < 200
    terms = np.where(up, r, q) + np.abs(xt) * q * r
    b = np.where(live, terms * (18 * np.abs(t) + 20) * U, np.abs(s) * 2 * U)
    return s, b + np.where(np.abs(t) < 20, np.abs(xt) * 4 * U, 0.0) + 2.0 ** -117


def rounded(v, bound, dt):
    half_sub = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}[dt]
    return bound + (np.abs(v) + bound) * plain.HALF_EPS[dt] + half_sub


def evaluate(what, h, kind, dt):
    """(result, definition, bound, the inputs it was taken at) of one pass over h."""
    x = h.to(DEV)
    q = torch.empty(h.shape, dtype=torch.uint8, device=DEV)
    e = torch.empty((h.shape[0], -(-h.shape[1] // 32)), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x)
    zs.zero_act_save(q, e, x, act=ACTS[kind], y=out)
    if what == "forward":
        v = plain.f64(h)
        return (plain.f64(out), *value(v, kind, dt), v)
    zs.zero_act_backward(out, torch.ones_like(x), q, e, ACTS[kind])
    v = plain.decode(q.cpu().numpy(), e.cpu().numpy())
    return (plain.f64(out), *slope(v, kind, dt), v)


MAGNITUDES = [1e-40, 2.0 ** -126, 1e-20, 0.75, 12.0, 16.0, 20.0, 44.0, 64.0, 80.0, 86.0, 87.0, 87.5,
              88.0, 88.5, 89.0, 95.0, 100.0, 103.0, 104.0, 105.0, 110.0, 120.0, 126.0, 128.0, 130.0,
              200.0, 1e3, 1e4, 6e4, 1e6, 1e12, 1e20, 1e30, 1e36, 1e37, 1e38, 3e38]


@pytest.mark.parametrize("kind", ["gelu", "silu"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("what", ["forward", "slope"])
def test_far_inputs(what, dt, kind):
    # each alone in its block, of both signs, so that its checkpoint is within 2^-4 of it
    m = [v for v in MAGNITUDES if v < (6.2e4 if dt == "f16" else 3.1e38)] + [plain.TOP[dt]]
    h = torch.zeros(2 * len(m), 32)
    for i, v in enumerate(m):
        h[2 * i, i % 32], h[2 * i + 1, i % 32] = v, -v
    got, want, bound, x = evaluate(what, h.to(plain.TORCH[dt]), kind, dt)
    assert np.isfinite(got).all()
    tol = rounded(want, bound, dt)
    bad = [(float(x[i, j]), float(got[i, j]), float(want[i, j]), float(tol[i, j]))
           for i, j in np.argwhere(np.abs(got - want) > tol)]
    assert not bad, bad


@pytest.mark.parametrize("kind", ["gelu", "silu"])
@pytest.mark.parametrize("what", ["forward", "slope"])
def test_fp32_to_the_last_bits(what, kind):
    g = torch.Generator().manual_seed(21)
    got, want, bound, _ = evaluate(what, torch.randn(1024, 1024, generator=g) * 2, kind, "f32")
    worst = float((np.abs(got - want) / rounded(want, bound, "f32")).max())
    log(f"  {kind} FP32 {what}: worst {worst:.2f} of the bound, error "
        f"{np.linalg.norm(got - want) / np.linalg.norm(want):.3g} of the norm")
    assert worst <= 1


@pytest.mark.parametrize("kind", ["gelu", "silu"])
@pytest.mark.parametrize("what", ["forward", "slope"])
def test_fp32_no_further_off_than_the_elementary_form(what, kind):
    # error over 2^20 normal values against 64 bits, next to the formulas in elementary FP32
    # operations: the form by e^-|t| has the fewer roundings where the results are large
    g = torch.Generator().manual_seed(22)
    got, want, _, v = evaluate(what, torch.randn(1024, 1024, generator=g), kind, "f32")
    x, c, a = torch.from_numpy(v).float(), float(plain.GELU_C), plain.GELU_A
    if kind == "silu":
        s = 1 / (1 + torch.exp(-x))
        form = x / (1 + torch.exp(-x)) if what == "forward" else s + x * s * (1 - s)
    else:
        t = torch.tanh(c * (x + a * x * x * x))
        form = 0.5 * x * (1 + t) if what == "forward" else \
            0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * a * x * x)
    ours, theirs = np.linalg.norm(got - want), np.linalg.norm(plain.f64(form) - want)
    assert ours <= theirs


def test_infinite_inputs_of_the_forward_pass():
    for dt in ("f16", "bf16", "f32"):
        for kind in ("gelu", "silu"):
            h = torch.zeros(1, 64, dtype=plain.TORCH[dt])
            h[0, 3], h[0, 40], h[0, 41] = float("inf"), float("nan"), 100.0
            with np.errstate(invalid="ignore"):
                y = evaluate("forward", h, kind, dt)[0]
            assert y[0, 3] == np.inf and np.isnan(y[0, 40]) and y[0, 41] == 100.0
            assert np.isfinite(np.delete(y[0], [3, 40])).all()
