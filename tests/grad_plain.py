"""64-bit definitions of the gradient operators and their error bounds, for the tests.

Everything is NumPy in FP64 from the formulas; the e4m3 rounding is a search in the
table of the format's values.  U is half a step of FP32, the largest relative error
of one FP32 operation.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_EPS = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # one rounding, relative
HALF_SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -126}  # near zero (FP32: flush)
TOP = {"f16": 15.0 * 2.0 ** 12, "bf16": 15.0 * 2.0 ** 124, "f32": 15.0 * 2.0 ** 124}


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def _code_values() -> np.ndarray:
    """Value of each of the 128 non-negative e4m3 codes (127 is NaN)."""
    c = np.arange(128)
    e, m = c >> 3, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[127] = np.nan
    return v


CODE_VALUES = _code_values()
_MID = (CODE_VALUES[:126] + CODE_VALUES[1:127]) / 2     # border between code c and c + 1


def encode(x: np.ndarray, dt: str):
    """(q, e) of the 8-bit checkpoint of x (FP64 copies of format-dt values)."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    fin = np.isfinite(b)
    amax = np.abs(np.where(fin, b, 0)).max(-1)
    k = np.full(amax.shape, -124)
    while True:
        up = amax > 448.0 * np.ldexp(1.0, k)
        if not up.any():
            break
        k = k + up
    v = np.ldexp(np.minimum(np.abs(np.where(fin, b, 0)), TOP[dt]), -k[..., None])
    lo = np.searchsorted(_MID, v, side="left")           # codes whose upper border is < v
    tie = (lo < 126) & (v == _MID[np.minimum(lo, 125)])
    code = lo + (tie & (lo % 2 == 1))                    # a tie goes to the even code
    code = np.where(fin, code, 127) | (np.signbit(b).astype(int) << 7)
    q = code.reshape(rows, -1)[:, :cols].astype(np.uint8)
    return q, (k + 127).astype(np.uint8)


def decode(q: np.ndarray, e: np.ndarray) -> np.ndarray:
    v = CODE_VALUES[q & 127] * np.where(q > 127, -1.0, 1.0)
    k = np.repeat(e.astype(int), 32, axis=1)[:, :q.shape[1]] - 127
    return np.ldexp(v, k)


def _sig(t):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t))


GELU_C, GELU_A = np.sqrt(2.0 / np.pi), 0.044715


def _inner(x, act):
    """t and dt/dx of act(x) = x s(t)."""
    if act == "silu":
        return x, np.ones_like(x)
    return 2 * GELU_C * (x + GELU_A * x ** 3), 2 * GELU_C * (1 + 3 * GELU_A * x ** 2)


def act(x, kind):
    """(value, bound on the FP32 evaluation's error).

    t takes seven FP32 roundings at most (three products, a sum, a product and two
    constants), x log2 e two more, all without cancellation, so the exponent is off by at
    most 9 U |t|; 2^x and the reciprocal are within 2 U each and two more operations
    round: a relative error of (9 |t| + 6) U, held at (9 |t| + 8) U.  Below e^-87 the
    logistic leaves FP32's normal range: |x| 2^-125 absolute."""
    t, _ = _inner(x, kind)
    y = x * _sig(t)
    return y, np.abs(y) * (9 * np.abs(t) + 8) * U + np.abs(x) * 2.0 ** -125


def act_slope(x, kind):
    """(slope, bound): s + x s(t) s(-t) t', each factor as in act; the sum may cancel, so the
    bound goes by the terms' magnitudes; two factors carry the exponent's error, and eleven
    more roundings at most."""
    t, dt = _inner(x, kind)
    s, o = _sig(t), _sig(-t)
    a, b = s, x * s * o * dt
    return a + b, (np.abs(a) + np.abs(b)) * (18 * np.abs(t) + 20) * U + \
        (1 + np.abs(x) * dt * o) * 2.0 ** -125


def rounded(value, bound, dt):
    """Bound on a result that is computed within `bound` and rounded once to dt."""
    return bound + (np.abs(value) + bound) * HALF_EPS[dt] + HALF_SUB[dt]


def lookup(table, ids, scale):
    """FP32 product, rounded once more by the caller's cast: exact to the bit."""
    out = np.zeros((len(ids), table.shape[1]), np.float32)
    ok = (ids >= 0) & (ids < table.shape[0])
    out[ok] = table.astype(np.float32)[ids[ok]] * np.float32(scale)
    return out


def embed_grad(dy, ids, vocab, scale):
    """(G, bound): a run of n rows takes n - 1 FP32 additions, whatever their grouping, and
    the scale one product: n U times the sum of magnitudes."""
    g, mag, n = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1])), np.zeros(vocab)
    ok = (ids >= 0) & (ids < vocab)
    np.add.at(g, ids[ok], dy[ok])
    np.add.at(mag, ids[ok], np.abs(dy[ok]))
    np.add.at(n, ids[ok], 1)
    s = float(np.float32(scale))
    return g * s, mag * abs(s) * n[:, None] * U * 1.01


def weight_grad(dy, v):
    """(G, bound): products are exact; T FP32 additions in any order, each off by at most a
    whole step of FP32 (2 U) whether the matrix unit rounds or truncates."""
    return dy.T @ v, (np.abs(dy).T @ np.abs(v)) * dy.shape[0] * 2 * U


def policy(z, targets, old, ref, adv, w, lo, hi, kl, S):
    """Outputs and bounds of the policy loss, FP64.  z: FP64 copies of the logits."""
    rows, V = z.shape
    f = lambda x: float(np.float32(x))
    low, high, kl = f(np.float32(1) - np.float32(lo)), f(np.float32(1) + np.float32(hi)), f(kl)
    out = {k: np.zeros(rows) for k in ("token_loss", "logp", "b_token", "b_logp")}
    dz, b_dz = np.zeros((rows, V)), np.zeros((rows, V))
    near = np.zeros(rows, bool)      # the clip border lies within the ratio's error
    for t in range(rows):
        if w[t] == 0:
            continue
        if not 0 <= targets[t] < V:
            for k in out:
                out[k][t] = np.nan
            dz[t] = np.nan
            continue
        m = z[t].max()
        x = np.where(np.isneginf(z[t]), -1e4, z[t] - m)
        ex = np.where(np.isneginf(z[t]), 0.0, np.exp(x))
        s = ex.sum()
        p = ex / s
        # e^x: the difference and the product with log2 e round (and its constant): 3 U |x|,
        # 2^x itself 2 U; the sum adds at most 24 * 8 terms a lane, then a tree over 1024
        # lanes, or V / 1024 a lane
        n_add = 208 + V / 1024
        e_sum = (ex * (3 * np.abs(x) + 4)).sum() / s * U + n_add * U
        xa = x[targets[t]]
        logp = xa - np.log(s)
        e_logp = (abs(xa) + 3 * abs(np.log(s)) + abs(logp) + 2) * U + e_sum
        old_t = old[t] if old is not None else logp
        r = np.exp(logp - old_t)
        e_r = 0.0 if old is None else r * (e_logp + (2 * abs(logp - old_t) + 4) * U)
        rc = min(max(r, low), high)
        A = adv[t]
        L = max(-r * A, -rc * A)
        cut = (A > 0 and r > high) or (A < 0 and r < low)
        near[t] = min(abs(r - low), abs(r - high)) <= e_r
        g = 0.0 if cut else -A * r
        e_L, e_g = abs(A) * e_r + abs(L) * 2 * U, abs(A) * e_r + abs(g) * U
        if ref is not None and kl != 0:
            d = ref[t] - logp
            e_d = e_logp + abs(d) * U
            em = np.expm1(d)
            e_em = abs(em) * 4 * U + np.exp(d) * e_d * 1.01
            L += kl * (em - d)
            g -= kl * em
            e_L += kl * (abs(em) * e_d * 1.01 + (abs(em) * 5 + abs(em - d) + abs(d)) * U * 2)
            e_g += kl * (e_em + abs(em) * U)
            e_L += abs(L) * U
            e_g += abs(g) * U
        c = S * w[t] * g
        e_c = S * abs(w[t]) * e_g + abs(c) * 2 * U
        out["token_loss"][t], out["logp"][t] = L, logp
        out["b_token"][t], out["b_logp"][t] = e_L * 1.01, e_logp * 1.01
        dz[t] = -c * p
        dz[t, targets[t]] += c
        e_p = p * ((3 * np.abs(x) + 8) * U + e_sum)
        b_dz[t] = (abs(c) * e_p + p * e_c + abs(c) * p * 3 * U) * 1.01
        b_dz[t, targets[t]] += (e_c + abs(dz[t, targets[t]]) * U) * 1.01
    out["loss"] = float((out["token_loss"] * w)[w != 0].sum())
    out["b_loss"] = float((out["b_token"] * np.abs(w))[w != 0].sum() + abs(out["loss"]) * U)
    out["dlogits"], out["b_dlogits"], out["near"] = dz, b_dz, near
    return out
