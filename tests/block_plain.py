"""64-bit definitions of the operators around a block's linear layers and their error
bounds, for the tests.

Everything is NumPy in FP64 (the generator in unsigned 64-bit words) from the formulas.  U
is half a step of FP32, the largest relative error of one FP32 operation.
"""
from __future__ import annotations

import numpy as np

from grad_plain import CODE_VALUES, TOP, U, _MID, rounded  # noqa: F401

BLOCK = 128
TINY = 2.0 ** -118          # what FP32's and the formats' smallest numbers may cost


def _tiles(x, tall, block):
    """x padded with zeros to whole blocks, [blocks down, tall, blocks across, block]."""
    rows, cols = x.shape
    nr, nc = -(-rows // tall), -(-cols // block)
    p = np.zeros((nr * tall, nc * block))
    p[:rows, :cols] = x
    return p.reshape(nr, tall, nc, block)


def _spread(e, shape, tall, block):
    return np.repeat(np.repeat(e, tall, 0)[:shape[0]], block, 1)[:, :shape[1]]


def encode(x, dt, tall=1, block=BLOCK):
    """(q, e) of x (FP64 copies of format-dt values): nearest code, ties to the even one."""
    fin = np.isfinite(x)
    mag = np.abs(np.where(fin, x, 0.0))
    amax = _tiles(mag, tall, block).max((1, 3))
    k = np.full(amax.shape, -124)
    while True:
        up = amax > 448.0 * np.ldexp(1.0, k)
        if not up.any():
            break
        k = k + up
    v = np.ldexp(np.minimum(mag, TOP[dt]), -_spread(k, x.shape, tall, block))
    lo = np.searchsorted(_MID, v, side="left")
    tie = (lo < 126) & (v == _MID[np.minimum(lo, 125)])
    code = lo + (tie & (lo % 2 == 1))
    code = np.where(fin, code, 127) | (np.signbit(x).astype(int) << 7)
    return code.astype(np.uint8), (k + 127).astype(np.uint8)


def decode(q, e, tall=1, block=BLOCK):
    v = CODE_VALUES[q & 127] * np.where(q > 127, -1.0, 1.0)
    return np.ldexp(v, _spread(e.astype(int), q.shape, tall, block) - 127)


def product(a, b, dt):
    """(y, bound).  FP32: exact products, k additions in any order, each off by at most a step
    of FP32 (2 U) whether the matrix unit rounds or truncates.  16-bit: from each product of a
    group of eight a part below 2^-13 of the group's largest may be lost, seven such parts a
    group: 7 * 2^-13 <= 2^-10 of the sum of magnitudes."""
    y, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    e = mag * (a.shape[1] * 2 * U + (0.0 if dt == "f32" else 2.0 ** -10))
    return y, rounded(y, e, dt)


# ---- the mask ------------------------------------------------------------------------------

M32 = np.uint64(0xffffffff)


def philox(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., 2011) of arrays of counters (four uint64 arrays of 32-bit
    words) under a key (two numbers)."""
    c, k = [np.asarray(x, np.uint64) for x in counter], [int(x) for x in key]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & M32,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & M32]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def threshold(p):
    return int(np.rint(np.float64(np.float32(p)) * 65536.0))


def mask(rows, cols, p, seed, offset):
    """(keep [rows, cols], factor as FP32)."""
    groups = -(-cols // 8)
    g, r = np.meshgrid(np.arange(groups), np.arange(rows))
    offset %= 2 ** 64
    c = philox((g, r, np.full_like(g, offset % 2 ** 32), np.full(g.shape, offset >> 32)),
               (seed % 2 ** 32, seed >> 32))
    halves = [h for w in c for h in (w & np.uint64(0xffff), w >> np.uint64(16))]
    bits = np.stack(halves, -1).reshape(rows, groups * 8)[:, :cols]
    t = threshold(p)
    f = np.float32(0.0) if t == 65536 else np.float32(65536.0) / np.float32(65536 - t)
    return bits >= t, f


def dropout(x, p, seed, offset):
    """FP32 array of the result before its rounding to the format; exact to the bit."""
    keep, f = mask(*x.shape, p, seed, offset)
    with np.errstate(over="ignore", invalid="ignore"):
        return np.where(keep, x.astype(np.float32) * f, np.float32(0.0))


# ---- the step between two blocks -------------------------------------------------------------

def row_adds(cols):
    """FP32 additions that any element of a row's sum goes through, at most: eight a group of
    a lane that owns every 2048th element or more, then a tree over a workgroup."""
    return 32 + cols // 256


def normed(x, ex, kind, eps):
    """(z, bound, mean, rho) of each row of x known within ex.

    The mean takes row_adds additions and a division; the deviation from it one rounding;
    the squares' sum is at its least around the true mean, so an error of the mean enters by
    its square; sqrt, the quotient and the sum with eps round."""
    cols = x.shape[1]
    n = row_adds(cols)
    layer = kind == "layer"
    mean = x.mean(1, keepdims=True) if layer else np.zeros((x.shape[0], 1))
    em = ((np.abs(x).mean(1, keepdims=True) * (n + 2) * U + ex.mean(1, keepdims=True))
          if layer else np.zeros_like(mean))
    d = x - mean
    ed = ex + em + np.abs(d) * U
    var = (d * d).mean(1, keepdims=True)
    e_var = var * (n + 4) * U + (2 * np.abs(d) * ex + (ed * ed)).mean(1, keepdims=True) * 1.01 \
        + 2 * U * (d * d).mean(1, keepdims=True)
    rho = 1.0 / np.sqrt(var + eps)
    rel = 0.5 * e_var / (var + eps) * 1.02 + 4 * U
    z = d * rho
    return z, np.abs(z) * (rel + 2 * U) + rho * ed * 1.01, mean[:, 0], rho[:, 0]


def forward(r, f, P):
    """(u, e_u, h, e_h, stats) in FP64; P: dict of post, pre ('none', 'rms', 'layer'), w1, b1,
    gate, w2, b2 (arrays or None), eps, scale, p, seed, offset.  f None: u is r."""
    rows, cols = r.shape
    one = lambda name, other: np.full(cols, other) if P.get(name) is None else P[name]
    eps, s = float(np.float32(P["eps"])), float(np.float32(P["scale"]))
    stats = np.tile(np.array([0.0, 1.0, 0.0, 1.0]), (rows, 1))
    u, eu = r, np.zeros_like(r)
    if f is not None:
        z, ez = f, np.zeros_like(f)
        if P["post"] != "none":
            z, ez, stats[:, 0], stats[:, 1] = normed(f, ez, P["post"], eps)
        w, b, g = one("w1", 1.0), one("b1", 0.0), one("gate", 1.0)
        n = z * w + b
        en = np.abs(w) * ez + (np.abs(z * w) + np.abs(n)) * U
        v, ev = n * g, np.abs(g) * en + np.abs(n * g) * U
        if threshold(P["p"]):
            keep, k = mask(rows, cols, P["p"], P["seed"], P["offset"])
            v, ev = np.where(keep, v * float(k), 0), np.where(keep, ev * float(k), 0)
            ev = ev + np.abs(v) * U
        u = s * r + v
        eu = ev * 1.01 + (np.abs(s * r) + np.abs(u)) * U + TINY
    if P["pre"] == "none":
        return u, eu, None, None, stats
    z, ez, stats[:, 2], stats[:, 3] = normed(u, eu, P["pre"], eps)
    w, b = one("w2", 1.0), one("b2", 0.0)
    h = z * w + b
    return u, eu, h, np.abs(w) * ez * 1.01 + (np.abs(z * w) + np.abs(h)) * U + TINY, stats


def backward(dh, du, f, u, stats, P):
    """{name: (gradient, bound)} for dr, df and the parameters, from the statistics as they
    are held (FP32 values).

    A normalised value takes two roundings; a mean of products row_adds additions more than
    its products' own; each difference and product one.  Sums over the rows take one addition
    a row at most, whatever their grouping."""
    rows, cols = u.shape
    one = lambda name, other: np.full(cols, other) if P.get(name) is None else P[name]
    n, s = row_adds(cols), float(np.float32(P["scale"]))
    out = {}

    def column(name, terms, e_terms, factor=1.0):
        t = terms.sum(0) * factor
        e = (e_terms.sum(0) + np.abs(terms).sum(0) * (rows + 1) * U) * np.abs(factor)
        out[name] = (t, e * 1.01 + np.abs(t) * U + TINY)

    def through(g, eg, z, rho, kind):
        """A norm's Jacobian on g known within eg."""
        ez = 2 * U * np.abs(z)
        gz = g * z
        c = gz.mean(1, keepdims=True)
        ec = (np.abs(gz) * (n + 2) * U + np.abs(z) * eg + np.abs(g) * ez).mean(1, keepdims=True)
        c0, e0 = np.zeros_like(c), np.zeros_like(c)
        if kind == "layer":
            c0 = g.mean(1, keepdims=True)
            e0 = (np.abs(g) * (n + 2) * U + eg).mean(1, keepdims=True)
        t = g - c0 - z * c
        mag = np.abs(g) + np.abs(c0) + np.abs(z * c)
        et = eg + e0 + np.abs(z) * ec * 1.01 + np.abs(c) * ez + 5 * U * mag
        return rho * t, np.abs(rho) * (et * 1.01 + U * mag)

    G = np.zeros_like(u) if du is None else du
    eG = np.zeros_like(u)
    if P["pre"] != "none":
        z = (u - stats[:, 2:3]) * stats[:, 3:4]
        g = one("w2", 1.0) * dh
        back, eb = through(g, np.abs(g) * U, z, stats[:, 3:4], P["pre"])
        G, eG = G + back, eb + (np.abs(G) + np.abs(back)) * U
        eG = eG + np.abs(G) * U
        column("w2", dh * z, 3 * U * np.abs(dh * z))
        column("b2", dh, np.zeros_like(dh))
    out["dr"] = (s * G, abs(s) * eG * 1.01 + np.abs(s * G) * U + TINY)
    if f is None:
        return out
    if threshold(P["p"]):
        keep, k = mask(rows, cols, P["p"], P["seed"], P["offset"])
        G, eG = np.where(keep, G * float(k), 0), np.where(keep, eG * float(k), 0)
        eG = eG * 1.01 + np.abs(G) * U
    z = f
    if P["post"] != "none":
        z = (f - stats[:, 0:1]) * stats[:, 1:2]
    w, b, gate = one("w1", 1.0), one("b1", 0.0), one("gate", 1.0)
    ez = 2 * U * np.abs(z)
    e_az = np.abs(z) * eG + np.abs(G) * ez + np.abs(G * z) * U
    column("w1", G * z, e_az, gate)
    column("b1", G, eG, gate)
    column("_a", G * z, e_az)
    column("_b", G, eG)
    (a, ea), (c, ec) = out.pop("_a"), out.pop("_b")
    gg = w * a + b * c
    out["gate"] = (gg, np.abs(w) * ea + np.abs(b) * ec + 2 * U * (np.abs(w * a) + np.abs(b * c)))
    g = gate * G
    eg = np.abs(gate) * eG + np.abs(g) * U
    if P["post"] == "none":
        out["df"] = (g, eg * 1.01 + TINY)
    else:
        g, eg = w * g, np.abs(w) * eg + np.abs(w * g) * U
        df, e = through(g, eg, z, stats[:, 1:2], P["post"])
        out["df"] = (df, e + np.abs(df) * U + TINY)
    return out
