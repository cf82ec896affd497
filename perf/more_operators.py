"""Cases and plain forms of the operators around a block's linear layers.

* ``quant``     a matrix into 8-bit codes with one power of two for each block of 128:
  128 neighbours of a row, or 128 x 128 (weights, which also get transposed codes for
  the product of the backward pass), and read back;
* ``product``   y = a b^T of two such matrices; a may be an activation checkpoint
  (blocks of 32) too;
* ``dropout``   dropout by a counter-based generator, forward and backward: the mask is
  computed again and never stored;
* ``residual``  the step between two blocks: u = s r + gate * drop(post-norm(f)) and
  h = pre-norm(u);
* ``residual_grad``  its backward pass, with the gradients of the norms' weights and
  biases and of the gate.

With ``own`` false, ``run`` computes each in elementary torch operations in FP32.
With ``own`` true it makes the calls a user makes of the package.

The generator is Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel
random numbers: as easy as 1, 2, 3", 2011).  Element (row, col) has 16 of the 128 bits
of counter (col / 8, row, offset mod 2^32, offset / 2^32) under the seed as key: word
(col mod 8) / 2, its low half for even columns.  An element stays where its bits are at
least t = rint(65536 p), and is multiplied by 65536 / (65536 - t).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
KMIN = -124
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# largest magnitude a code stands for: 15/16 of the power of two above the format's range
TOP = {"f16": 15.0 * 2.0 ** 12, "bf16": 15.0 * 2.0 ** 124, "f32": 15.0 * 2.0 ** 124}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5


# ---- cases -----------------------------------------------------------------------

def listed():
    return [
        # hidden states of one padded sequence of a small model, odd width
        {"name": "quant_f16_127x1601", "kind": "quant", "dt": "f16", "rows": 127, "cols": 1601,
         "square": False},
        # an MLP's weights, coded for both passes after each optimizer step
        {"name": "quant_bf16_8192x8192_square", "kind": "quant", "dt": "bf16", "rows": 8192,
         "cols": 8192, "square": True},
        # one token of generation through the GPT-2-small template's attention projection
        {"name": "product_f16_1x2304x768", "kind": "product", "dt": "f16", "m": 1, "n": 2304,
         "k": 768, "a_block": 128},
        # short answers' logits in FP32 over a vocabulary of odd size
        {"name": "product_f32_61x50257x768", "kind": "product", "dt": "f32", "m": 61, "n": 50257,
         "k": 768, "a_block": 128},
        # one ragged sequence of that template, from the layer's activation checkpoint
        {"name": "product_f16_1023x2304x768_checkpoint", "kind": "product", "dt": "f16",
         "m": 1023, "n": 2304, "k": 768, "a_block": 32},
        # an MLP projection of a large model over a long micro-batch
        {"name": "product_bf16_16384x8192x4096", "kind": "product", "dt": "bf16", "m": 16384,
         "n": 8192, "k": 4096, "a_block": 128},
        # a short ragged batch of odd width
        {"name": "dropout_f16_61x769", "kind": "dropout", "dt": "f16", "rows": 61, "cols": 769,
         "p": 0.1},
        # a long micro-batch's hidden states of a large model
        {"name": "dropout_bf16_16384x8192", "kind": "dropout", "dt": "bf16", "rows": 16384,
         "cols": 8192, "p": 0.1},
        # the GPT-2-small template: dropout after the projection, residual, layer norm
        {"name": "residual_f16_64x768_layer", "kind": "residual", "dt": "f16", "res": "f16",
         "rows": 64, "cols": 768, "post": "none", "pre": "layer", "bias": True, "gate": False,
         "p": 0.1, "scale": 1.0},
        # a large model with norms on both sides of the block, a learned gate, and the
        # residual stream in FP32
        {"name": "residual_bf16_16384x8192_rms", "kind": "residual", "dt": "bf16", "res": "f32",
         "rows": 16384, "cols": 8192, "post": "rms", "pre": "rms", "bias": False, "gate": True,
         "p": 0.0, "scale": 0.5},
        # one ragged sequence of the template backward
        {"name": "residual_grad_f16_1023x768_layer", "kind": "residual_grad", "dt": "f16",
         "res": "f16", "out": "f16", "rows": 1023, "cols": 768, "post": "none", "pre": "layer",
         "bias": True, "gate": False, "p": 0.1, "scale": 1.0},
        # the large model backward, parameter gradients into the FP32 accumulator
        {"name": "residual_grad_bf16_16384x8192_rms", "kind": "residual_grad", "dt": "bf16",
         "res": "bf16", "out": "f32", "rows": 16384, "cols": 8192, "post": "rms", "pre": "rms",
         "bias": False, "gate": True, "p": 0.0, "scale": 0.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width; every second one a multiple of 64, as models have them."""
    n = _log_int(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    kind = rng.choice(["quant", "product", "dropout", "residual", "residual_grad"])
    if kind == "quant":
        cols = _width(rng, 33, 8192)
        return {"kind": kind, "dt": rng.choice(["f16", "bf16", "f32"]),
                "rows": _log_int(rng, 1, 8192), "cols": cols, "square": rng.random() < 0.5}
    if kind == "product":
        n, k = _width(rng, 64, 50257), _width(rng, 64, 8192)
        most = min(16384, (1 << 27) // n, (1 << 39) // (n * k))
        return {"kind": kind, "dt": rng.choice(["f16", "bf16", "f32"]),
                "m": _log_int(rng, 1, max(2, most)), "n": n, "k": k,
                "a_block": rng.choice([32, 128])}
    cols = _width(rng, 64, 16384)
    rows = _log_int(rng, 1, min(16384, (1 << 26) // cols))
    if kind == "dropout":
        return {"kind": kind, "dt": rng.choice(["f16", "bf16", "f32"]), "rows": rows,
                "cols": cols, "p": rng.choice([0.05, 0.1, 0.5])}
    dt = rng.choice(["f16", "bf16", "f32"])
    case = {"kind": kind, "dt": dt, "res": rng.choice([dt, "f32"]), "rows": rows, "cols": cols,
            "post": rng.choice(["none", "rms", "layer"]), "pre": rng.choice(["rms", "layer"]),
            "bias": rng.random() < 0.5, "gate": rng.random() < 0.5,
            "p": rng.choice([0.0, 0.1]), "scale": rng.choice([1.0, 0.7])}
    if kind == "residual_grad":
        case["out"] = rng.choice([dt, "f32"])
    return case


# ---- inputs ------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, g, std=1.0, mean=0.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(std).add_(mean).to(dtype)


def _hidden(rows, cols, dtype, g):
    """Hidden states: unit-scale values with a few columns far larger than the rest."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    gain = torch.ones(cols, device="cuda")
    gain[torch.randint(0, cols, (max(1, cols // 200),), generator=g, device="cuda")] = 20.0
    return x.mul_(gain).to(dtype)


def _stats_of(x, norm):
    """(mean, reciprocal deviation) of each row, FP64."""
    x = x.double()
    mean = x.mean(1) if norm == "layer" else torch.zeros_like(x[:, 0])
    return mean, 1.0 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + EPS)


def prepare(case, seed):
    g, kind, st = _gen(seed), case["kind"], {"case": case}
    dtype = DTYPES[case["dt"]]
    if kind == "quant":
        st["x"] = _normal((case["rows"], case["cols"]), dtype, g, 0.02) if case["square"] else \
            _hidden(case["rows"], case["cols"], dtype, g)
        return st
    if kind == "product":
        m, n, k = case["m"], case["n"], case["k"]
        src = "bf16" if case["dt"] == "f32" else case["dt"]
        st["qa"], st["ea"] = _encode(_hidden(m, k, DTYPES[src], g), src, case["a_block"], False)
        st["qb"], st["eb"] = _encode(_normal((n, k), DTYPES[src], g, 0.02), src, BLOCK, True)
        return st
    rows, cols = case["rows"], case["cols"]
    st["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=g, device="cuda"))
    st["offset"] = int(torch.randint(0, 1 << 40, (1,), generator=g, device="cuda"))
    if kind == "dropout":
        st["x"] = _hidden(rows, cols, dtype, g)
        st["dy"] = _normal((rows, cols), dtype, g, 1e-2)
        return st
    st["f"] = _hidden(rows, cols, dtype, g)
    for name, there, mean in (("w1", case["post"] != "none", 1.0),
                              ("b1", case["post"] != "none" and case["bias"], 0.0),
                              ("gate", case["gate"], 0.5), ("w2", True, 1.0),
                              ("b2", case["bias"], 0.0)):
        st[name] = _normal((cols,), dtype, g, 0.1, mean) if there else None
    r = _hidden(rows, cols, DTYPES[case["res"]], g)
    if kind == "residual":
        st["r"] = r
        return st
    # what the forward pass left: the stream after the step, and the rows' statistics
    st["u"] = r
    stats = torch.zeros((rows, 4), dtype=torch.float64, device="cuda")
    for r0 in range(0, rows, 2048):
        s = slice(r0, r0 + 2048)
        if case["post"] != "none":
            stats[s, 0], stats[s, 1] = _stats_of(st["f"][s], case["post"])
        stats[s, 2], stats[s, 3] = _stats_of(st["u"][s], case["pre"])
    st["stats"] = stats.float()
    st["dh"] = _normal((rows, cols), dtype, g, 1e-2)
    st["du"] = _normal((rows, cols), DTYPES[case["res"]], g, 1e-2)
    return st


# ---- plain forms, FP32 ---------------------------------------------------------------

def _pow2(k):
    """2^k in FP32 for whole -126 <= k <= 127, by its exponent bits."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _spread(e, rows, cols, block, square):
    """A block's value at each of its elements, [rows, cols]."""
    e = e.repeat_interleave(block, 1)[:, :cols]
    return e.repeat_interleave(block, 0)[:rows] if square else e


def _encode(x, dt, block, square):
    """(codes, exponents) of x in blocks, each uint8."""
    rows, cols = x.shape
    x = x.float()
    good = torch.isfinite(x)
    tall = block if square else 1
    nr, nc = -(-rows // tall), -(-cols // block)
    mag = x.new_zeros((nr * tall, nc * block))
    mag[:rows, :cols] = torch.where(good, x.abs(), torch.zeros_like(x))
    amax = mag.view(nr, tall, nc, block).amax((1, 3))
    mant, exp = torch.frexp(amax)
    k = exp - 9 + (mant > 0.875).to(exp.dtype)     # amax = (2 mant) * 2^(exp - 1)
    k = torch.where(amax > 0, k, torch.full_like(k, KMIN)).clamp_(min=KMIN)
    v = x.clamp(-TOP[dt], TOP[dt]) * _spread(_pow2(-k), rows, cols, block, square)
    v = torch.where(good, v, torch.full_like(v, float("nan")))
    return v.to(torch.float8_e4m3fn).view(torch.uint8), (k + 127).to(torch.uint8)


def _decode(q, e, block, square):
    """The values codes stand for, FP32."""
    rows, cols = q.shape
    k = _spread(e.to(torch.int32) - 127, rows, cols, block, square)
    return q.view(torch.float8_e4m3fn).float() * _pow2(k)


def _mul32(a, b):
    """(high, low) words of the 64-bit product of words a (int64 tensor) and b (a number)."""
    lo, hi = a * (b & 0xffff), a * (b >> 16)          # below 2^48 each
    mid = hi + (lo >> 16)
    return mid >> 16, ((mid & 0xffff) << 16) | (lo & 0xffff)


def _keep(rows, cols, p, seed, offset):
    """The mask [rows, cols] and the factor of what stays."""
    groups = -(-cols // 8)
    c0 = torch.arange(groups, device="cuda").expand(rows, groups)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, groups)
    c2 = torch.full((rows, groups), offset & 0xffffffff, device="cuda")
    c3 = torch.full((rows, groups), offset >> 32, device="cuda")
    k0, k1 = seed & 0xffffffff, seed >> 32
    for _ in range(10):
        h0, l0 = _mul32(c0, 0xD2511F53)
        h1, l1 = _mul32(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    words = torch.stack((c0, c1, c2, c3), -1)
    bits = torch.stack((words & 0xffff, words >> 16), -1).view(rows, groups * 8)[:, :cols]
    t = round(float(np.float32(p)) * 65536.0)
    return bits >= t, (65536.0 / (65536 - t) if t < 65536 else 0.0)


def _drop(x, p, seed, offset):
    if p == 0.0:
        return x
    keep, factor = _keep(x.shape[0], x.shape[1], p, seed, offset)
    return torch.where(keep, x * factor, torch.zeros_like(x))


def _norm(x, kind):
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    return x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)


def _affine(x, w, b):
    x = x if w is None else x * w.float()
    return x if b is None else x + b.float()


def _norm_back(g, xhat, rho, kind):
    """Gradient through a norm: g that of the normalised row xhat, rho 1 / deviation."""
    g = g - xhat * (g * xhat).mean(1, keepdim=True) - \
        (g.mean(1, keepdim=True) if kind == "layer" else 0.0)
    return g * rho


def _plain_residual(st):
    case = st["case"]
    n = st["f"].float()
    if case["post"] != "none":
        n = _affine(_norm(n, case["post"]), st["w1"], st["b1"])
    v = _drop(_affine(n, st["gate"], None), case["p"], st["seed"], st["offset"])
    u = st["r"].float() * case["scale"] + v
    h = _affine(_norm(u, case["pre"]), st["w2"], st["b2"])
    return {"u": u.to(DTYPES[case["res"]]), "h": h.to(DTYPES[case["dt"]])}


def _plain_residual_grad(st):
    case, s = st["case"], st["stats"]
    out, dh = {}, st["dh"].float()
    uhat = (st["u"].float() - s[:, 2:3]) * s[:, 3:4]
    out["w2"] = (dh * uhat).sum(0)
    out["b2"] = dh.sum(0) if st["b2"] is not None else None
    du = st["du"].float() + _norm_back(_affine(dh, st["w2"], None), uhat, s[:, 3:4], case["pre"])
    out["dr"] = (du * case["scale"]).to(DTYPES[case["res"]])
    dv = _drop(du, case["p"], st["seed"], st["offset"])
    fhat = st["f"].float()
    if case["post"] != "none":
        fhat = (fhat - s[:, 0:1]) * s[:, 1:2]
    out["gate"] = (dv * _affine(fhat, st["w1"], st["b1"])).sum(0) if case["gate"] else None
    dn = _affine(dv, st["gate"], None)
    out["w1"] = (dn * fhat).sum(0) if st["w1"] is not None else None
    out["b1"] = dn.sum(0) if st["b1"] is not None else None
    df = dn if case["post"] == "none" else \
        _norm_back(_affine(dn, st["w1"], None), fhat, s[:, 1:2], case["post"])
    out["df"] = df.to(DTYPES[case["dt"]])
    for name in ("w1", "b1", "gate", "w2", "b2"):
        out[name] = None if out[name] is None else out[name].to(DTYPES[case["out"]])
    return {name: x for name, x in out.items() if x is not None}


def _plain(st):
    case, kind = st["case"], st["case"]["kind"]
    dtype = DTYPES[case["dt"]]
    if kind == "quant":
        q, e = _encode(st["x"], case["dt"], BLOCK, case["square"])
        out = {"values": _decode(q, e, BLOCK, case["square"]).to(dtype)}
        if case["square"]:
            out["transposed"] = _decode(q.t().contiguous(), e.t().contiguous(), BLOCK,
                                        True).to(dtype)
        return out
    if kind == "product":
        a = _decode(st["qa"], st["ea"], case["a_block"], False)
        return (a @ _decode(st["qb"], st["eb"], BLOCK, True).t()).to(dtype)
    if kind == "dropout":
        keep, factor = _keep(case["rows"], case["cols"], case["p"], st["seed"], st["offset"])
        zero = torch.zeros((), device="cuda")
        return {"y": torch.where(keep, st["x"].float() * factor, zero).to(dtype),
                "dx": torch.where(keep, st["dy"].float() * factor, zero).to(dtype)}
    return _plain_residual(st) if kind == "residual" else _plain_residual_grad(st)


# ---- the package's calls ---------------------------------------------------------------

def _u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def _block_of(zs, st):
    """What both passes of the step between blocks are told alike."""
    case = st["case"]
    kinds = {"none": zs.NORM_NONE, "rms": zs.NORM_RMS, "layer": zs.NORM_LAYER}
    return dict(post=kinds[case["post"]], pre=kinds[case["pre"]], post_weight=st["w1"],
                post_bias=st["b1"], gate=st["gate"], pre_weight=st["w2"], pre_bias=st["b2"],
                eps=EPS, res_scale=case["scale"], p=case["p"], seed=st["seed"],
                offset=st["offset"])


def _own(st):
    import zero_sharded_mixed_shard_amd as zs

    case, kind = st["case"], st["case"]["kind"]
    dtype = DTYPES[case["dt"]]
    if kind == "quant":
        x, square = st["x"], case["square"]
        rows, cols = x.shape
        nr, nc = (-(-rows // BLOCK) if square else rows), -(-cols // BLOCK)
        q, e, values = _u8(rows, cols), _u8(nr, nc), torch.empty_like(x)
        if not square:
            zs.zero_block_quant(q, e, x)
            zs.zero_block_load(values, q, e)
            return {"values": values}
        qt, et = _u8(cols, rows), _u8(nc, nr)
        transposed = torch.empty((cols, rows), dtype=dtype, device="cuda")
        zs.zero_block_quant(q, e, x, square=True, qt=qt, et=et)
        zs.zero_block_load(values, q, e, square=True)
        zs.zero_block_load(transposed, qt, et, square=True)
        return {"values": values, "transposed": transposed}
    if kind == "product":
        m, n, k = case["m"], case["n"], case["k"]
        y = torch.empty((m, n), dtype=dtype, device="cuda")
        ws = _u8(zs.zero_block_product_workspace(m, n, k))
        zs.zero_block_product(y, st["qa"], st["ea"], st["qb"], st["eb"], workspace=ws)
        return y
    if kind == "dropout":
        y, dx = torch.empty_like(st["x"]), torch.empty_like(st["dy"])
        zs.zero_dropout(y, st["x"], case["p"], st["seed"], st["offset"])
        zs.zero_dropout(dx, st["dy"], case["p"], st["seed"], st["offset"])
        return {"y": y, "dx": dx}
    rows, cols = case["rows"], case["cols"]
    if kind == "residual":
        u, h = torch.empty_like(st["r"]), torch.empty_like(st["f"])
        stats = torch.empty((rows, 4), device="cuda")
        zs.zero_residual_norm(u, h, stats, st["r"], st["f"], **_block_of(zs, st))
        return {"u": u, "h": h}
    df, dr = torch.empty_like(st["f"]), torch.empty_like(st["u"])
    grads = {name: None if st[name] is None else
             torch.empty(cols, dtype=DTYPES[case["out"]], device="cuda")
             for name in ("w1", "b1", "gate", "w2", "b2")}
    ws = _u8(zs.zero_residual_norm_workspace(rows, cols))
    zs.zero_residual_norm_backward(df, dr, st["dh"], st["du"], st["f"], st["u"], st["stats"],
                                   d_post_weight=grads["w1"], d_post_bias=grads["b1"],
                                   d_gate=grads["gate"], d_pre_weight=grads["w2"],
                                   d_pre_bias=grads["b2"], first=True, workspace=ws,
                                   **_block_of(zs, st))
    out = {**grads, "df": df, "dr": dr}
    return {name: x for name, x in out.items() if x is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---- 64-bit definitions ------------------------------------------------------------------

def _exact_pow2(k):
    """2^k in FP64 for whole -1022 <= k <= 1023 (a library pow may be an ulp off)."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quant(x, dt, square):
    """The values x's codes stand for: in a block of 2^k a grid of spacing
    2^(max(floor(log2 |x|), k - 6) - 3)."""
    rows, cols = x.shape
    out = torch.empty((rows, cols), dtype=torch.float64, device=x.device)
    for r0 in range(0, rows, 1024):
        part = x[r0:r0 + 1024].double()
        for c0 in range(0, cols, BLOCK):
            b = part[:, c0:c0 + BLOCK]
            fin = b.isfinite()
            mag = torch.where(fin, b, torch.zeros_like(b)).abs()
            top = mag.amax(1, keepdim=True)
            if square:
                n = b.shape[0]
                tall = torch.zeros((-(-n // BLOCK) * BLOCK, 1), dtype=b.dtype, device=b.device)
                tall[:n] = top
                top = tall.view(-1, BLOCK).amax(1).repeat_interleave(BLOCK)[:n, None]
            k = torch.ceil(torch.log2(top.clamp_min(2.0 ** -200) / 448.0))
            # log2 is not exact at the borders: settle k by the comparison itself
            k = torch.where(top > 448.0 * _exact_pow2(k), k + 1, k)
            k = torch.where(top <= 448.0 * _exact_pow2(k - 1), k - 1, k).clamp_min(KMIN)
            low = torch.frexp(mag)[1].double() - 1.0
            grid = _exact_pow2(torch.maximum(low, k - 6.0) - 3.0)
            v = torch.round(torch.clamp_max(mag, TOP[dt]) / grid) * grid       # halves to even
            out[r0:r0 + 1024, c0:c0 + BLOCK] = torch.where(
                fin, torch.copysign(v, b), torch.full_like(b, float("nan")))
    return out


def _exact_values(q, e, block, tall):
    """Codes by their fields: sign, four exponent bits, three of the significand."""
    q = q.int()
    frac, ex = (q & 7).double(), ((q >> 3) & 15).double()
    mag = torch.where(ex > 0, (8.0 + frac) * _exact_pow2(ex - 10.0), frac * 2.0 ** -9)
    r = torch.arange(q.shape[0], device=q.device)[:, None] // tall
    c = torch.arange(q.shape[1], device=q.device)[None, :] // block
    return torch.where(q > 127, -mag, mag) * _exact_pow2(e.double()[r, c] - 127.0)


def _exact_keep(rows, cols, p, seed, offset):
    """The mask on the host, in unsigned 64-bit words, a few rows at a time."""
    word, mask = np.uint64, np.uint64(0xffffffff)
    t = int(np.rint(np.float64(np.float32(p)) * 65536.0))
    groups = (cols + 7) // 8
    out = np.empty((rows, cols), dtype=bool)
    step = max(1, (1 << 20) // groups)
    for r0 in range(0, rows, step):
        n = min(step, rows - r0)
        c = [np.tile(np.arange(groups, dtype=word), (n, 1)),
             np.repeat(np.arange(r0, r0 + n, dtype=word)[:, None], groups, 1),
             np.full((n, groups), offset % (1 << 32), dtype=word),
             np.full((n, groups), offset >> 32, dtype=word)]
        key = [seed % (1 << 32), seed >> 32]
        for _ in range(10):
            a, b = c[0] * word(0xD2511F53), c[2] * word(0xCD9E8D57)
            c = [(b >> word(32)) ^ c[1] ^ word(key[0]), b & mask,
                 (a >> word(32)) ^ c[3] ^ word(key[1]), a & mask]
            key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
        bits = np.empty((n, groups, 8), dtype=np.uint32)
        for j in range(4):
            bits[:, :, 2 * j] = c[j] & word(0xffff)
            bits[:, :, 2 * j + 1] = c[j] >> word(16)
        out[r0:r0 + n] = bits.reshape(n, groups * 8)[:, :cols] >= t
    return torch.from_numpy(out).to("cuda").double() * (65536.0 / (65536 - t))


def _exact_residual(st):
    case = st["case"]
    rows, cols = st["f"].shape
    double = lambda x, other: torch.full((cols,), other, dtype=torch.float64, device="cuda") \
        if x is None else x.double()
    w1, b1, gate = double(st["w1"], 1.0), double(st["b1"], 0.0), double(st["gate"], 1.0)
    w2, b2 = double(st["w2"], 1.0), double(st["b2"], 0.0)
    scale = float(np.float32(case["scale"]))
    keep = _exact_keep(rows, cols, case["p"], st["seed"], st["offset"]) if case["p"] else None
    out = {"u": torch.empty((rows, cols), dtype=torch.float64, device="cuda")}
    out["h"] = torch.empty_like(out["u"])
    for r0 in range(0, rows, 2048):
        s = slice(r0, r0 + 2048)
        n = st["f"][s].double()
        if case["post"] != "none":
            mean, rho = _stats_of(n, case["post"])
            n = (n - mean[:, None]) * rho[:, None] * w1 + b1
        v = n * gate if keep is None else n * gate * keep[s]
        u = scale * st["r"][s].double() + v
        mean, rho = _stats_of(u, case["pre"])
        out["u"][s], out["h"][s] = u, (u - mean[:, None]) * rho[:, None] * w2 + b2
    return out


def _exact_residual_grad(st):
    """The norm's Jacobian applied to each row: with z = (x - mean) rho,
    J^T g = rho (g - [mean(g)] - z mean(g z))."""
    case = st["case"]
    rows, cols = st["f"].shape
    double = lambda x: 1.0 if x is None else x.double()
    keep = _exact_keep(rows, cols, case["p"], st["seed"], st["offset"]) if case["p"] else None
    total = {n: torch.zeros(cols, dtype=torch.float64, device="cuda")
             for n in ("w1", "b1", "gate", "w2", "b2") if st[n] is not None}
    full = {n: torch.empty((rows, cols), dtype=torch.float64, device="cuda") for n in ("df", "dr")}

    def through(g, z, rho, kind):
        back = g - z * ((g * z).sum(1) / cols)[:, None]
        if kind == "layer":
            back = back - (g.sum(1) / cols)[:, None]
        return back * rho[:, None]

    for r0 in range(0, rows, 2048):
        s = slice(r0, r0 + 2048)
        dh, f, u = st["dh"][s].double(), st["f"][s].double(), st["u"][s].double()
        mean, rho = _stats_of(u, case["pre"])
        z = (u - mean[:, None]) * rho[:, None]
        total["w2"] += (dh * z).sum(0)
        if "b2" in total:
            total["b2"] += dh.sum(0)
        du = st["du"][s].double() + through(dh * double(st["w2"]), z, rho, case["pre"])
        full["dr"][s] = float(np.float32(case["scale"])) * du
        dv = du if keep is None else du * keep[s]
        z = f
        if case["post"] != "none":
            mean, rho = _stats_of(f, case["post"])
            z = (f - mean[:, None]) * rho[:, None]
        if "gate" in total:
            n = z * double(st["w1"])
            total["gate"] += (dv * (n if st["b1"] is None else n + st["b1"].double())).sum(0)
        dn = dv * double(st["gate"])
        if "w1" in total:
            total["w1"] += (dn * z).sum(0)
        if "b1" in total:
            total["b1"] += dn.sum(0)
        full["df"][s] = dn if case["post"] == "none" else \
            through(dn * double(st["w1"]), z, rho, case["post"])
    return {**total, **full}


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "quant":
        v = _exact_quant(st["x"], case["dt"], case["square"])
        return {"values": v, "transposed": v.t().contiguous()} if case["square"] else \
            {"values": v}
    if kind == "product":
        a = _exact_values(st["qa"], st["ea"], case["a_block"], 1)
        return a @ _exact_values(st["qb"], st["eb"], BLOCK, BLOCK).t().contiguous()
    if kind == "dropout":
        keep = _exact_keep(case["rows"], case["cols"], case["p"], st["seed"], st["offset"])
        return {"y": st["x"].double() * keep, "dx": st["dy"].double() * keep}
    return _exact_residual(st) if kind == "residual" else _exact_residual_grad(st)


# ---- work ----------------------------------------------------------------------------------

def work(case):
    kind, b = case["kind"], BYTES[case["dt"]]
    if kind == "product":
        m, n, k = case["m"], case["n"], case["k"]
        scales = m * -(-k // case["a_block"]) + -(-n // BLOCK) * -(-k // BLOCK)
        return {"bytes": m * k + n * k + scales + m * n * b, "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if kind == "quant":             # read x; write and read the codes, write what they stand for
        forms = 2 if case["square"] else 1
        scales = -(-rows // (BLOCK if case["square"] else 1)) * -(-cols // BLOCK)
        return {"bytes": b * n + forms * (b * n + 2 * n + 2 * scales), "flops": 4 * n}
    if kind == "dropout":
        return {"bytes": 4 * b * n, "flops": 2 * n}
    rb = BYTES[case["res"]]
    params = 2 + (case["post"] != "none") + case["gate"] + 2 * case["bias"]
    if kind == "residual":
        return {"bytes": (2 * b + 2 * rb) * n + params * cols * b, "flops": 12 * n}
    return {"bytes": (3 * b + 3 * rb) * n + 16 * rows + params * cols * (b + BYTES[case["out"]]),
            "flops": 30 * n}
