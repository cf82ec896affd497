"""Cases and plain forms of the operators that make a rank's gradients.

The sharded step reads gradients.  The operators measured here produce them:

* ``checkpoint``  an activation tensor written to its 8-bit checkpoint and read back;
* ``activation``  the activation function forward, saving its input in 8 bits, and its
  backward pass from that checkpoint;
* ``weight_grad`` the weight gradient of a linear layer whose input is kept in 8 bits;
* ``lookup``      embedding rows of the working weights, scaled;
* ``embed_grad``  the gradient of that lookup, by sorted tokens;
* ``policy``      the clipped policy loss with a KL term, and its scaled gradient.

With ``own`` false, ``run`` computes each in elementary torch operations in FP32.
With ``own`` true it makes the calls a user makes of the package.

The 8-bit checkpoint: every 32 neighbours of a row share a power of two 2^k, the
smallest with max|x| <= 448 * 2^k over the finite elements (k >= -124); each element
is x / 2^k rounded to nearest even in e4m3.  Magnitudes above 15/16 of the power of two that
ends the input format's range are held at it, so that every value read back is finite
in the input's format; an infinity or NaN is kept as NaN.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
KMIN = -124
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# largest magnitude a checkpoint stands for: 15/16 of the power of two above the format's range
TOP = {"f16": 15.0 * 2.0 ** 12, "bf16": 15.0 * 2.0 ** 124, "f32": 15.0 * 2.0 ** 124}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
GELU_C = math.sqrt(2.0 / math.pi)
GELU_A = 0.044715


# ---- cases -----------------------------------------------------------------------

def listed():
    return [
        # one padded sequence's hidden states of a small model, kept in FP32, odd width
        {"name": "checkpoint_f32_127x1601", "kind": "checkpoint", "dt": "f32",
         "rows": 127, "cols": 1601},
        # one layer's hidden states for a long micro-batch
        {"name": "checkpoint_bf16_16384x8192", "kind": "checkpoint", "dt": "bf16",
         "rows": 16384, "cols": 8192},
        # an MLP's hidden layer whose width no power of two divides, short batch
        {"name": "activation_silu_f16_509x2050", "kind": "activation", "dt": "f16",
         "act": "silu", "rows": 509, "cols": 2050},
        # the MLP hidden layer of a large model over a long micro-batch
        {"name": "activation_gelu_bf16_16384x10240", "kind": "activation", "dt": "bf16",
         "act": "gelu", "rows": 16384, "cols": 10240},
        # the attention input projection of the GPT-2-small template, one ragged sequence,
        # into the FP32 accumulator
        {"name": "weight_grad_f16_1023x2304x768", "kind": "weight_grad", "dt": "f16",
         "out": "f32", "tokens": 1023, "n_out": 2304, "n_in": 768, "accumulate": False},
        # an MLP projection of a large model over a long micro-batch
        {"name": "weight_grad_bf16_16384x8192x4096", "kind": "weight_grad", "dt": "bf16",
         "out": "bf16", "tokens": 16384, "n_out": 8192, "n_in": 4096, "accumulate": False},
        # the tokens of one step of generation
        {"name": "lookup_f16_64x768", "kind": "lookup", "dt": "f16", "tokens": 64,
         "vocab": 50257, "width": 768, "scale": 1.0},
        # a long micro-batch with the sqrt(width) scaling
        {"name": "lookup_bf16_65536x4096", "kind": "lookup", "dt": "bf16", "tokens": 65536,
         "vocab": 50257, "width": 4096, "scale": 64.0},
        # one sequence of the GPT-2-small template, 16-bit gradients
        {"name": "embed_grad_f16_1024x768", "kind": "embed_grad", "dt": "f16", "out": "f16",
         "tokens": 1024, "vocab": 50257, "width": 768, "scale": 1.0, "accumulate": False},
        # a long micro-batch, padded sequences, into the FP32 accumulator
        {"name": "embed_grad_bf16_65536x4096", "kind": "embed_grad", "dt": "bf16", "out": "f32",
         "tokens": 65536, "vocab": 50257, "width": 4096, "scale": 64.0, "accumulate": False},
        # one short answer, a vocabulary of odd size
        {"name": "policy_f16_61x50257", "kind": "policy", "dt": "f16", "rows": 61,
         "vocab": 50257, "kl": 0.05},
        # a batch of answers over a large vocabulary
        {"name": "policy_bf16_8192x131072", "kind": "policy", "dt": "bf16", "rows": 8192,
         "vocab": 131072, "kl": 0.02},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["checkpoint", "activation", "weight_grad", "lookup", "embed_grad",
                       "policy"])
    if kind in ("checkpoint", "activation"):
        dt = rng.choice(["f16", "bf16", "f32"])
        cols = _log_int(rng, 33, 16384)
        rows = _log_int(rng, 8, min(16384, (1 << 26) // cols))
        if rng.random() < 0.5:
            cols = (cols + 31) // 32 * 32
        case = {"kind": kind, "dt": dt, "rows": rows, "cols": cols}
        if kind == "activation":
            case["act"] = rng.choice(["gelu", "silu"])
        return case
    if kind == "weight_grad":
        dt = rng.choice(["f16", "bf16"])
        n_out, n_in = _log_int(rng, 64, 8192), _log_int(rng, 64, 4096)
        return {"kind": kind, "dt": dt, "out": rng.choice([dt, "f32"]),
                "tokens": _log_int(rng, 33, 16384), "n_out": n_out, "n_in": n_in,
                "accumulate": False}
    if kind == "lookup":
        return {"kind": kind, "dt": rng.choice(["f16", "bf16", "f32"]),
                "tokens": _log_int(rng, 1, 32768), "vocab": _log_int(rng, 500, 60000),
                "width": _log_int(rng, 64, 4096), "scale": rng.choice([1.0, 0.5, 27.7])}
    if kind == "embed_grad":
        dt = rng.choice(["f16", "bf16"])
        out = rng.choice([dt, "f32"])
        return {"kind": kind, "dt": dt, "out": out, "tokens": _log_int(rng, 16, 65536),
                "vocab": _log_int(rng, 500, 50257), "width": _log_int(rng, 64, 2048),
                "scale": rng.choice([1.0, 27.7]),
                "accumulate": out == "f32" and rng.random() < 0.5}
    vocab = _log_int(rng, 500, 200000)
    return {"kind": "policy", "dt": rng.choice(["f16", "bf16", "f32"]),
            "rows": _log_int(rng, 1, max(2, min(8192, (1 << 28) // vocab))), "vocab": vocab,
            "kl": rng.choice([0.0, 0.05])}


# ---- inputs ------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _hidden(rows, cols, dtype, g):
    """Hidden states: unit-scale values with a few columns far larger than the rest."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    gain = torch.ones(cols, device="cuda")
    far = torch.randint(0, cols, (max(1, cols // 200),), generator=g, device="cuda")
    gain[far] = 20.0
    return (x * gain).to(dtype)


def _zipf(vocab):
    p = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return p / p.sum()


def _ids(tokens, vocab, g, padding=0.0):
    """Token ids by frequency rank; a share of positions hold the padding id 0."""
    cdf = torch.from_numpy(np.cumsum(_zipf(vocab))).to("cuda")
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.searchsorted(cdf, u).clamp_(max=vocab - 1)
    if padding:
        ids[torch.rand(tokens, generator=g, device="cuda") < padding] = 0
    return ids


def prepare(case, seed):
    g, kind, st = _gen(seed), case["kind"], {"case": case}
    dtype = DTYPES[case["dt"]]
    if kind in ("checkpoint", "activation"):
        st["x"] = _hidden(case["rows"], case["cols"], dtype, g)
        if kind == "activation":
            st["dy"] = _normal((case["rows"], case["cols"]), dtype, g, 1e-2)
    elif kind == "weight_grad":
        st["dy"] = _normal((case["tokens"], case["n_out"]), dtype, g, 1e-2)
        st["q"], st["e"] = _encode(_hidden(case["tokens"], case["n_in"], dtype, g), case["dt"])
    elif kind in ("lookup", "embed_grad"):
        st["ids"] = _ids(case["tokens"], case["vocab"], g,
                         0.25 if kind == "embed_grad" else 0.0)
        if kind == "lookup":
            st["table"] = _normal((case["vocab"], case["width"]), dtype, g, 0.02)
        else:
            st["dy"] = _normal((case["tokens"], case["width"]), dtype, g, 1e-2)
            if case["accumulate"]:
                st["base"] = _normal((case["vocab"], case["width"]), torch.float32, g, 1e-2)
    else:
        rows, vocab = case["rows"], case["vocab"]
        z = torch.empty((rows, vocab), dtype=dtype, device="cuda")
        for r in range(0, rows, 512):
            z[r:r + 512] = torch.randn((min(512, rows - r), vocab), generator=g, device="cuda",
                                       dtype=torch.float32).mul_(2.0).to(dtype)
        st["targets"] = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        t = torch.arange(rows, device="cuda")
        z[t, st["targets"]] += 8.0      # sampled answers are likely ones
        logp = torch.empty(rows, device="cuda")
        for r in range(0, rows, 512):
            zf = z[r:r + 512].float()
            logp[r:r + 512] = zf.gather(1, st["targets"][r:r + 512, None])[:, 0] - \
                torch.logsumexp(zf, 1)
        st["logits"] = z
        st["old"] = logp + torch.randn(rows, generator=g, device="cuda") * 0.15
        st["ref"] = logp + torch.randn(rows, generator=g, device="cuda") * 0.25
        st["adv"] = torch.randn(rows, generator=g, device="cuda")
        w = (torch.rand(rows, generator=g, device="cuda") >= 0.2).float()   # prompt positions: 0
        w[0] = 1.0
        st["weight"] = w / w.sum()
        st["scale"] = 65536.0 if case["dt"] == "f16" else 1.0
    return st


# ---- plain forms, FP32 ---------------------------------------------------------------

def _blocks(x):
    """[rows, ceil(cols / 32), 32] with zeros past the last column."""
    rows, cols = x.shape
    nb = (cols + BLOCK - 1) // BLOCK
    if nb * BLOCK != cols:
        pad = x.new_zeros((rows, nb * BLOCK))
        pad[:, :cols] = x
        x = pad
    return x.view(rows, nb, BLOCK)


def _pow2(k):
    """2^k in FP32 for whole -126 <= k <= 127, by its exponent bits."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x, dt):
    """(codes, exponents) of the 8-bit checkpoint of x, each uint8."""
    rows, cols = x.shape
    b = _blocks(x.float())
    good = torch.isfinite(b)
    amax = torch.where(good, b.abs(), torch.zeros_like(b)).amax(-1)
    mant, exp = torch.frexp(amax)
    k = exp - 9 + (mant > 0.875).to(exp.dtype)     # amax = (2 mant) * 2^(exp - 1)
    k = torch.where(amax > 0, k, torch.full_like(k, KMIN)).clamp_(min=KMIN)
    v = b.clamp(-TOP[dt], TOP[dt]) * _pow2(-k)[..., None]
    v = torch.where(good, v, torch.full_like(v, float("nan")))
    q = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(rows, -1)[:, :cols].contiguous(), (k + 127).to(torch.uint8)


def _decode(q, e):
    """The values a checkpoint stands for, FP32."""
    rows, cols = q.shape
    v = _blocks(q.view(torch.float8_e4m3fn).float())
    return (v * _pow2(e.to(torch.int32) - 127)[..., None]).view(rows, -1)[:, :cols]


def _act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return 0.5 * x * (1.0 + torch.tanh(GELU_C * (x + GELU_A * x * x * x)))


def _act_slope(x, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return s + x * s * (1.0 - s)
    t = torch.tanh(GELU_C * (x + GELU_A * x * x * x))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_A * x * x)


def _plain_policy(st):
    case = st["case"]
    z = st["logits"].float()
    rows, w = case["rows"], st["weight"]
    m = z.amax(1, keepdim=True)
    ex = torch.exp(z - m)
    total = ex.sum(1, keepdim=True)
    logp = (z.gather(1, st["targets"][:, None]) - m - torch.log(total))[:, 0]
    r = torch.exp(logp - st["old"])
    lo, hi = 1.0 - 0.2, 1.0 + 0.28
    adv = st["adv"]
    cut = ((adv > 0) & (r > hi)) | ((adv < 0) & (r < lo))
    token = -torch.minimum(r * adv, r.clamp(lo, hi) * adv)
    d = st["ref"] - logp
    token = token + case["kl"] * (torch.exp(d) - d - 1.0)
    slope = torch.where(cut, torch.zeros_like(r), -adv * r) + case["kl"] * (1.0 - torch.exp(d))
    zero = torch.zeros_like(w)
    live = w != 0
    token, logp = torch.where(live, token, zero), torch.where(live, logp, zero)
    c = torch.where(live, slope * w * st["scale"], zero)
    dz = ex.mul_(-(c[:, None] / total))
    dz[torch.arange(rows, device=z.device), st["targets"]] += c
    return {"loss": (token.double() * w.double()).sum().float(), "token_loss": token,
            "logp": logp, "dlogits": dz.to(st["logits"].dtype)}


def _plain(st):
    case, kind = st["case"], st["case"]["kind"]
    dtype = DTYPES[case["dt"]]
    if kind == "checkpoint":
        return _decode(*_encode(st["x"], case["dt"])).to(dtype)
    if kind == "activation":
        y = _act(st["x"].float(), case["act"]).to(dtype)
        slope = _act_slope(_decode(*_encode(st["x"], case["dt"])), case["act"])
        return {"y": y, "dx": (st["dy"].float() * slope).to(dtype)}
    if kind == "weight_grad":
        return (st["dy"].float().t() @ _decode(st["q"], st["e"])).to(DTYPES[case["out"]])
    if kind == "lookup":
        return (st["table"][st["ids"]].float() * case["scale"]).to(dtype)
    if kind == "embed_grad":
        s = torch.zeros((case["vocab"], case["width"]), device="cuda")
        s.index_add_(0, st["ids"], st["dy"].float())
        s *= case["scale"]
        return st["base"] + s if case["accumulate"] else s.to(DTYPES[case["out"]])
    return _plain_policy(st)


# ---- the package's calls ---------------------------------------------------------------

def _empty_u8(n, like):
    return torch.empty(n, dtype=torch.uint8, device=like.device)


def _own(st):
    import zero_sharded_mixed_shard_amd as zs

    case, kind = st["case"], st["case"]["kind"]
    dtype = DTYPES[case["dt"]]
    if kind in ("checkpoint", "activation"):
        x = st["x"]
        rows, cols = x.shape
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        e = torch.empty((rows, (cols + BLOCK - 1) // BLOCK), dtype=torch.uint8, device=x.device)
        out = torch.empty_like(x)
        if kind == "checkpoint":
            zs.zero_act_save(q, e, x)
            zs.zero_act_load(out, q, e)
            return out
        act = zs.ACT_SILU if case["act"] == "silu" else zs.ACT_GELU
        y = torch.empty_like(x)
        zs.zero_act_save(q, e, x, act=act, y=y)
        zs.zero_act_backward(out, st["dy"], q, e, act)
        return {"y": y, "dx": out}
    if kind == "weight_grad":
        dy = st["dy"]
        dw = torch.empty((case["n_out"], case["n_in"]), dtype=DTYPES[case["out"]],
                         device=dy.device)
        ws = _empty_u8(zs.zero_weight_grad_workspace(case["tokens"], case["n_out"],
                                                     case["n_in"]), dy)
        zs.zero_weight_grad(dw, dy, st["q"], st["e"], first=True, workspace=ws)
        return dw
    if kind == "lookup":
        out = torch.empty((case["tokens"], case["width"]), dtype=dtype,
                          device=st["ids"].device)
        zs.zero_embed_lookup(out, st["table"], st["ids"], scale=case["scale"])
        return out
    if kind == "embed_grad":
        dy = st["dy"]
        ws = _empty_u8(zs.zero_embed_grad_workspace(case["tokens"], case["vocab"],
                                                    case["width"]), dy)
        if case["accumulate"]:
            dw = st["base"].clone()
        else:
            dw = torch.empty((case["vocab"], case["width"]), dtype=DTYPES[case["out"]],
                             device=dy.device)
        zs.zero_embed_grad(dw, dy, st["ids"], scale=case["scale"],
                           first=not case["accumulate"], workspace=ws)
        return dw
    z = st["logits"]
    loss = torch.empty(1, device=z.device)
    token, logp = (torch.empty(case["rows"], device=z.device) for _ in range(2))
    dz = torch.empty_like(z)
    zs.zero_policy_loss(loss, token, logp, z, st["targets"], st["adv"], st["weight"],
                        old_logp=st["old"], ref_logp=st["ref"], clip_low=0.2, clip_high=0.28,
                        kl_coef=case["kl"], loss_scale=st["scale"], dlogits=dz)
    return {"loss": loss[0], "token_loss": token, "logp": logp, "dlogits": dz}


def run(state):
    return _own(state) if own else _plain(state)


# ---- 64-bit definitions ------------------------------------------------------------------

def _exact_pow2(k):
    """2^k in FP64 for whole -1022 <= k <= 1023 (a library pow may be an ulp off)."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_checkpoint(x, dt):
    """Checkpoint values in FP64: a grid of spacing 2^(max(floor(log2 |x|), k - 6) - 3)."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    b = torch.zeros((rows, nb * BLOCK), dtype=torch.float64, device=x.device)
    b[:, :cols] = x.double()
    b = b.view(rows, nb, BLOCK)
    fin = b.isfinite()
    mag = torch.where(fin, b, torch.zeros_like(b)).abs()
    top = mag.amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(top.clamp_min(2.0 ** -200) / 448.0))
    # log2 is not exact at the borders: settle k by the comparison itself
    k = torch.where(top > 448.0 * _exact_pow2(k), k + 1, k)
    k = torch.where(top <= 448.0 * _exact_pow2(k - 1), k - 1, k).clamp_min(KMIN)
    low = torch.frexp(mag)[1].double() - 1.0
    grid = _exact_pow2(torch.maximum(low, k - 6.0) - 3.0)
    v = torch.round(torch.clamp_max(mag, TOP[dt]) / grid) * grid       # halves to even
    v = torch.where(fin, torch.copysign(v, b), torch.full_like(b, float("nan")))
    return v.view(rows, -1)[:, :cols]


def _exact_act(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    return x * torch.sigmoid(2.0 * GELU_C * (x + GELU_A * x ** 3))


def _exact_slope(x, act):
    u, du = (x, torch.ones_like(x)) if act == "silu" else \
        (2.0 * GELU_C * (x + GELU_A * x ** 3), 2.0 * GELU_C * (1.0 + 3.0 * GELU_A * x ** 2))
    s = torch.sigmoid(u)
    return s + x * s * torch.sigmoid(-u) * du


def _exact_policy(st):
    case = st["case"]
    rows = case["rows"]
    token, logp = (torch.zeros(rows, dtype=torch.float64, device="cuda") for _ in range(2))
    dz = torch.zeros(st["logits"].shape, dtype=torch.float64, device="cuda")
    for r0 in range(0, rows, 256):
        s = slice(r0, min(rows, r0 + 256))
        z = st["logits"][s].double()
        a, w, adv = st["targets"][s], st["weight"][s].double(), st["adv"][s].double()
        lp_all = torch.log_softmax(z, 1)
        lp = lp_all.gather(1, a[:, None])[:, 0]
        r = torch.exp(lp - st["old"][s].double())
        lo, hi = 1.0 - float(np.float32(0.2)), 1.0 + float(np.float32(0.28))
        kl = float(np.float32(case["kl"]))
        d = st["ref"][s].double() - lp
        first, second = r * adv, r.clamp(lo, hi) * adv
        t = torch.maximum(-first, -second) + kl * (torch.expm1(d) - d)
        c = torch.where(first <= second, -adv * r, torch.zeros_like(r)) - kl * torch.expm1(d)
        live = w != 0
        token[s] = torch.where(live, t, torch.zeros_like(t))
        logp[s] = torch.where(live, lp, torch.zeros_like(lp))
        c = torch.where(live, c * w * st["scale"], torch.zeros_like(c))
        part = torch.exp(lp_all) * -c[:, None]
        part.scatter_add_(1, a[:, None], c[:, None])
        dz[s] = part
    return {"loss": (token * st["weight"].double()).sum(), "token_loss": token, "logp": logp,
            "dlogits": dz}


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "checkpoint":
        return _exact_checkpoint(st["x"], case["dt"])
    if kind == "activation":
        return {"y": _exact_act(st["x"].double(), case["act"]),
                "dx": st["dy"].double() * _exact_slope(_exact_checkpoint(st["x"], case["dt"]),
                                                       case["act"])}
    if kind == "weight_grad":
        q = st["q"].int()
        k = st["e"].double().repeat_interleave(BLOCK, 1)[:, :case["n_in"]] - 127.0
        frac, ex = (q & 7).double(), ((q >> 3) & 15).double()
        mag = torch.where(ex > 0, (8.0 + frac) * _exact_pow2(ex - 10.0), frac * 2.0 ** -9)
        x = torch.where(q > 127, -mag, mag) * _exact_pow2(k)
        return st["dy"].double().t().contiguous() @ x
    if kind == "lookup":
        return st["table"].double()[st["ids"]] * float(np.float32(case["scale"]))
    if kind == "embed_grad":
        out = torch.zeros((case["vocab"], case["width"]), dtype=torch.float64, device="cuda")
        out.index_add_(0, st["ids"], st["dy"].double())
        out *= float(np.float32(case["scale"]))
        return out + st["base"].double() if case["accumulate"] else out
    return _exact_policy(st)


# ---- work ----------------------------------------------------------------------------------

def work(case):
    kind, b = case["kind"], BYTES[case["dt"]]
    if kind in ("checkpoint", "activation"):
        n = case["rows"] * case["cols"]
        held = n + case["rows"] * -(-case["cols"] // BLOCK)
        if kind == "checkpoint":        # read x, write and read the checkpoint, write x
            return {"bytes": 2 * b * n + 2 * held, "flops": 4 * n}
        return {"bytes": 4 * b * n + 2 * held, "flops": 40 * n}
    if kind == "weight_grad":
        t, o, i = case["tokens"], case["n_out"], case["n_in"]
        return {"bytes": b * t * o + t * i + t * -(-i // BLOCK) + BYTES[case["out"]] * o * i,
                "flops": 2 * t * o * i}
    if kind == "lookup":
        t, d = case["tokens"], case["width"]
        rows = float((1.0 - (1.0 - _zipf(case["vocab"])) ** t).sum())   # distinct ids expected
        return {"bytes": int((rows + t) * d * b) + 8 * t, "flops": t * d}
    if kind == "embed_grad":
        t, v, d, ob = case["tokens"], case["vocab"], case["width"], BYTES[case["out"]]
        return {"bytes": t * d * b + 8 * t + v * d * ob * (2 if case["accumulate"] else 1),
                "flops": t * d}
    n = case["rows"] * case["vocab"]
    return {"bytes": 2 * b * n + 36 * case["rows"], "flops": 10 * n}
