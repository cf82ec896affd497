"""The clipped policy loss and its gradient on the GPU against the 64-bit definition."""
import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs
from gpu_util import log
from test_gpu_o_act import Framed

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
LO, HI = 0.2, 0.28


def inputs(rows, vocab, dt, seed, masked=True):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(rows, vocab, generator=g) * 3).to(plain.TORCH[dt])
    a = torch.randint(0, vocab, (rows,), generator=g)
    logp = torch.log_softmax(z.double(), 1).gather(1, a[:, None])[:, 0].float()
    old = logp + torch.randn(rows, generator=g) * 0.25
    ref = logp + torch.randn(rows, generator=g) * 0.5
    adv = torch.randn(rows, generator=g)
    w = torch.rand(rows, generator=g) / rows
    if masked and rows > 2:
        w[torch.rand(rows, generator=g) < 0.3] = 0
    return z, a, old, ref, adv, w


def run(z, a, old, ref, adv, w, kl, S, grads=True, in_place=False, gap=0, lead=0, ctl=None):
    rows, vocab = z.shape
    zf = Framed(rows, vocab, z.dtype, vocab + gap, lead)
    zf.t.copy_(z)
    df = None
    if grads:
        df = zf if in_place else Framed(rows, vocab, z.dtype, vocab + 2 * gap, lead + 1)
    loss = torch.full((1,), 9.0, device=DEV)
    token, logp = Framed(1, rows, torch.float32), Framed(1, rows, torch.float32)
    kw = dict(old_logp=None if old is None else old.to(DEV),
              ref_logp=None if ref is None else ref.to(DEV), clip_low=LO, clip_high=HI,
              kl_coef=kl, dlogits=None if df is None else df.t)
    args = (loss, token.t[0], logp.t[0], zf.t, a.to(DEV), adv.to(DEV), w.to(DEV))
    if ctl is None:
        zs.zero_policy_loss(*args, loss_scale=S, **kw)
    else:
        zs.zero_policy_loss_dev(*args, ctl=ctl, **kw)
    torch.cuda.synchronize()
    for f in (zf, df, token, logp):
        assert f is None or f.intact()
    if not in_place:
        assert torch.equal(zf.t.cpu().nan_to_num(), z.nan_to_num())
    return loss, token.t[0], logp.t[0], None if df is None else df.t


def check(got, z, a, old, ref, adv, w, kl, S, dt, what=""):
    loss, token, logp, dl = got
    n = lambda t: None if t is None else t.double().numpy()
    ex = plain.policy(plain.f64(z), a.numpy(), n(old), n(ref), n(adv), n(w), LO, HI, kl, S)
    for k, t, b in (("token_loss", token, "b_token"), ("logp", logp, "b_logp")):
        err = np.abs(plain.f64(t) - ex[k])
        tol = ex[b] + np.abs(ex[k]) * plain.U
        assert np.all(err <= tol), (what, k, (err - tol).max())
    assert abs(float(loss) - ex["loss"]) <= ex["b_loss"] + 2 * abs(ex["loss"]) * plain.U
    if dl is None:
        return
    far = ~ex["near"]                       # the cut is decided beyond the ratio's error
    assert far.sum() >= 0.8 * len(far)
    err = np.abs(plain.f64(dl) - ex["dlogits"])[far]
    tol = plain.rounded(ex["dlogits"], ex["b_dlogits"], dt)[far]
    assert np.all(err <= tol), (what, (err / tol).max())
    log(f"  policy {dt} {z.shape}: worst {float((err / tol).max()):.2f} of the bound")


# vocabularies around every block size's edge, one to many rows
SHAPES = [(1, 1), (3, 2), (5, 7), (4, 8), (6, 9), (9, 511), (7, 1024), (3, 1025), (5, 2047),
          (4, 4096), (3, 8193), (2, 16385), (3, 32771), (2, 50257), (2, 65537), (2, 131072),
          (2, 131073), (1, 200_003), (40, 300), (130, 65), (3, 49_153), (2, 98_305), (1, 262_144),
          (2, 262_161), (1, 300_007), (2, 102_400), (2, 102_409), (3, 51_200), (3, 51_205)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_loss_and_gradient(rows, vocab, dt):
    x = inputs(rows, vocab, dt, rows + vocab)
    S = 1024.0 if dt == "f16" else 3.0
    gap, lead = (0, 0) if vocab % 2 else (8, 0)
    got = run(*x, 0.07, S, gap=gap, lead=lead)
    check(got, *x, 0.07, S, dt)
    loss, token, logp, none = run(*x, 0.07, S, grads=False, gap=gap)
    check((loss, token, logp, none), *x, 0.07, S, dt)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,gap,lead", [(5, 100, 0, 1), (4, 3001, 3, 2), (3, 50257, 0, 5),
                                                 (2, 200_003, 1, 3), (2, 24_576, 0, 7),
                                                 (2, 270_001, 5, 1)])
def test_in_place_equals_apart(rows, vocab, gap, lead, dt):
    x = inputs(rows, vocab, dt, 5)
    apart = run(*x, 0.05, 64.0, gap=gap, lead=lead)
    here = run(*x, 0.05, 64.0, in_place=True, gap=gap, lead=lead)
    for p, q in zip(apart, here):
        assert torch.equal(p, q)
    check(here, *x, 0.05, 64.0, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [60, 5000, 40_000, 250_000, 280_000])
def test_on_policy_and_without_kl(vocab, dt):
    z, a, old, ref, adv, w = inputs(4, vocab, dt, 6)
    x = (z, a, None, None, adv, w)
    check(run(*x, 0.0, 2.0), *x, 0.0, 2.0, dt)
    x = (z, a, old, None, adv, w)
    check(run(*x, 0.0, 2.0), *x, 0.0, 2.0, dt)
    x = (z, a, None, ref, adv, w)
    check(run(*x, 0.3, 2.0), *x, 0.3, 2.0, dt)


@pytest.mark.parametrize("vocab", [40, 3000, 30_000, 250_000, 280_000])
def test_skipped_rows_are_not_read(vocab):
    z, a, old, ref, adv, w = inputs(6, vocab, "bf16", 7, masked=False)
    w[1] = w[4] = 0.0
    clean = run(z, a, old, ref, adv, w, 0.1, 8.0)
    for t in (z[1], old[1:2], ref[1:2], adv[1:2], z[4]):
        t.fill_(float("nan"))
    adv[4] = float("inf")
    a[1], a[4] = -100, 2 ** 40
    got = run(z, a, old, ref, adv, w, 0.1, 8.0)
    for p, q in zip(clean, got):
        assert torch.equal(p, q)
    loss, token, logp, dl = got
    assert bool((dl[[1, 4]] == 0).all()) and float(token[1]) == float(logp[4]) == 0.0
    none = run(z, a, old, ref, adv, torch.zeros(6), 0.1, 8.0)
    assert float(none[0]) == 0.0 and bool((none[3] == 0).all())


@pytest.mark.parametrize("vocab", [40, 3000, 30_000, 250_000, 280_000])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_excluded_tokens_and_bad_rows(vocab, dt):
    z, a, old, ref, adv, w = inputs(8, vocab, dt, 8, masked=False)
    ninf, inf, nan = -float("inf"), float("inf"), float("nan")
    z[0, ::2] = ninf                      # half the vocabulary excluded
    a[0] = 1
    lp = torch.log_softmax(z[0].double(), 0)[1].item()
    old[0], ref[0] = lp + 0.01, lp - 0.2
    z[1, :] = ninf                        # nothing left
    z[2, 5] = inf
    z[3, 7] = nan
    a[4] = -1
    a[5] = vocab
    z[6, a[6]] = ninf                     # the target itself excluded
    got = run(z, a, old, ref, adv, w, 0.1, 2.0)
    loss, token, logp, dl = (t.cpu() for t in got)
    assert bool((dl[0, ::2] == 0).all())
    for r in (1, 2, 3, 4, 5):
        assert torch.isnan(logp[r]) and torch.isnan(token[r]) and bool(torch.isnan(dl[r]).any()), r
    assert logp[6].item() == ninf and not torch.isfinite(token[6])
    assert not torch.isfinite(dl[6]).all() and torch.isnan(loss[0])
    keep = [0, 7]
    sub = tuple(t[keep] for t in (z, a, old, ref, adv, w))
    check((torch.tensor(float(sum(token[k].double() * w[k].double() for k in keep))),
           token[keep], logp[keep], dl[keep]), *sub, 0.1, 2.0, dt)


def test_the_clip_and_its_borders():
    # one logit pair, ratios set by old_logp: the gradient vanishes exactly beyond the cut
    z = torch.zeros(7, 2)
    lp = float(np.log(0.5))
    ratios = [0.5, 0.9, 1.0, 1.25, 1.5, 3.0, 1e-3]
    old = torch.tensor([lp - np.log(r) for r in ratios], dtype=torch.float32)
    a = torch.zeros(7, dtype=torch.int64)
    for sign in (1.0, -1.0, 0.0):
        adv = torch.full((7,), sign)
        _, token, _, dl = run(z, a, old, None, adv, torch.ones(7), 0.0, 1.0)
        for t, r in enumerate(ratios):
            cut = (sign > 0 and r > 1 + HI) or (sign < 0 and r < 1 - LO)
            want = 0.0 if cut else -sign * r * 0.5
            assert abs(float(dl[t, 0]) - want) <= 1e-5 * max(1, r), (sign, r)
            assert float(dl[t, 0]) == -float(dl[t, 1])
            if cut:
                assert float(dl[t, 0]) == 0.0


def test_gradient_against_differences():
    # FP64 differences of the 64-bit loss, second order: h^2 times the loss's third derivative
    z, a, old, ref, adv, w = inputs(5, 30, "f32", 11, masked=False)
    old = torch.log_softmax(z.double(), 1).gather(1, a[:, None])[:, 0].float() + \
        torch.tensor([0.05, -0.05, 0.1, -0.1, 0.0])
    got = run(z, a, old, ref, adv, w, 0.2, 4.0)
    n = lambda t: t.double().numpy()
    f = lambda zz: plain.policy(zz, a.numpy(), n(old), n(ref), n(adv), n(w), LO, HI, 0.2, 4.0)
    ex, h = f(n(z)), 1e-4
    for t, v in ((0, 3), (1, int(a[1])), (4, 29), (2, int(a[2]))):
        up, dn = n(z).copy(), n(z).copy()
        up[t, v] += h
        dn[t, v] -= h
        diff = 4.0 * (f(up)["loss"] - f(dn)["loss"]) / (2 * h)
        tol = ex["b_dlogits"][t, v] + 100 * h * h + 1e-9
        assert abs(diff - float(got[3][t, v])) <= tol + abs(diff) * plain.U


def test_device_scale_and_int32_targets():
    z, a, old, ref, adv, w = inputs(9, 700, "bf16", 12)
    ctl = zs.device_ctl_new(512.0, DEV)
    host = run(z, a, old, ref, adv, w, 0.1, 512.0)
    dev = run(z, a.int(), old, ref, adv, w, 0.1, None, ctl=ctl)
    for p, q in zip(host, dev):
        assert torch.equal(p, q)


def test_no_rows_and_a_lowered_cap():
    loss = torch.full((1,), 5.0, device=DEV)
    e = torch.empty(0, device=DEV)
    zs.zero_policy_loss(loss, e, e, torch.empty(0, 10, device=DEV),
                        torch.empty(0, dtype=torch.int64, device=DEV), e, e, clip_low=0.2,
                        clip_high=0.2, kl_coef=0.0, loss_scale=1.0)
    assert float(loss) == 0.0
    x = inputs(50, 90, "f32", 13)
    free = run(*x, 0.1, 2.0)
    zs.zero_set_grid_cap(3)
    try:
        capped = run(*x, 0.1, 2.0)
    finally:
        zs.zero_set_grid_cap(0)
    for p, q in zip(free, capped):
        assert torch.equal(p, q)


def test_logits_past_4_gib():
    rows, vocab = 20_000, 131_072                     # 5.2 GB of BF16
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device=DEV)
    h, a, old, ref, adv, w = inputs(3, vocab, "bf16", 14, masked=False)
    z[-3:] = h.to(DEV)
    pad = lambda t: torch.cat([torch.zeros(rows - 3, dtype=t.dtype), t]).to(DEV)
    loss, token, logp = torch.empty(1, device=DEV), torch.empty(rows, device=DEV), \
        torch.empty(rows, device=DEV)
    dz = torch.full_like(z, 1.0)
    zs.zero_policy_loss(loss, token, logp, z, pad(a), pad(adv), pad(w), old_logp=pad(old),
                        ref_logp=pad(ref), clip_low=LO, clip_high=HI, kl_coef=0.1,
                        loss_scale=2.0, dlogits=dz)
    check((loss, token[-3:], logp[-3:], dz[-3:]), h, a, old, ref, adv, w, 0.1, 2.0, "bf16")
    assert not bool(dz[:-3].any())


@pytest.mark.parametrize("vocab", [50, 20_000, 270_000])
def test_unusual_arguments(vocab):
    # no upper cut, a full lower one, a negative KL weight, negative weights, int32 targets
    z, a, old, ref, adv, w = inputs(6, vocab, "f32", 15, masked=False)
    w[2] = -w[2]
    f = lambda lo, hi, kl, t: (lambda o: (zs.zero_policy_loss(
        o[0], o[1], o[2], z.to(DEV), t.to(DEV), adv.to(DEV), w.to(DEV), old_logp=old.to(DEV),
        ref_logp=ref.to(DEV), clip_low=lo, clip_high=hi, kl_coef=kl, loss_scale=2.0,
        dlogits=o[3]), o)[1])([torch.empty(1, device=DEV), torch.empty(6, device=DEV),
                               torch.empty(6, device=DEV), torch.empty(6, vocab, device=DEV)])
    n = lambda t: t.double().numpy()
    for lo, hi, kl in ((1.0, float("inf"), 0.1), (0.0, 0.0, -0.2)):
        got = f(lo, hi, kl, a)
        ex = plain.policy(n(z), a.numpy(), n(old), n(ref), n(adv), n(w), lo, hi, kl, 2.0)
        far = ~ex["near"]
        err = np.abs(plain.f64(got[3]) - ex["dlogits"])
        # the bounds count kl by its magnitude
        bound = plain.policy(n(z), a.numpy(), n(old), n(ref), n(adv), n(w), lo, hi, abs(kl), 2.0)
        tol = plain.rounded(np.maximum(np.abs(ex["dlogits"]), np.abs(bound["dlogits"])),
                            bound["b_dlogits"], "f32") + np.abs(bound["dlogits"]) * 8 * plain.U
        assert np.all(err[far] <= tol[far])
        for p, q in zip(got, f(lo, hi, kl, a.int())):
            assert torch.equal(p, q)


@pytest.mark.parametrize("vocab", [40, 3000, 30_000, 250_000, 280_000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_logits(vocab, dt):
    # rows far from zero up to the end of the range: the terms go by z - m
    td = plain.TORCH[dt]
    for v in (2.0 ** 19, 2.0 ** 21, 1e12, 1e38, 3e38):
        z = torch.zeros(3, vocab, dtype=td)
        z[0, 3], z[1, 5] = v, -v
        z[2] = v
        z[2, 7] = -v
        a, one = torch.tensor([3, 3, 4]), torch.ones(3)
        for in_place in (False, True):
            loss, token, logp, dl = run(z, a, None, None, one, one, 0.0, 1.0, in_place=in_place)
            assert float(logp[0]) == 0.0 and bool((dl[0] == 0).all())
            for r in (1, 2):        # one token of the row excluded, the others alike
                p = 1.0 / (vocab - 1)
                assert abs(float(logp[r]) + np.log(vocab - 1)) <= 40 * plain.U * np.log(vocab)
                assert float(dl[r, 5 if r == 1 else 7]) == 0.0
                tol = plain.rounded(np.float64(p), p * (208 + vocab / 1024) * plain.U, dt)
                assert abs(float(dl[r, 0]) - p) <= tol, (v, r)


def test_rows_past_the_sum_kernels_stride():
    # more rows than the loss's sum takes at once: whole numbers, an exact total
    rows = 30_011
    z = torch.zeros(rows, 2, device=DEV)
    t = torch.zeros(rows, dtype=torch.int64, device=DEV)
    w = torch.ones(rows, device=DEV)
    w[::7] = 0
    adv = (torch.arange(rows, device=DEV) % 5).float()
    loss, token, logp = torch.empty(1, device=DEV), torch.empty(rows, device=DEV), \
        torch.empty(rows, device=DEV)
    zs.zero_policy_loss(loss, token, logp, z, t, adv, w, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                        loss_scale=1.0)
    assert torch.equal(token, torch.where(w != 0, -adv, torch.zeros_like(adv)))
    assert float(loss) == -float((adv * w).double().sum())
