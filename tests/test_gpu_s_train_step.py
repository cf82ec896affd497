"""The gradient operators together, as a rank's training step uses them: lookup, 8-bit
checkpoints, policy loss, activation backward, weight and embedding gradients into one
flat buffer, then overflow check, decision and step.

Every operator's result is compared with the 64-bit definition on the inputs it really
had; the sequence is captured into a graph and replayed; micro-batches accumulate.
"""
import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
V, D, H = 331, 40, 75            # vocabulary, width, hidden width: nothing divides 32
PSI = V * D + H * D + V * H      # table, W1[H, D], W2[V, H]


def parts(flat):
    """The three parameters' places in a flat buffer of PSI elements."""
    a, b = V * D, V * D + H * D
    return flat[:a].view(V, D), flat[a:b].view(H, D), flat[b:].view(V, H)


class Rank:
    def __init__(self, dtype, seed, S=64.0, tokens=170):
        g = torch.Generator().manual_seed(seed)
        self.T, self.dtype = tokens, dtype
        # the flat buffers start one element in: no parameter is aligned to anything
        big = lambda dt: torch.zeros(PSI + 1, dtype=dt, device=DEV)[1:]
        self.master, self.m, self.v = big(torch.float32), big(torch.float32), big(torch.float32)
        self.master.copy_(torch.randn(PSI, generator=g) * 0.3)
        self.w16, self.g16 = big(dtype), big(dtype)
        self.w16.copy_(self.master)
        self.acc = big(torch.float32)
        self.ctl = zs.device_ctl_new(S, DEV)
        self.bias = zs.zero_bias_corrections(HP["beta1"], HP["beta2"], 1, 64).to(DEV)
        self.S = S
        u8 = lambda r, c: torch.empty(r, c, dtype=torch.uint8, device=DEV)
        ck = lambda c: (u8(tokens, c), u8(tokens, -(-c // 32)))
        t = lambda c: torch.empty(tokens, c, dtype=dtype, device=DEV)
        self.cx, self.ca, self.ch = ck(D), ck(H), ck(H)
        self.x, self.a, self.h, self.z = t(D), t(H), t(H), t(V)
        self.dh, self.dx = t(H), t(D)
        f = lambda n: torch.empty(n, device=DEV)
        self.loss, self.token, self.logp = f(1), f(tokens), f(tokens)
        ws = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)
        self.ws1 = ws(zs.zero_weight_grad_workspace(tokens, H, D))
        self.ws2 = ws(zs.zero_weight_grad_workspace(tokens, V, H))
        self.ws3 = ws(zs.zero_embed_grad_workspace(tokens, V, D))

    def batch(self, seed):
        g = torch.Generator().manual_seed(seed)
        ids = torch.randint(0, V, (self.T,), generator=g)
        ids[torch.rand(self.T, generator=g) < 0.2] = 7
        targets = torch.randint(0, V, (self.T,), generator=g)
        w = (torch.rand(self.T, generator=g) >= 0.3).float()
        w[0] = 1.0
        self.ids, self.targets = ids.to(DEV), targets.to(DEV)
        self.weight = (w / w.sum()).to(DEV)
        self.adv = torch.randn(self.T, generator=g).to(DEV)
        self.old = (torch.randn(self.T, generator=g) * 0.1 - 5.8).to(DEV)
        self.ref = self.old + 0.05

    def forward(self):
        table, w1, w2 = parts(self.w16)
        zs.zero_embed_lookup(self.x, table, self.ids, scale=1.5)
        zs.zero_act_save(*self.cx, self.x)
        self.a.copy_(self.x.float() @ w1.float().t())
        zs.zero_act_save(*self.ca, self.a, act=zs.ACT_GELU, y=self.h)
        zs.zero_act_save(*self.ch, self.h)
        self.z.copy_(self.h.float() @ w2.float().t())

    def loss_and_backward(self, grads, first):
        """Gradients into the flat buffer `grads`; the logits become their gradient."""
        gt, g1, g2 = parts(grads)
        _, w1, w2 = parts(self.w16)
        zs.zero_policy_loss_dev(self.loss, self.token, self.logp, self.z, self.targets, self.adv,
                                self.weight, old_logp=self.old, ref_logp=self.ref, clip_low=0.2,
                                clip_high=0.3, kl_coef=0.1, ctl=self.ctl, dlogits=self.z)
        zs.zero_weight_grad(g2, self.z, *self.ch, first=first, workspace=self.ws2)
        self.dh.copy_(self.z.float() @ w2.float())
        zs.zero_act_backward(self.dh, self.dh, *self.ca, zs.ACT_GELU)
        zs.zero_weight_grad(g1, self.dh, *self.cx, first=first, workspace=self.ws1)
        self.dx.copy_(self.dh.float() @ w1.float())
        zs.zero_embed_grad(gt, self.dx, self.ids, scale=1.5, first=first, workspace=self.ws3)

    def step16(self):
        zs.zero_overflow_check_dev(self.g16, PSI, 1, 0, self.ctl)
        zs.zero_scaler_update_dev(self.ctl, self.bias, 1)
        zs.zero_adam_step_dev(self.w16, self.g16, self.master, self.m, self.v, PSI, 1, 0,
                              ctl=self.ctl, **HP)

    def state(self):
        return [t.clone() for t in (self.w16, self.master, self.m, self.v, self.loss, self.ctl)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_every_operator_of_a_step(dt):
    r = Rank(plain.TORCH[dt], 3)
    r.batch(4)
    w0 = r.w16.clone()
    table, w1, w2 = (plain.f64(p) for p in parts(w0))
    ids, tg = r.ids.cpu().numpy(), r.targets.cpu().numpy()
    r.forward()
    x = plain.f64(r.x)
    want = torch.from_numpy(plain.lookup(table, ids, 1.5)).to(r.dtype)
    assert torch.equal(r.x.cpu(), want)
    for (q, e), t in ((r.cx, r.x), (r.ca, r.a), (r.ch, r.h)):
        wq, we = plain.encode(plain.f64(t), dt)
        assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(e.cpu().numpy(), we)
    val, bound = plain.act(plain.f64(r.a), "gelu")
    assert np.all(np.abs(plain.f64(r.h) - val) <= plain.rounded(val, bound, dt))
    logits = r.z.clone()
    r.loss_and_backward(r.g16, True)
    n = lambda t: t.double().cpu().numpy()
    ex = plain.policy(plain.f64(logits), tg, n(r.old), n(r.ref), n(r.adv), n(r.weight), 0.2, 0.3,
                      0.1, r.S)
    far = ~ex["near"]
    err = np.abs(plain.f64(r.z) - ex["dlogits"])[far]
    assert np.all(err <= plain.rounded(ex["dlogits"], ex["b_dlogits"], dt)[far])
    assert abs(float(r.loss) - ex["loss"]) <= ex["b_loss"] + abs(ex["loss"]) * 2 * plain.U
    dec = lambda c: plain.decode(c[0].cpu().numpy(), c[1].cpu().numpy())
    gt, g1, g2 = (plain.f64(p) for p in parts(r.g16))
    want, bound = plain.weight_grad(plain.f64(r.z), dec(r.ch))
    assert np.all(np.abs(g2 - want) <= plain.rounded(want, bound, dt))
    want, bound = plain.weight_grad(plain.f64(r.dh), dec(r.cx))
    assert np.all(np.abs(g1 - want) <= plain.rounded(want, bound, dt))
    want, bound = plain.embed_grad(plain.f64(r.dx), ids, V, 1.5)
    assert np.all(np.abs(gt - want) <= plain.rounded(want, bound, dt))
    r.step16()
    c = zs.device_ctl_read(r.ctl)
    assert (c.found_inf, c.apply, c.scaler.step) == (0, 1, 1)
    assert not torch.equal(r.w16, w0)


def test_checkpointed_gradient_against_the_unquantised_one():
    # W2's gradient against dz^T h with the hidden layer as it was, not as its checkpoint
    # holds it, and the logits' gradient in FP64.  Each value is off by at most 2^-4 of
    # itself or 2^(k - 10) (the checkpoint), each dz by its own bound and one BF16
    # rounding, the sums by FP32, the result by one rounding
    r = Rank(torch.bfloat16, 5)
    r.batch(6)
    r.forward()
    logits, h = plain.f64(r.z), plain.f64(r.h)
    r.loss_and_backward(r.g16, True)
    n = lambda t: t.double().cpu().numpy()
    ex = plain.policy(logits, r.targets.cpu().numpy(), n(r.old), n(r.ref), n(r.adv), n(r.weight),
                      0.2, 0.3, 0.1, r.S)
    assert not ex["near"].any()
    dz = ex["dlogits"]
    e_dz = plain.rounded(dz, ex["b_dlogits"], "bf16")
    k = np.repeat(r.ch[1].cpu().numpy().astype(int), 32, axis=1)[:, :H] - 127
    e_h = np.maximum(np.abs(h) * 2.0 ** -4, np.ldexp(1.0, k - 10))
    want = dz.T @ h
    bound = np.abs(dz).T @ e_h + e_dz.T @ (np.abs(h) + e_h)
    bound += ((np.abs(dz) + e_dz).T @ (np.abs(h) + e_h)) * r.T * 2 * plain.U
    err = np.abs(plain.f64(parts(r.g16)[2]) - want)
    assert np.all(err <= plain.rounded(want, bound, "bf16"))


def test_micro_batches_accumulate_in_fp32():
    r = Rank(torch.bfloat16, 7)
    each = []
    for k in range(3):
        r.batch(20 + k)
        r.forward()
        logits = r.z.clone()
        r.loss_and_backward(r.acc, k == 0)
        total = r.acc.clone()
        r.z.copy_(logits)
        one = torch.empty(PSI + 1, device=DEV)[1:]
        r.loss_and_backward(one, True)
        each.append(one)
        want = each[0].clone()
        for e in each[1:]:
            want += e
        assert torch.equal(total, want)
        r.acc.copy_(total)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    zs.zero_overflow_check_g32(r.acc, PSI, 1, 0, r.S, flag)
    assert int(flag) == 0


def test_an_overflow_in_the_forward_pass_skips_the_step():
    r = Rank(torch.float16, 8)
    r.batch(9)
    r.forward()
    r.x[3, 5] = float("inf")
    zs.zero_act_save(*r.cx, r.x)
    before = r.state()
    r.loss_and_backward(r.g16, True)
    r.step16()
    c = zs.device_ctl_read(r.ctl)
    assert (c.found_inf, c.apply, c.scaler.loss_scale) == (1, 0, r.S / 2)
    for a, b in zip(before[:4], r.state()[:4]):
        assert torch.equal(a, b)


def test_step_captured_in_a_graph_and_replayed():
    # the operators and the step in one graph; the plain products between them are left
    # out (their results stand in place, refreshed between replays by eager work)
    def operators(r):
        table, w1, w2 = parts(r.w16)
        gt, g1, g2 = parts(r.g16)
        zs.zero_embed_lookup(r.x, table, r.ids, scale=1.5)
        zs.zero_act_save(*r.cx, r.x)
        zs.zero_act_save(*r.ca, r.a, act=zs.ACT_SILU, y=r.h)
        zs.zero_act_save(*r.ch, r.h)
        zs.zero_policy_loss_dev(r.loss, r.token, r.logp, r.z, r.targets, r.adv, r.weight,
                                old_logp=r.old, ref_logp=r.ref, clip_low=0.2, clip_high=0.3,
                                kl_coef=0.1, ctl=r.ctl, dlogits=r.z)
        zs.zero_weight_grad(g2, r.z, *r.ch, workspace=r.ws2)
        zs.zero_act_backward(r.dh, r.dh, *r.ca, zs.ACT_SILU)
        zs.zero_weight_grad(g1, r.dh, *r.cx, workspace=r.ws1)
        zs.zero_embed_grad(gt, r.dx, r.ids, scale=1.5, workspace=r.ws3)
        r.step16()

    tokens = 9000                          # split products and the radix sort
    E, G = Rank(torch.bfloat16, 10, tokens=tokens), Rank(torch.bfloat16, 10, tokens=tokens)
    assert E.ws1.numel() > 0
    names = ("a", "z", "dh", "dx", "ids", "targets", "weight", "adv", "old", "ref")
    for r in (E, G):
        r.batch(11)

    def refresh(k):
        g = torch.Generator().manual_seed(100 + k)
        E.batch(50 + k)
        for n in ("a", "z", "dh", "dx"):
            t = getattr(E, n)
            t.copy_(torch.randn(t.shape, generator=g))
        for n in names:                    # same inputs, in place
            getattr(G, n).copy_(getattr(E, n))

    refresh(0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        operators(G)
    for k in range(4):
        refresh(k)
        torch.cuda.synchronize()
        graph.replay()
        operators(E)
        torch.cuda.synchronize()
        for a, b in zip(E.state() + [E.g16, E.z, E.dh, E.token], G.state() +
                        [G.g16, G.z, G.dh, G.token]):
            assert torch.equal(a, b), k
    assert zs.device_ctl_read(G.ctl).scaler.step == 4
    del graph


def test_work_goes_to_the_given_stream():
    # a long fill on a side stream, then the operators on that stream, once as its current
    # stream and once by argument: they must see the filled values
    for by_argument in (False, True):
        side = torch.cuda.Stream()
        x = torch.zeros(4096, 8192, dtype=torch.bfloat16, device=DEV)
        q = torch.zeros(4096, 8192, dtype=torch.uint8, device=DEV)
        e = torch.zeros(4096, 256, dtype=torch.uint8, device=DEV)
        back = torch.zeros_like(x)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for v in range(1, 30):
                x.fill_(float(v))
            if not by_argument:
                zs.zero_act_save(q, e, x)
                zs.zero_act_load(back, q, e)
        if by_argument:
            zs.zero_act_save(q, e, x, stream=side)
            zs.zero_act_load(back, q, e, stream=side)
        side.synchronize()
        v = plain.decode(*plain.encode(np.full((1, 1), 29.0), "bf16"))[0, 0]
        assert bool((back == v).all())


def test_two_streams_with_workspaces_of_their_own():
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, 500, (20_000,), generator=g).to(DEV)
    dy = torch.randint(-4, 5, (20_000, 256), generator=g).bfloat16().to(DEV)
    want = torch.zeros(500, 256, dtype=torch.float64)
    want.index_add_(0, ids.cpu(), dy.double().cpu())
    n = zs.zero_embed_grad_workspace(20_000, 500, 256)
    outs = [torch.empty(500, 256, device=DEV) for _ in range(2)]
    spaces = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w in zip(streams, outs, spaces):
            zs.zero_embed_grad(o, dy, ids, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.cpu().double(), want)
