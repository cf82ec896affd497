"""The operators around a block's linear layers together, as a rank's training step uses them:
lookup, first norm, a block in 8-bit products with its activation, dropout, gate, residual and
norm, logits, policy loss, and all of it backward into one flat buffer, then check, decision
and step.

Every operator's result is compared with the 64-bit definition on the inputs it really had;
the whole step is captured into a graph and replayed; streams; two graphs with workspaces of
their own.
"""
import numpy as np
import pytest
import torch

import block_plain as plain
import grad_plain
import zero_sharded_mixed_shard_amd as zs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HP = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
V, D, H, T = 203, 136, 299, 170      # vocabulary, width, hidden width, tokens
SHAPES = dict(table=(V, D), w0=(D,), W1=(H, D), W2=(D, H), gate=(D,), w2=(D,), b2=(D,),
              out=(V, D))
PSI = sum(int(np.prod(s)) for s in SHAPES.values())
F64 = grad_plain.f64


def parts(flat):
    p, at = {}, 0
    for name, shape in SHAPES.items():
        n = int(np.prod(shape))
        p[name] = flat[at:at + n].view(shape)
        at += n
    return p


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device=DEV)


def blocks(n):
    return -(-n // 128)


class Rank:
    def __init__(self, dtype, seed, S=64.0, p=0.2):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.S, self.p = dtype, S, p
        big = lambda dt: torch.zeros(PSI + 1, dtype=dt, device=DEV)[1:]   # aligned to nothing
        self.master, self.m, self.v = big(torch.float32), big(torch.float32), big(torch.float32)
        start = parts(torch.randn(PSI, generator=g) * 0.2)
        for name in ("w0", "w2", "gate"):
            start[name] += 1.0
        self.master.copy_(torch.cat([t.reshape(-1) for t in start.values()]))
        self.w16, self.g16 = big(dtype), big(dtype)
        self.w16.copy_(self.master)
        self.ctl = zs.device_ctl_new(S, DEV)
        self.bias = zs.zero_bias_corrections(HP["beta1"], HP["beta2"], 1, 64).to(DEV)
        self.step = torch.zeros(1, dtype=torch.int64, device=DEV)
        t = lambda c, dt=dtype: torch.zeros(T, c, dtype=dt, device=DEV)
        ck = lambda c: (u8(T, c), u8(T, -(-c // 32)))
        self.x, self.h0, self.a, self.y = t(D), t(D), t(H), t(H)
        self.f, self.h, self.z = t(D), t(D), t(V)
        self.x32, self.u = t(D, torch.float32), t(D, torch.float32)   # the stream in FP32
        self.st0, self.st1 = (torch.zeros(T, 4, device=DEV) for _ in range(2))
        self.c0, self.ca, self.cy, self.ch = ck(D), ck(H), ck(H), ck(D)
        self.dz, self.dh, self.df, self.dy, self.dh0, self.dx = t(V), t(D), t(D), t(H), t(D), t(D)
        self.du, self.dr = t(D, torch.float32), t(D, torch.float32)
        self.codes = {}
        for name in ("W1", "W2", "out"):
            n, k = SHAPES[name]
            self.codes[name] = (u8(n, k), u8(blocks(n), blocks(k)), u8(k, n),
                                u8(blocks(k), blocks(n)))
        self.qz, self.qf, self.qy = ((u8(T, c), u8(T, blocks(c))) for c in (V, D, H))
        f = lambda n: torch.zeros(n, device=DEV)
        self.loss, self.token, self.logp = f(1), f(T), f(T)
        most = max([zs.zero_block_product_workspace(T, n, k)
                    for n, k in ((H, D), (D, H), (V, D), (D, V))] +
                   [zs.zero_weight_grad_workspace(T, n, k)
                    for n, k in ((H, D), (D, H), (V, D))] +
                   [zs.zero_embed_grad_workspace(T, V, D), zs.zero_residual_norm_workspace(T, D)])
        self.ws = u8(most)

    def batch(self, seed):
        g = torch.Generator().manual_seed(seed)
        ids = torch.randint(0, V, (T,), generator=g)
        ids[torch.rand(T, generator=g) < 0.2] = 7
        w = (torch.rand(T, generator=g) >= 0.3).float()
        w[0] = 1.0
        new = dict(ids=ids, targets=torch.randint(0, V, (T,), generator=g), weight=w / w.sum(),
                   adv=torch.randn(T, generator=g), old=torch.randn(T, generator=g) * 0.1 - 5.5)
        for name, t in new.items():
            if hasattr(self, name):
                getattr(self, name).copy_(t)
            else:
                setattr(self, name, t.to(DEV))

    def told0(self):
        return dict(pre=zs.NORM_RMS, pre_weight=parts(self.w16)["w0"], eps=1e-5)

    def told1(self):
        w = parts(self.w16)
        return dict(post=zs.NORM_NONE, pre=zs.NORM_LAYER, gate=w["gate"], pre_weight=w["w2"],
                    pre_bias=w["b2"], eps=1e-5, res_scale=0.5, p=self.p, seed=99, offset=1000,
                    d_offset=self.step)

    def product(self, y, coded, name, transposed=False):
        w = self.codes[name]
        zs.zero_block_product(y, *coded, *(w[2:] if transposed else w[:2]), workspace=self.ws)

    def forward(self):
        w = parts(self.w16)
        for name in self.codes:
            q, e, qt, et = self.codes[name]
            zs.zero_block_quant(q, e, w[name], square=True, qt=qt, et=et)
        zs.zero_embed_lookup(self.x, w["table"], self.ids)
        self.x32.copy_(self.x)
        zs.zero_residual_norm(None, self.h0, self.st0, self.x32, **self.told0())
        zs.zero_act_save(*self.c0, self.h0)
        self.product(self.a, self.c0, "W1")
        zs.zero_act_save(*self.ca, self.a, act=zs.ACT_SILU, y=self.y)
        zs.zero_act_save(*self.cy, self.y)
        self.product(self.f, self.cy, "W2")
        zs.zero_residual_norm(self.u, self.h, self.st1, self.x32, self.f, **self.told1())
        zs.zero_act_save(*self.ch, self.h)
        self.product(self.z, self.ch, "out")

    def backward(self):
        g = parts(self.g16)
        zs.zero_policy_loss_dev(self.loss, self.token, self.logp, self.z, self.targets, self.adv,
                                self.weight, old_logp=self.old, clip_low=0.2, clip_high=0.3,
                                kl_coef=0.0, ctl=self.ctl, dlogits=self.dz)
        zs.zero_weight_grad(g["out"], self.dz, *self.ch, workspace=self.ws)
        zs.zero_block_quant(*self.qz, self.dz)
        self.product(self.dh, self.qz, "out", True)
        zs.zero_residual_norm_backward(self.df, self.dr, self.dh, None, self.f, self.u, self.st1,
                                       d_gate=g["gate"], d_pre_weight=g["w2"],
                                       d_pre_bias=g["b2"], workspace=self.ws, **self.told1())
        zs.zero_weight_grad(g["W2"], self.df, *self.cy, workspace=self.ws)
        zs.zero_block_quant(*self.qf, self.df)
        self.product(self.dy, self.qf, "W2", True)
        zs.zero_act_backward(self.dy, self.dy, *self.ca, zs.ACT_SILU)
        zs.zero_weight_grad(g["W1"], self.dy, *self.c0, workspace=self.ws)
        zs.zero_block_quant(*self.qy, self.dy)
        self.product(self.dh0, self.qy, "W1", True)
        zs.zero_residual_norm_backward(None, self.du, self.dh0, self.dr, None, self.x32, self.st0,
                                       d_pre_weight=g["w0"], workspace=self.ws, **self.told0())
        self.dx.copy_(self.du)
        zs.zero_embed_grad(g["table"], self.dx, self.ids, workspace=self.ws)

    def update(self):
        zs.zero_overflow_check_dev(self.g16, PSI, 1, 0, self.ctl)
        zs.zero_scaler_update_dev(self.ctl, self.bias, 1)
        zs.zero_adam_step_dev(self.w16, self.g16, self.master, self.m, self.v, PSI, 1, 0,
                              ctl=self.ctl, **HP)
        self.step.add_(1)

    def whole(self):
        self.forward()
        self.backward()
        self.update()

    def state(self):
        return [t.clone() for t in (self.w16, self.g16, self.master, self.m, self.v, self.loss,
                                    self.ctl, self.z, self.u, self.dz, self.step)]


def near(got, want, bound, dt):
    return np.all(np.abs(F64(got) - want) <= grad_plain.rounded(want, bound, dt))


def test_every_operator_of_a_step():
    r = Rank(torch.bfloat16, 3)
    r.batch(4)
    r.step.fill_(5)
    w = {k: F64(t) for k, t in parts(r.w16).items()}
    r.forward()
    r.backward()
    dec = lambda c, block, tall=1: plain.decode(c[0].cpu().numpy(), c[1].cpu().numpy(), tall, block)
    W = {k: dec(c, 128, 128) for k, c in r.codes.items()}
    for k, (q, e, qt, et) in r.codes.items():
        wq, we = plain.encode(w[k], "bf16", 128)
        assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(e.cpu().numpy(), we)
        assert torch.equal(qt, q.t()) and torch.equal(et, e.t())
    P0 = dict(post="none", pre="rms", w2=w["w0"], eps=1e-5, scale=1.0, p=0.0, seed=0, offset=0)
    P1 = dict(post="none", pre="layer", gate=w["gate"], w2=w["w2"], b2=w["b2"], eps=1e-5,
              scale=0.5, p=r.p, seed=99, offset=1005)
    _, _, h0, e, _ = plain.forward(F64(r.x32), None, P0)
    assert near(r.h0, h0, e, "bf16")
    for y, coded, name in ((r.a, r.c0, "W1"), (r.f, r.cy, "W2"), (r.z, r.ch, "out")):
        want, bound = plain.product(dec(coded, 32), W[name], "bf16")
        assert np.all(np.abs(F64(y) - want) <= bound), name
    u, eu, h, eh, _ = plain.forward(F64(r.x32), F64(r.f), P1)
    assert near(r.u, u, eu, "f32") and near(r.h, h, eh, "bf16")
    # backward, from the last layer on
    for y, src, coded, name in ((r.dh, r.dz, r.qz, "out"), (r.dh0, r.dy, r.qy, "W1")):
        q, ex = plain.encode(F64(src), "bf16")
        assert np.array_equal(coded[0].cpu().numpy(), q)
        assert np.array_equal(coded[1].cpu().numpy(), ex)
        want, bound = plain.product(dec(coded, 128), W[name].T, "bf16")
        assert np.all(np.abs(F64(y) - want) <= bound), name
    b1 = plain.backward(F64(r.dh), None, F64(r.f), F64(r.u), F64(r.st1), P1)
    g = parts(r.g16)
    assert near(r.df, *b1["df"], "bf16") and near(r.dr, *b1["dr"], "f32")
    for name in ("gate", "w2", "b2"):
        assert near(g[name], *b1[name], "bf16"), name
    b0 = plain.backward(F64(r.dh0), F64(r.dr), None, F64(r.x32), F64(r.st0), P0)
    assert near(r.du, *b0["dr"], "f32") and near(g["w0"], *b0["w2"], "bf16")
    for name, dy, coded in (("out", r.dz, r.ch), ("W2", r.df, r.cy), ("W1", r.dy, r.c0)):
        want, bound = grad_plain.weight_grad(F64(dy), dec(coded, 32))
        assert near(g[name], want, bound, "bf16"), name
    before = r.w16.clone()
    r.update()
    c = zs.device_ctl_read(r.ctl)
    assert (c.found_inf, c.apply, c.scaler.step) == (0, 1, 1)
    assert not torch.equal(r.w16, before) and int(r.step) == 6


def test_an_infinity_on_the_way_skips_the_step():
    r = Rank(torch.float16, 8)
    r.batch(9)
    r.forward()
    r.f[3, 5] = float("inf")
    zs.zero_residual_norm(r.u, r.h, r.st1, r.x32, r.f, **r.told1())
    before = r.master.clone()
    r.backward()
    r.update()
    c = zs.device_ctl_read(r.ctl)
    assert (c.found_inf, c.apply, c.scaler.loss_scale) == (1, 0, r.S / 2)
    assert torch.equal(r.master, before)


def test_whole_step_captured_and_replayed():
    # eager and captured ranks see the same batches; every replay draws its own masks
    E, G = Rank(torch.bfloat16, 10), Rank(torch.bfloat16, 10)
    for r in (E, G):
        r.batch(11)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        G.whole()
    masks = []
    for k in range(4):
        for r in (E, G):
            r.batch(50 + k)
        torch.cuda.synchronize()
        graph.replay()
        E.whole()
        torch.cuda.synchronize()
        for a, b in zip(E.state(), G.state()):
            assert torch.equal(a, b), k
        masks.append((G.df == 0).float())
    assert int(G.step) == 4 and zs.device_ctl_read(G.ctl).scaler.step == 4
    assert not torch.equal(masks[0], masks[1])
    del graph


def test_two_streams_with_workspaces_of_their_own():
    ranks = [Rank(torch.bfloat16, 20 + i) for i in range(2)]
    want = []
    for i in range(2):
        r = Rank(torch.bfloat16, 20 + i)
        r.batch(30 + i)
        r.whole()
        r.whole()
        want.append(r.state())
    for i, r in enumerate(ranks):
        r.batch(30 + i)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(2):
        for r, s in zip(ranks, streams):
            with torch.cuda.stream(s):
                r.whole()
    torch.cuda.synchronize()
    for r, w in zip(ranks, want):
        for a, b in zip(r.state(), w):
            assert torch.equal(a, b)


def test_work_goes_to_the_given_stream():
    # a long fill on a side stream, then the calls on it by argument: they see its values
    side = torch.cuda.Stream()
    n = 4096
    x = torch.zeros(n, n, dtype=torch.bfloat16, device=DEV)
    q, e = u8(n, n), u8(n, 32)
    qw, ew = u8(256, n), u8(2, 32)
    one = torch.ones(256, n, dtype=torch.bfloat16, device=DEV)
    zs.zero_block_quant(qw, ew, one, square=True)
    y, d = torch.zeros(n, 256, device=DEV), torch.zeros_like(x)
    u, h = torch.zeros_like(x), torch.zeros_like(x)
    ws = u8(zs.zero_block_product_workspace(n, 256, n))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for v in range(1, 30):
            x.fill_(float(v))
    zs.zero_block_quant(q, e, x, stream=side)
    zs.zero_block_product(y, q, e, qw, ew, workspace=ws, stream=side)
    zs.zero_dropout(d, x, 0.0, 1, stream=side)
    zs.zero_residual_norm(u, h, None, x, x, res_scale=2.0, stream=side)
    side.synchronize()
    v = plain.decode(*plain.encode(np.full((1, 1), 29.0), "bf16"))[0, 0]
    assert bool((y == v * n).all()) and bool((d == 29.0).all()) and bool((u == 87.0).all())
    assert bool((h == 1.0).all())


def test_products_with_a_small_grid():
    # a workgroup's tiles one after another: every tile size, ragged and whole
    for m, n, k, dt in ((700, 1030, 300, torch.bfloat16), (2100, 3100, 256, torch.bfloat16),
                        (300, 200, 128, torch.float32), (2100, 2060, 200, torch.float16),
                        (1300, 2050, 1100, torch.float32)):
        g = torch.Generator().manual_seed(m)
        a, b = (torch.randn(r, k, generator=g).to(DEV) for r in (m, n))
        qa, ea, qb, eb = u8(m, k), u8(m, blocks(k)), u8(n, k), u8(blocks(n), blocks(k))
        zs.zero_block_quant(qa, ea, a)
        zs.zero_block_quant(qb, eb, b, square=True)
        ys = [torch.zeros(m, n, dtype=dt, device=DEV) for _ in range(2)]
        ws = u8(zs.zero_block_product_workspace(m, n, k))
        for y, cap in zip(ys, (0, 3)):
            zs.zero_set_grid_cap(cap)
            try:
                zs.zero_block_product(y, qa, ea, qb, eb, workspace=ws)
            finally:
                zs.zero_set_grid_cap(0)
        assert torch.equal(*ys), (m, n, k)
        want, bound = plain.product(plain.decode(qa.cpu().numpy(), ea.cpu().numpy()),
                                    plain.decode(qb.cpu().numpy(), eb.cpu().numpy(), 128),
                                    {v: s for s, v in grad_plain.TORCH.items()}[dt])
        assert np.all(np.abs(F64(ys[0]) - want) <= bound)


def test_past_four_gigabytes():
    # matrices whose bytes pass 2^32: the last rows are what the first rows' copies are
    rows, cols = 70_000, 65_536
    q, e = u8(rows, cols), u8(rows, cols // 128)
    last = slice(rows - 64, rows)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(64, cols, generator=g).bfloat16().to(DEV)
    small = u8(64, cols), u8(64, cols // 128)
    zs.zero_block_quant(*small, x)
    q[last], e[last] = small
    w = torch.randn(200, cols, generator=g).bfloat16().to(DEV)
    qw, ew = u8(200, cols), u8(2, cols // 128)
    zs.zero_block_quant(qw, ew, w, square=True)
    y = torch.zeros(rows, 200, dtype=torch.bfloat16, device=DEV)
    zs.zero_block_product(y, q, e, qw, ew,
                          workspace=u8(zs.zero_block_product_workspace(rows, 200, cols)))
    one = torch.zeros(64, 200, dtype=torch.float32, device=DEV)
    zs.zero_block_product(one, *small, qw, ew,
                          workspace=u8(zs.zero_block_product_workspace(64, 200, cols)))
    want, bound = plain.product(plain.decode(small[0].cpu().numpy(), small[1].cpu().numpy()),
                                plain.decode(qw.cpu().numpy(), ew.cpu().numpy(), 128), "bf16")
    assert np.all(np.abs(F64(y[last]) - want) <= bound) and bool((y[:-64] == 0).all())
    assert np.all(np.abs(F64(one) - want) <= plain.product(
        plain.decode(small[0].cpu().numpy(), small[1].cpu().numpy()),
        plain.decode(qw.cpu().numpy(), ew.cpu().numpy(), 128), "f32")[1])
    big = torch.zeros(rows, 40_000, dtype=torch.bfloat16, device=DEV)
    big[last] = x[:, :40_000]
    out = torch.empty_like(big)
    zs.zero_dropout(out, big, 0.5, 3, 4)
    keep, f = plain.mask(rows, 16, 0.5, 3, 4)
    want = np.where(keep[last], F64(big[last])[:, :16] * float(f), 0.0)
    assert np.array_equal(F64(out[last])[:, :16], want)
