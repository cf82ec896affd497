"""The step between two blocks on the GPU, forward and backward, against the 64-bit
definitions within their derived bounds."""
import itertools

import numpy as np
import pytest
import torch

import block_plain as plain
import grad_plain
import zero_sharded_mixed_shard_amd as zs
from test_gpu_x_block_codes import place, untouched

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TORCH = grad_plain.TORCH
KIND = {"none": zs.NORM_NONE, "rms": zs.NORM_RMS, "layer": zs.NORM_LAYER}
F64 = grad_plain.f64


class Case:
    def __init__(self, rows, cols, dt="bf16", res="bf16", post="rms", pre="rms", bias=True,
                 weight=True, gate=True, p=0.1, scale=0.75, eps=1e-5, seed=1, mean=0.5,
                 size=1.0):
        g = torch.Generator().manual_seed(seed + rows * 31 + cols)
        n = lambda shape, s, m: (torch.randn(shape, generator=g) * s + m)
        self.rows, self.cols, self.dt, self.res = rows, cols, dt, res
        self.r = (n((rows, cols), 1.0, mean) * size).to(TORCH[res])
        self.f = (n((rows, cols), 2.0, -mean) * size).to(TORCH[dt])
        self.dh = n((rows, cols), 0.01, 0.0).to(TORCH[dt])
        self.du = n((rows, cols), 0.01, 0.0).to(TORCH[res])
        there = dict(w1=weight and post != "none", b1=bias and post != "none", gate=gate,
                     w2=weight and pre != "none", b2=bias and pre != "none")
        self.par = {k: n(cols, 0.3, {"w1": 1.0, "w2": 1.0, "gate": 0.5}.get(k, 0.0)).to(TORCH[dt])
                    if on else None for k, on in there.items()}
        self.P = dict(post=post, pre=pre, eps=eps, scale=scale, p=p, seed=0x1234567890ab,
                      offset=17 << 34,
                      **{k: None if t is None else t.double().numpy()
                         for k, t in self.par.items()})

    def told(self, par=None):
        par = par or {k: None if t is None else t.to(DEV) for k, t in self.par.items()}
        P = self.P
        return dict(post=KIND[P["post"]], pre=KIND[P["pre"]], post_weight=par["w1"],
                    post_bias=par["b1"], gate=par["gate"], pre_weight=par["w2"],
                    pre_bias=par["b2"], eps=P["eps"], res_scale=P["scale"], p=P["p"],
                    seed=P["seed"], offset=P["offset"])

    def check_forward(self, ld=0, off=0, in_place=False):
        rb, r = place(self.r, ld, off)
        _, f = place(self.f, ld * 2, off)
        ub, u = (rb, r) if in_place else place(torch.zeros_like(self.r), ld, off)
        hb, h = place(torch.zeros_like(self.f), ld + 1, off)
        stats = torch.full((self.rows, 4), 99.0, device=DEV)
        h = None if self.P["pre"] == "none" else h
        zs.zero_residual_norm(u, h, stats, r, f, **self.told())
        wu, eu, wh, eh, ws = plain.forward(F64(self.r), F64(self.f), self.P)
        assert np.all(np.abs(F64(u) - wu) <= plain.rounded(wu, eu, self.res))
        assert untouched(ub, u, off)
        if h is not None:
            assert np.all(np.abs(F64(h) - wh) <= plain.rounded(wh, eh, self.dt))
            assert untouched(hb, h, off)
        got = F64(stats)
        for k, kind in ((0, self.P["post"]), (2, self.P["pre"])):
            if kind == "none":
                assert np.all(got[:, k] == 0) and np.all(got[:, k + 1] == 1)
            else:
                x, ex = (F64(self.f), np.zeros_like(wu)) if k == 0 else (wu, eu)
                _, _, mean, rho = plain.normed(x, ex, kind, float(np.float32(self.P["eps"])))
                em = (np.abs(x).mean(1) * (plain.row_adds(self.cols) + 3) * plain.U +
                      ex.mean(1)) * (kind == "layer")
                assert np.all(np.abs(got[:, k] - mean) <= em * 1.01)
                d = x - mean[:, None]
                var = (d * d).mean(1)
                ed = ex + em[:, None] + np.abs(d) * plain.U
                ev = var * (plain.row_adds(self.cols) + 6) * plain.U + \
                    (2 * np.abs(d) * ex + ed * ed).mean(1) * 1.01
                rel = 0.5 * ev / (var + self.P["eps"]) * 1.02 + 5 * plain.U
                assert np.all(np.abs(got[:, k + 1] - rho) <= rho * rel)
        return u, h, stats

    def check_backward(self, out="f32", first=True, ld=0, off=0, in_place=False, du=True,
                       want=("w1", "b1", "gate", "w2", "b2")):
        u64, _, _, _, st = plain.forward(F64(self.r), F64(self.f), self.P)
        u = torch.from_numpy(u64).to(TORCH[self.res])
        stats = torch.from_numpy(st).float()
        dh = None if self.P["pre"] == "none" else self.dh
        exact = plain.backward(None if dh is None else F64(dh), F64(self.du) if du else None,
                               F64(self.f), F64(u), stats.double().numpy(), self.P)
        _, dev_u = place(u, ld, off)
        _, dev_f = place(self.f, ld + 3, off)
        dhb, dev_dh = (None, None) if dh is None else place(dh, ld, off)
        dub, dev_du = place(self.du, ld + 2, off) if du else (None, None)
        dfb, df = (dhb, dev_dh) if in_place and dh is not None else \
            place(torch.zeros_like(self.f), ld, off)
        drb, dr = (dub, dev_du) if in_place and du else place(torch.zeros_like(self.r), ld, off)
        base, grads = {}, {}
        for k, t in self.par.items():
            if t is None or k not in want:
                grads[k] = None
                continue
            base[k] = torch.randn(self.cols, generator=torch.Generator().manual_seed(3))
            buf = torch.full((self.cols + 2,), 77.0, device=DEV).to(TORCH[out])
            buf[1:-1] = base[k].to(TORCH[out])
            base[k], grads[k] = buf[1:-1].cpu().clone(), buf[1:-1]
        ws = torch.full((zs.zero_residual_norm_workspace(self.rows, self.cols),), 255,
                        dtype=torch.uint8, device=DEV)
        zs.zero_residual_norm_backward(
            df, dr, dev_dh, dev_du, dev_f, dev_u, stats.to(DEV), d_post_weight=grads["w1"],
            d_post_bias=grads["b1"], d_gate=grads["gate"], d_pre_weight=grads["w2"],
            d_pre_bias=grads["b2"], first=first, workspace=ws, **self.told())
        for name, t, fmt in (("dr", dr, self.res), ("df", df, self.dt)):
            v, e = exact[name]
            assert np.all(np.abs(F64(t) - v) <= plain.rounded(v, e, fmt)), name
        assert untouched(dfb, df, off) and untouched(drb, dr, off)
        for k, t in grads.items():
            if t is None:
                continue
            v, e = exact[k]
            if not first:
                b = F64(base[k])
                v, e = v + b, e + np.abs(v + b) * plain.U
            assert np.all(np.abs(F64(t) - v) <= plain.rounded(v, e, out)), k
        return df, dr, grads


NORMS = list(itertools.product(["none", "rms", "layer"], ["none", "rms", "layer"]))


@pytest.mark.parametrize("post,pre", NORMS)
@pytest.mark.parametrize("dt,res", [("f16", "f16"), ("bf16", "f32"), ("f32", "f32")])
def test_every_pair_of_norms(post, pre, dt, res):
    c = Case(37, 203, dt, res, post, pre)
    c.check_forward(ld=3, off=1)
    c.check_backward(out="f32", ld=3, off=1)
    c.check_backward(out=dt)


# widths around a group of eight, a wave, a workgroup and past what one holds
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 2), (1, 8), (3, 9), (5, 63), (4, 511), (3, 512),
                                       (2, 513), (6, 768), (5, 1024), (7, 1025), (3, 1601),
                                       (4, 2048), (2, 2056), (5, 4096), (3, 5120), (2, 8192),
                                       (3, 8193), (2, 12552), (2, 16384), (2, 16385), (1, 40001)])
@pytest.mark.parametrize("dt,res,post,pre", [("bf16", "bf16", "layer", "rms"),
                                             ("f16", "f32", "rms", "layer"),
                                             ("f32", "f32", "layer", "layer")])
def test_widths(rows, cols, dt, res, post, pre):
    c = Case(rows, cols, dt, res, post, pre)
    c.check_forward(off=cols % 2)
    c.check_backward(off=cols % 2)


@pytest.mark.parametrize("rows,cols", [(255, 64), (257, 130), (1023, 768), (600, 2048), (2500, 96),
                                       (5000, 24)])
@pytest.mark.parametrize("dt,res,post,pre,p", [("bf16", "f32", "rms", "rms", 0.0),
                                               ("f16", "f16", "none", "layer", 0.1)])
def test_many_rows(rows, cols, dt, res, post, pre, p):
    c = Case(rows, cols, dt, res, post, pre, p=p)
    c.check_forward()
    c.check_backward(out=dt)
    c.check_backward(first=False)


@pytest.mark.parametrize("cols", [96, 768, 3000, 17000])
def test_in_place(cols):
    c = Case(20, cols, "bf16", "bf16", "layer", "rms")
    a = c.check_forward()
    b = c.check_forward(in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    a = c.check_backward()
    b = c.check_backward(in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("weight,bias,gate", list(itertools.product([False, True], repeat=3)))
def test_parameters_that_are_not_there(weight, bias, gate):
    c = Case(40, 300, "bf16", "f32", "rms", "layer", weight=weight, bias=bias, gate=gate)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("p", [0.0, 0.5, 1.0])
def test_dropout_inside_is_the_operators_own(p):
    # without norms and gate: u - scale r is what zero_dropout makes of f
    c = Case(50, 123, "f32", "f32", "none", "none", gate=False, p=p, scale=0.0)
    u, _, _ = c.check_forward()
    y = torch.empty(50, 123, device=DEV)
    zs.zero_dropout(y, c.f.to(DEV), p, c.P["seed"], c.P["offset"])
    assert torch.equal(u + 0.0, y + 0.0)
    df, _, _ = c.check_backward()
    zs.zero_dropout(y, c.du.to(DEV), p, c.P["seed"], c.P["offset"])
    assert torch.equal(df + 0.0, y + 0.0)


@pytest.mark.parametrize("cols", [100, 1500, 20000])
def test_without_a_gradient_of_the_stream(cols):
    c = Case(9, cols, "bf16", "bf16", "rms", "layer")
    c.check_backward(du=False)
    c.check_backward(want=("gate",))
    c.check_backward(want=())


@pytest.mark.parametrize("cols", [64, 777, 3000, 20000])
@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_first_norm_of_a_stack(cols, pre):
    c = Case(11, cols, "f16", "f32", "none", pre, gate=False, p=0.0, scale=1.0)
    told = c.told()
    h, stats = torch.zeros(11, cols, dtype=torch.float16, device=DEV), \
        torch.zeros(11, 4, device=DEV)
    r = c.r.to(DEV)
    zs.zero_residual_norm(None, h, stats, r, **told)
    _, _, wh, eh, _ = plain.forward(F64(c.r), None, c.P)
    assert np.all(np.abs(F64(h) - wh) <= plain.rounded(wh, eh, "f16"))
    assert bool((stats[:, 0] == 0).all()) and bool((stats[:, 1] == 1).all())
    dr = torch.zeros_like(r)
    gw, gb = torch.zeros(cols, device=DEV), torch.zeros(cols, device=DEV)
    ws = torch.empty(zs.zero_residual_norm_workspace(11, cols), dtype=torch.uint8, device=DEV)
    zs.zero_residual_norm_backward(None, dr, c.dh.to(DEV), c.du.to(DEV), None, r, stats,
                                   d_pre_weight=gw, d_pre_bias=gb, workspace=ws, **told)
    exact = plain.backward(F64(c.dh), F64(c.du), None, F64(c.r), F64(stats), c.P)
    for name, t in (("dr", dr), ("w2", gw), ("b2", gb)):
        v, e = exact[name]
        assert np.all(np.abs(F64(t) - v) <= plain.rounded(v, e, "f32")), name


@pytest.mark.parametrize("cols", [60, 3000, 20000])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_of_large_and_of_equal_values(cols, kind):
    # values whose squares leave FP32, and rows without any deviation
    for size in (1e25, 1e30, 1e-12):
        c = Case(5, cols, "bf16", "f32", kind, kind, bias=False, p=0.0, size=size, gate=False)
        c.check_forward()
    c = Case(5, cols, "f32", "f32", "none", kind, gate=False, bias=False, weight=False, p=0.0,
             scale=1.0)
    c.f.zero_()
    c.r[:] = torch.tensor([0.0, 1.0, -3.0, 1e30, 2.5e38])[:, None]
    u, h, _ = torch.zeros(5, cols, device=DEV), torch.zeros(5, cols, device=DEV), None
    zs.zero_residual_norm(u, h, None, c.r.to(DEV), c.f.to(DEV), **c.told())
    assert torch.equal(u.cpu(), c.r)
    if kind == "layer":
        # the mean of equal values is off by its sum's rounding, at most row_adds half steps
        lim = plain.row_adds(cols) * 2 * plain.U * np.abs(F64(c.r)[:, 0]) / np.sqrt(1e-5)
        assert np.all(np.abs(F64(h))[:3] <= lim[:3, None])
        assert bool(h.isfinite().all())
    else:
        want = F64(c.r) / np.sqrt(F64(c.r) ** 2 + 1e-5)
        assert np.all(np.abs(F64(h) - want) <= plain.row_adds(cols) * 2 * plain.U)


@pytest.mark.parametrize("cols", [70, 3000, 20000])
def test_rows_that_are_not_finite_leave_the_others_alone(cols):
    c = Case(6, cols, "bf16", "bf16", "layer", "rms")
    f = c.f.to(DEV)
    told = c.told()
    u, h = torch.zeros_like(f), torch.zeros_like(f)
    zs.zero_residual_norm(u, h, None, c.r.to(DEV), f, **told)
    f2 = f.clone()
    f2[1, 3], f2[4, cols - 1] = float("nan"), float("inf")
    u2, h2 = torch.zeros_like(f), torch.zeros_like(f)
    zs.zero_residual_norm(u2, h2, None, c.r.to(DEV), f2, **told)
    bad = torch.tensor([False, True, False, False, True, False])
    assert torch.equal(u2[~bad], u[~bad]) and torch.equal(h2[~bad], h[~bad])
    assert bool(h2[bad].isnan().all())


def test_repeats_and_small_grids():
    for cols in (100, 900, 3000, 17000):
        c = Case(70, cols, "bf16", "f32", "rms", "layer")
        a, b = c.check_forward(), c.check_backward()
        zs.zero_set_grid_cap(2)
        try:
            a2, b2 = c.check_forward(), c.check_backward()
        finally:
            zs.zero_set_grid_cap(0)
        for x, y in zip(a[:3] + b[:2], a2[:3] + b2[:2]):
            assert torch.equal(x, y)
        for k in b[2]:
            assert torch.equal(b[2][k], b2[2][k])


def test_no_rows():
    c = Case(5, 40, "bf16", "f32", "rms", "rms")
    g = torch.ones(40, device=DEV)
    e = torch.zeros(0, 40, dtype=torch.bfloat16, device=DEV)
    e32, st = torch.zeros(0, 40, device=DEV), torch.zeros(0, 4, device=DEV)
    told = c.told()
    zs.zero_residual_norm(e32, e, st, e32, e, **told)
    zs.zero_residual_norm_backward(e, e32, e, e32, e, e32, st, d_gate=g, first=False, **told)
    assert bool((g == 1).all())
    zs.zero_residual_norm_backward(e, e32, e, e32, e, e32, st, d_gate=g, **told)
    assert bool((g == 0).all())


def test_refusals():
    c = Case(5, 40, "bf16", "f32", "rms", "rms")
    told = c.told()
    f, r = c.f.to(DEV), c.r.to(DEV)
    u, h, st = torch.zeros_like(r), torch.zeros_like(f), torch.zeros(5, 4, device=DEV)
    for bad in (dict(u=u.bfloat16()), dict(h=h.float()), dict(stats=st[:4]), dict(r=r[:4]),
                dict(f=f[:, :39]), dict(gate=told["gate"][:39]), dict(gate=told["gate"].float()),
                dict(r=r.cpu())):
        a = dict(u=u, h=h, stats=st, r=r, f=f, **told)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            zs.zero_residual_norm(**a)
    ws = torch.empty(zs.zero_residual_norm_workspace(5, 40), dtype=torch.uint8, device=DEV)
    a = dict(df=h, dr=u, dh=c.dh.to(DEV), du=c.du.to(DEV), f=f, u=r, stats=st, workspace=ws,
             **told)
    g = torch.zeros(40, device=DEV)
    for bad in (dict(d_gate=g[:39]), dict(d_gate=g, d_pre_bias=g.bfloat16()), dict(d_gate=g.half()),
                dict(df=h.float()), dict(workspace=g)):
        with pytest.raises((ValueError, TypeError)):
            zs.zero_residual_norm_backward(**dict(a, **bad))
    for bad in (dict(workspace=None), dict(d_gate=g.bfloat16(), first=False), dict(eps=0.0)):
        with pytest.raises(zs.ZeroError):
            zs.zero_residual_norm_backward(**dict(a, **bad))


@pytest.mark.parametrize("cols", [60, 3000, 20000])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_a_large_epsilon_beside_large_values(cols, kind):
    # where rows are summed scaled, epsilon is still part of the deviation
    for eps, size in ((1e36, 1e18), (1e38, 1e19), (1e30, 1e18)):
        c = Case(5, cols, "bf16", "f32", kind, kind, bias=False, p=0.0, size=size, gate=False,
                 eps=eps, scale=1.0)
        c.check_forward()
