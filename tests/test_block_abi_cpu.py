"""The operators around a block's linear layers, host side only: every refusal comes back
as a code before anything touches a device, empty calls are no-ops, the structures match
the header, and the 64-bit definitions that the GPU tests compare with hold.

Pointers are made up and never dereferenced.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import block_plain as plain
import zero_sharded_mixed_shard_amd as zs
from zero_sharded_mixed_shard_amd import _block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EDTYPE = -1, -2
A = 0x10_0000_0000          # far-apart, 256-B aligned made-up addresses
STEP = 1 << 32
INF, NAN, BIG = float("inf"), float("nan"), 0x80000000


def at(i, off=0):
    return A + i * STEP + off


def call(name, base, **over):
    args = dict(base)
    args.update(over)
    return getattr(zs.lib, name)(*args.values(), None)


QUANT = dict(q=at(0), e=at(1), qt=None, et=None, x=at(4), ldx=200, dt=0, blocks=0, rows=7,
             cols=200)
SQUARE = dict(QUANT, qt=at(2), et=at(3), blocks=1)
LOAD = dict(x=at(0), ldx=200, dt=0, q=at(1), e=at(2), blocks=0, rows=7, cols=200)
PRODUCT = dict(y=at(0), ldy=64, dt=0, qa=at(1), ea=at(2), a_block=128, qb=at(3), eb=at(4), m=9,
               n=64, k=300, ws=at(5), ws_bytes=1 << 31)
DROP = dict(y=at(0), ldy=100, x=at(1), ldx=100, dt=0, rows=7, cols=100, p=0.1, seed=1, offset=2,
            d_offset=at(2))

REFUSED = [
    ("zero_block_quant", QUANT, EDTYPE, [dict(dt=3), dict(dt=-1)]),
    ("zero_block_quant", QUANT, EINVAL, [
        dict(blocks=2), dict(blocks=-1), dict(q=None), dict(e=None), dict(x=None), dict(ldx=199),
        dict(x=at(4, 1)), dict(dt=2, x=at(4, 2)), dict(rows=BIG), dict(cols=BIG),
        dict(qt=at(2)), dict(et=at(3)), dict(qt=at(2), et=at(3)), dict(q=at(4, 10)),
        dict(e=at(4, 2799)), dict(e=at(0, 1399)), dict(ldx=1 << 63)]),
    ("zero_block_quant", SQUARE, EINVAL, [
        dict(et=None), dict(qt=None), dict(qt=at(0, 1399)), dict(et=at(1, 1)), dict(et=at(2)),
        dict(qt=at(4)), dict(et=at(4, 100)), dict(e=at(2, 1399))]),
    ("zero_block_load", LOAD, EDTYPE, [dict(dt=5)]),
    ("zero_block_load", LOAD, EINVAL, [
        dict(blocks=3), dict(x=None), dict(q=None), dict(e=None), dict(ldx=199), dict(x=at(0, 1)),
        dict(q=at(0, 4)), dict(e=at(0, 2799)), dict(rows=BIG), dict(cols=BIG)]),
    ("zero_block_product", PRODUCT, EDTYPE, [dict(dt=3), dict(dt=-1)]),
    ("zero_block_product", PRODUCT, EINVAL, [
        dict(a_block=64), dict(a_block=0), dict(y=None), dict(y=at(0, 1)), dict(ldy=63),
        dict(qa=None), dict(ea=None), dict(qb=None), dict(eb=None), dict(qa=at(0, 5)),
        dict(ea=at(0, 64)), dict(qb=at(0)), dict(eb=at(0, 1151)), dict(m=BIG), dict(n=BIG),
        dict(k=BIG), dict(dt=2, y=at(0, 2)), dict(k=0, y=None)]),
    ("zero_dropout", DROP, EDTYPE, [dict(dt=4)]),
    ("zero_dropout", DROP, EINVAL, [
        dict(p=-0.1), dict(p=1.1), dict(p=NAN), dict(y=None), dict(x=None), dict(ldy=99),
        dict(ldx=99), dict(y=at(0, 1)), dict(d_offset=at(2, 4)), dict(d_offset=at(0, 8)),
        dict(y=at(1, 2)), dict(y=at(1), ldy=101), dict(rows=BIG), dict(cols=BIG)]),
]


@pytest.mark.parametrize("name,base,code,over", [
    (n, b, c, o) for n, b, c, os_ in REFUSED for o in os_],
    ids=lambda v: v if isinstance(v, str) else "-".join(v) if isinstance(v, dict) and len(v) < 5
    else "")
def test_refusals(name, base, code, over):
    assert call(name, base, **over) == code


@pytest.mark.parametrize("name,base,over", [
    ("zero_block_quant", QUANT, dict(rows=0, x=None, q=None, e=None)),
    ("zero_block_quant", SQUARE, dict(cols=0, qt=None, et=None)),
    ("zero_block_load", LOAD, dict(cols=0, x=None)),
    ("zero_block_product", PRODUCT, dict(m=0, y=None, qa=None)),
    ("zero_block_product", PRODUCT, dict(n=0, qb=None)),
    ("zero_dropout", DROP, dict(rows=0, y=None)),
    ("zero_dropout", DROP, dict(cols=0)),
])
def test_empty_calls_do_nothing(name, base, over):
    assert call(name, base, **over) == 0


# ---- the step between two blocks ----------------------------------------------------------

def block(**over):
    d = dict(rows=7, cols=100, dt=1, res_dt=1, post=1, pre=2, post_weight=at(20),
             post_bias=at(21), gate=at(22), pre_weight=at(23), pre_bias=at(24), eps=1e-5,
             res_scale=1.0, p=0.1, seed=3, offset=4, d_offset=at(25))
    d.update(over)
    return _block._Residual(**d)


def forward(b, **over):
    a = dict(u=at(0), ldu=100, h=at(1), ldh=100, stats=at(2), r=at(3), ldr=100, f=at(4), ldf=100)
    a.update(over)
    return zs.lib.zero_residual_norm(*a.values(), None if b is None else ctypes.byref(b), None)


def backward(b, grads=None, **over):
    a = dict(df=at(0), lddf=100, dr=at(1), lddr=100, grads=None, grad_dt=1, first=1, dh=at(3),
             lddh=100, du=at(4), lddu=100, f=at(5), ldf=100, u=at(6), ldu=100, stats=at(7),
             block=None if b is None else ctypes.byref(b), ws=at(8), ws_bytes=1 << 31)
    if grads is not None:
        a["grads"] = ctypes.byref(_block._ResidualGrads(**grads))
    a.update(over)
    return zs.lib.zero_residual_norm_backward(*a.values(), None)


BAD_BLOCKS = [dict(post=3), dict(pre=-1), dict(rows=BIG), dict(cols=BIG), dict(eps=0.0),
              dict(eps=-1.0), dict(eps=INF), dict(eps=NAN), dict(eps=2.0 ** -81),
              dict(res_scale=INF), dict(res_scale=NAN), dict(p=-0.5), dict(p=2.0), dict(p=NAN),
              dict(d_offset=at(25, 4)), dict(post=0), dict(gate=at(22, 1)),
              dict(pre_weight=at(23, 1)), dict(post=0, post_weight=None),
              dict(post=0, post_bias=None)]


@pytest.mark.parametrize("over", BAD_BLOCKS, ids=str)
def test_residual_descriptions_refused(over):
    assert forward(block(**over)) == EINVAL
    assert backward(block(**over)) == EINVAL


@pytest.mark.parametrize("over", [dict(dt=3), dict(res_dt=0), dict(dt=2, res_dt=1)], ids=str)
def test_residual_formats_refused(over):
    assert forward(block(**over)) == EDTYPE
    assert backward(block(**over)) == EDTYPE


@pytest.mark.parametrize("over", [
    dict(u=None), dict(h=None), dict(r=None), dict(f=None), dict(ldu=99), dict(ldh=99),
    dict(ldr=99), dict(ldf=99), dict(u=at(0, 1)), dict(stats=at(2, 2)), dict(u=at(3, 2)),
    dict(u=at(3), ldu=101), dict(h=at(3)), dict(h=at(4)), dict(u=at(4)), dict(u=at(1)),
    dict(stats=at(0)), dict(stats=at(4, 4)), dict(stats=at(20)), dict(h=at(23, 8)),
    dict(u=at(25)), dict(h=at(22))], ids=str)
def test_residual_forward_refusals(over):
    assert forward(block(), **over) == EINVAL


def test_residual_forward_without_a_branch():
    alone = dict(post=0, post_weight=None, post_bias=None, gate=None, p=0.0)
    none = dict(u=None, f=None)
    assert forward(block(**dict(alone, rows=0)), **none) == 0
    assert forward(block(rows=0), u=None, h=None, r=None, f=None) == 0   # no rows, no pointers
    assert forward(block(cols=0), u=None, h=None, r=None, f=None) == 0
    assert forward(block(rows=0, post=3)) == EINVAL
    for over in (dict(post=1), dict(gate=at(22)), dict(p=0.1), dict(res_scale=0.5),
                 dict(pre=0, pre_weight=None, pre_bias=None)):
        assert forward(block(**dict(alone, **over)), **none) == EINVAL, over
    assert forward(None) == EINVAL
    assert forward(block(**alone), f=None) == EINVAL     # u without f


@pytest.mark.parametrize("over", [
    dict(df=None), dict(dr=None), dict(dh=None), dict(f=None), dict(u=None), dict(stats=None),
    dict(lddf=99), dict(lddr=99), dict(lddh=99), dict(lddu=99), dict(ldf=99), dict(ldu=99),
    dict(first=0), dict(ws=None), dict(ws=at(8, 8)), dict(ws_bytes=16), dict(stats=at(7, 2)),
    dict(df=at(3, 2)), dict(df=at(3), lddf=101), dict(dr=at(4), lddr=101), dict(dr=at(3)),
    dict(df=at(4)), dict(df=at(5)), dict(dr=at(6)), dict(dr=at(0)), dict(df=at(7)),
    dict(ws=at(0)), dict(ws=at(6)), dict(ws=at(3)), dict(dr=at(20)), dict(df=at(25))], ids=str)
def test_residual_backward_refusals(over):
    assert backward(block(), **over) == EINVAL


def test_residual_gradients_refused():
    ok = dict(post_weight=at(30), post_bias=at(31), gate=at(32), pre_weight=at(33),
              pre_bias=at(34))
    for name in ok:
        assert backward(block(**{name: None}), {name: ok[name]}) == EINVAL   # no such parameter
        assert backward(block(), {name: ok[name] + 1}) == EINVAL
        assert backward(block(), {name: ok[name] + 2}, grad_dt=2) == EINVAL
        for other in (0, 1, 3, 4, 5, 6, 7, 8, 20, 22, 23):
            assert backward(block(), {name: at(other)}) == EINVAL, (name, other)
    assert backward(block(), dict(ok, gate=ok["pre_bias"])) == EINVAL
    assert backward(block(), ok, grad_dt=0) == EDTYPE
    assert backward(block(), ok, grad_dt=7) == EDTYPE
    assert backward(None, ok) == EINVAL


def test_residual_backward_empty():
    assert backward(block(cols=0)) == 0
    assert backward(block(rows=0), None, dr=None, ws=None) == 0
    ok = dict(pre_weight=at(33))
    assert backward(block(rows=0), ok, grad_dt=2, first=0) == 0
    none = dict(pre=0, pre_weight=None, pre_bias=None)
    assert backward(block(**none), dh=None, du=None) == EINVAL
    assert backward(block(**none)) == EINVAL             # dh without a norm


def test_workspace_sizes():
    assert zs.zero_residual_norm_workspace(0, 5) == zs.zero_residual_norm_workspace(5, 0) == 0
    assert zs.zero_block_product_workspace(0, 5, 5) == 0
    assert zs.zero_block_product_workspace(5, 5, 0) == 0
    assert zs.lib.zero_residual_norm_workspace(1, 1, None) == EINVAL
    assert zs.lib.zero_block_product_workspace(1, 1, 1, None) == EINVAL
    for bad in ((BIG, 5), (5, BIG)):
        with pytest.raises(zs.ZeroError):
            zs.zero_residual_norm_workspace(*bad)
    for bad in ((BIG, 5, 5), (5, BIG, 5), (5, 5, BIG)):
        with pytest.raises(zs.ZeroError):
            zs.zero_block_product_workspace(*bad)


def test_binding_refuses_host_tensors_and_bad_shapes():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, e = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        zs.zero_block_quant(q, e, x)
    with pytest.raises(ValueError):
        zs.zero_block_load(x, q, e)
    with pytest.raises(ValueError):
        zs.zero_block_product(x, q, e, q, e)
    with pytest.raises(ValueError):
        zs.zero_dropout(x, x, 0.1, 1)
    with pytest.raises(ValueError):
        zs.zero_residual_norm(x, x, None, x, x)
    with pytest.raises(ValueError):
        zs.zero_residual_norm_backward(x, x, x, x, x, x, torch.zeros(4, 4))
    with pytest.raises(TypeError):
        zs.zero_dropout(x, [1.0], 0.1, 1)


def test_structures_match_the_header(tmp_path):
    src = tmp_path / "t.c"
    fields = [f for f, _ in _block._Residual._fields_]
    grads = [f for f, _ in _block._ResidualGrads._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "zero_shard_block.h"\n'
                   "int main(void) {\n"
                   'printf("%zu %zu", sizeof(zero_residual), sizeof(zero_residual_grads));\n' +
                   "".join(f'printf(" %zu", offsetof(zero_residual, {f}));\n' for f in fields) +
                   "".join(f'printf(" %zu", offsetof(zero_residual_grads, {f}));\n'
                           for f in grads) +
                   'printf(" %d %d %d %d", ZERO_BLOCK, ZERO_NORM_NONE, ZERO_NORM_RMS, '
                   "ZERO_NORM_LAYER);\nreturn 0;\n}\n")
    exe = str(tmp_path / "t")
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = [ctypes.sizeof(_block._Residual), ctypes.sizeof(_block._ResidualGrads)]
    want += [getattr(_block._Residual, f).offset for f in fields]
    want += [getattr(_block._ResidualGrads, f).offset for f in grads]
    assert got == want + [zs.BLOCK, zs.NORM_NONE, zs.NORM_RMS, zs.NORM_LAYER]


# ---- the 64-bit definitions -----------------------------------------------------------------

def test_philox_against_its_published_vectors():
    # the three test vectors of Philox4x32-10 that the authors publish with the method
    f = 0xffffffff
    for ctr, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((f, f, f, f), (f, f), (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        got = plain.philox([np.array([c]) for c in ctr], key)
        assert tuple(int(g[0]) for g in got) == want


def test_mask_keeps_its_share():
    # keep is binomial with the share 1 - t / 65536: within five deviations
    for p in (0.05, 0.1, 0.5):
        keep, f = plain.mask(500, 1003, p, 77, 5)
        t = plain.threshold(p) / 65536
        assert abs(keep.mean() - (1 - t)) < 5 * np.sqrt(t * (1 - t) / keep.size)
        assert abs(float(f) * (1 - t) - 1) < 2.0 ** -23
    assert plain.mask(3, 9, 0.0, 1, 1)[0].all() and not plain.mask(3, 9, 1.0, 1, 1)[0].any()
    # another seed or offset: another mask
    a = plain.mask(40, 40, 0.5, 1, 1)[0]
    for seed, off in ((2, 1), (1, 2), (1 + 2 ** 32, 1), (1, 1 + 2 ** 32)):
        assert (a != plain.mask(40, 40, 0.5, seed, off)[0]).mean() > 0.4


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_plain_gradients_against_differences(post, pre):
    # central differences of a random functional of u and h along random directions: the
    # quotient's error is of the order step^2 times a third derivative
    rng = np.random.default_rng(5)
    rows, cols = 4, 23
    v = lambda: rng.standard_normal(cols)
    P = dict(post=post, pre=pre, w1=v() if post != "none" else None,
             b1=v() if post != "none" else None, gate=v(),
             w2=v() if pre != "none" else None, b2=v() if pre != "none" else None, eps=1e-3,
             scale=0.75, p=0.25, seed=9, offset=11)
    r, f, cu, ch = (rng.standard_normal((rows, cols)) for _ in range(4))
    if pre == "none":
        ch = None

    def value(r, f, P):
        u, _, h, _, _ = plain.forward(r, f, P)
        return (u * cu).sum() + (0.0 if h is None else (h * ch).sum())

    u, _, _, _, stats = plain.forward(r, f, P)
    grads = plain.backward(ch, cu, f, u, stats, P)
    step = 1e-5
    for name in ("dr", "df", "w1", "b1", "gate", "w2", "b2"):
        x = {"dr": r, "df": f}.get(name, P.get(name))
        if x is None:
            continue
        d = rng.standard_normal(x.shape)
        sides = []
        for sign in (1, -1):
            y = x + sign * step * d
            sides.append(value(y if name == "dr" else r, y if name == "df" else f,
                               P if name in ("dr", "df") else dict(P, **{name: y})))
        slope = (sides[0] - sides[1]) / (2 * step)
        want = (grads[name][0] * d).sum()
        assert abs(slope - want) <= 1e-6 * (np.abs(grads[name][0] * d).sum() + 1), name
