"""Argument checks of the gradient operators, host only: every refusal comes back as a
code before anything touches a device, and empty calls are no-ops.

Pointers are made up and never dereferenced.
"""
import os
import subprocess

import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EDTYPE = -1, -2
A = 0x10_0000_0000          # far-apart, 256-B aligned made-up addresses
STEP = 1 << 32


def at(i, off=0):
    return A + i * STEP + off


def call(name, base, **over):
    args = dict(base)
    args.update(over)
    return getattr(zs.lib, name)(*args.values(), None)


SAVE = dict(q=at(0), e=at(1), y=None, ldy=0, x=at(3), ldx=100, dt=0, act=0, rows=7, cols=100)
LOAD = dict(x=at(0), ldx=100, dt=0, q=at(1), e=at(2), rows=7, cols=100)
BACK = dict(dx=at(0), lddx=100, dy=at(1), lddy=100, dt=0, act=1, q=at(2), e=at(3), rows=7,
            cols=100)
WGRAD = dict(dw=at(0), dw_dt=0, first=1, dy=at(1), lddy=64, dt=0, q=at(2), e=at(3), tokens=9,
             n_out=64, n_in=40, ws=at(4), ws_bytes=1 << 30)
LOOK = dict(out=at(0), ldo=64, table=at(1), dt=0, ids=at(2), it=1, tokens=5, vocab=11, width=64,
            scale=1.0)
EGRAD = dict(dw=at(0), dw_dt=0, first=1, dy=at(1), lddy=64, dt=0, ids=at(2), it=1, tokens=5,
             vocab=11, width=64, scale=1.0, ws=at(3), ws_bytes=1 << 30)
POLICY = dict(loss=at(0), token=at(1), logp=at(2), dl=at(3), ldd=50, z=at(4), ld=50, dt=0,
              targets=at(5), it=1, old=at(6), ref=at(7), adv=at(8), w=at(9), rows=6, vocab=50,
              lo=0.2, hi=0.2, kl=0.1, S=2.0)
INF, NAN = float("inf"), float("nan")
BIG = 0x80000000

REFUSED = [
    ("zero_act_save", SAVE, EDTYPE, [dict(dt=3), dict(dt=-1)]),
    ("zero_act_save", SAVE, EINVAL, [
        dict(act=3), dict(act=-1), dict(q=None), dict(e=None), dict(x=None), dict(ldx=99),
        dict(x=at(3, 1)), dict(dt=2, x=at(3, 2)), dict(rows=BIG), dict(cols=BIG),
        dict(y=at(5)), dict(act=1), dict(act=1, y=at(5), ldy=99), dict(act=1, y=at(5, 1), ldy=100),
        dict(q=at(3, 10)), dict(e=at(3, 1399)), dict(e=at(0, 699)),
        dict(act=1, y=at(3, 2), ldy=100), dict(act=1, y=at(3), ldy=101),
        dict(act=2, y=at(0, 600), ldy=100), dict(act=2, y=at(1), ldy=100),
        dict(rows=0x7fffffff, ldx=1 << 40), dict(ldx=1 << 63)]),
    ("zero_act_load", LOAD, EDTYPE, [dict(dt=5)]),
    ("zero_act_load", LOAD, EINVAL, [
        dict(x=None), dict(q=None), dict(e=None), dict(ldx=99), dict(x=at(0, 1)),
        dict(q=at(0, 4)), dict(e=at(0, 1399)), dict(rows=BIG), dict(cols=BIG)]),
    ("zero_act_backward", BACK, EDTYPE, [dict(dt=3)]),
    ("zero_act_backward", BACK, EINVAL, [
        dict(act=0), dict(act=3), dict(dx=None), dict(dy=None), dict(q=None), dict(e=None),
        dict(lddx=99), dict(lddy=99), dict(dx=at(1, 2)), dict(dx=at(1), lddx=101),
        dict(q=at(0)), dict(e=at(0, 100)), dict(rows=BIG)]),
    ("zero_weight_grad", WGRAD, EDTYPE, [dict(dt=2), dict(dt=7), dict(dw_dt=1), dict(dw_dt=9)]),
    ("zero_weight_grad", WGRAD, EINVAL, [
        dict(first=0), dict(dw=None), dict(dw=at(0, 1)), dict(dw_dt=2, dw=at(0, 2)),
        dict(dy=None), dict(dy=at(1, 1)), dict(lddy=63), dict(q=None), dict(e=None),
        dict(dw=at(1)), dict(dw=at(2)), dict(dw=at(3)), dict(tokens=BIG), dict(n_out=BIG),
        dict(n_in=BIG)]),
    ("zero_embed_lookup", LOOK, EDTYPE, [dict(dt=3), dict(it=2), dict(it=-1)]),
    ("zero_embed_lookup", LOOK, EINVAL, [
        dict(out=None), dict(table=None), dict(ids=None), dict(ldo=63), dict(out=at(0, 1)),
        dict(table=at(1, 1)), dict(ids=at(2, 4)), dict(it=0, ids=at(2, 2)), dict(out=at(1, 128)),
        dict(out=at(2)), dict(tokens=BIG), dict(vocab=BIG), dict(width=BIG)]),
    ("zero_embed_grad", EGRAD, EDTYPE, [dict(dt=2), dict(dw_dt=1), dict(it=5)]),
    ("zero_embed_grad", EGRAD, EINVAL, [
        dict(first=0), dict(dw=None), dict(dy=None), dict(ids=None), dict(lddy=63),
        dict(ids=at(2, 4)), dict(ws=None), dict(ws=at(3, 8)), dict(ws_bytes=100),
        dict(dw=at(1)), dict(dw=at(2)), dict(dw=at(3)), dict(ws=at(1)), dict(ws=at(2)),
        dict(tokens=BIG), dict(vocab=BIG), dict(width=BIG)]),
    ("zero_policy_loss", POLICY, EDTYPE, [dict(dt=3), dict(it=2)]),
    ("zero_policy_loss", POLICY, EINVAL, [
        dict(loss=None), dict(loss=at(0, 2)), dict(token=None), dict(logp=None), dict(z=None),
        dict(targets=None), dict(adv=None), dict(w=None), dict(ld=49), dict(ldd=49),
        dict(z=at(4, 1)), dict(dl=at(3, 1)), dict(targets=at(5, 4)), dict(old=at(6, 2)),
        dict(ref=None), dict(vocab=0), dict(lo=-0.1), dict(lo=1.5), dict(lo=NAN), dict(hi=-0.1),
        dict(hi=NAN), dict(kl=INF), dict(kl=NAN), dict(S=0.0), dict(S=-1.0), dict(S=INF),
        dict(S=NAN), dict(rows=BIG), dict(vocab=BIG), dict(dl=at(4, 2)), dict(dl=at(4), ldd=51),
        dict(loss=at(1)), dict(token=at(2)), dict(logp=at(4)), dict(token=at(9)),
        dict(dl=at(5)), dict(loss=at(7))]),
]


@pytest.mark.parametrize("name,base,code,over", [
    (n, b, c, o) for n, b, c, os in REFUSED for o in os],
    ids=lambda v: v if isinstance(v, str) else "-".join(v) if isinstance(v, dict) and len(v) < 4
    else "")
def test_refusals(name, base, code, over):
    assert call(name, base, **over) == code


def test_weight_grad_needs_its_workspace():
    need = zs.zero_weight_grad_workspace(4096, 64, 40)
    assert need > 0                                  # one tile: the tokens are split
    for over in (dict(ws=None), dict(ws=at(4, 8)), dict(ws_bytes=need - 1), dict(ws=at(1)),
                 dict(ws=at(2)), dict(ws=at(0))):
        assert call("zero_weight_grad", WGRAD, tokens=4096, **over) == EINVAL, over


def test_policy_dev_refusals():
    base = {k: v for k, v in POLICY.items() if k != "S"}
    base["ctl"] = at(10)
    for over in (dict(ctl=None), dict(ctl=at(10, 4)), dict(ctl=at(3)), dict(ctl=at(0)),
                 dict(ctl=at(1)), dict(kl=NAN)):
        assert call("zero_policy_loss_dev", base, **over) == EINVAL, over


@pytest.mark.parametrize("name,base,over", [
    ("zero_act_save", SAVE, dict(rows=0, x=None, q=None, e=None)),
    ("zero_act_save", SAVE, dict(cols=0)),
    ("zero_act_load", LOAD, dict(rows=0, x=None)),
    ("zero_act_backward", BACK, dict(cols=0)),
    ("zero_weight_grad", WGRAD, dict(n_out=0, dw=None)),
    ("zero_weight_grad", WGRAD, dict(n_in=0)),
    ("zero_weight_grad", WGRAD, dict(tokens=0, dw_dt=2, first=0)),
    ("zero_embed_lookup", LOOK, dict(tokens=0, out=None)),
    ("zero_embed_lookup", LOOK, dict(width=0)),
    ("zero_embed_grad", EGRAD, dict(vocab=0, dw=None)),
    ("zero_embed_grad", EGRAD, dict(tokens=0, dw_dt=2, first=0, ws=None)),
])
def test_empty_calls_do_nothing(name, base, over):
    assert call(name, base, **over) == 0


def test_workspace_sizes():
    assert zs.zero_weight_grad_workspace(0, 5, 5) == 0
    assert zs.zero_weight_grad_workspace(16384, 8192, 4096) == 0     # tiles fill the chip
    assert zs.zero_embed_grad_workspace(0, 5, 5) == 0
    assert zs.zero_embed_grad_workspace(100, 0, 5) == 0
    assert zs.zero_embed_grad_workspace(1024, 50257, 768) >= 2 * 4 * 1024
    for fn in (zs.zero_weight_grad_workspace, zs.zero_embed_grad_workspace):
        for bad in ((BIG, 5, 5), (5, BIG, 5), (5, 5, BIG)):
            with pytest.raises(zs.ZeroError):
                fn(*bad)
    assert zs.lib.zero_weight_grad_workspace(1, 1, 1, None) == EINVAL
    assert zs.lib.zero_embed_grad_workspace(1, 1, 1, None) == EINVAL


def test_binding_refuses_host_tensors_and_bad_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, e = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    ids = torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    with pytest.raises(ValueError):
        zs.zero_act_save(q, e, x)
    with pytest.raises(ValueError):
        zs.zero_act_load(x, q, e)
    with pytest.raises(ValueError):
        zs.zero_act_backward(x, x, q, e, zs.ACT_GELU)
    with pytest.raises(ValueError):
        zs.zero_weight_grad(torch.zeros(64, 64, dtype=torch.bfloat16), x, q, e)
    with pytest.raises(ValueError):
        zs.zero_embed_lookup(x, x, ids)
    with pytest.raises(ValueError):
        zs.zero_embed_grad(x, x, ids)
    with pytest.raises(ValueError):
        zs.zero_policy_loss(f[:1], f, f, x, ids, f, f, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                            loss_scale=1.0)
    with pytest.raises(TypeError):
        zs.zero_act_save(q, e, [1.0])


# ---- the 64-bit definitions the GPU tests compare with --------------------------------

def test_plain_codes_match_the_format():
    # the e4m3 facts: largest 448, smallest 2^-9, eight values a binade
    v = plain.CODE_VALUES
    assert v[126] == 448.0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6
    c = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c[:127], v[:127]) and np.isnan(c[127]) and np.isnan(c[255])


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_plain_checkpoint_is_exact_in_its_format_and_within_its_bound(dt):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 97, generator=g) * torch.logspace(-30 if dt != "f16" else -6, 4, 97)
    x = x.to(plain.TORCH[dt])
    x[3, 5], x[4, 40], x[5, 70] = float("inf"), float("nan"), float("-inf")
    x[6] = 0
    big = torch.finfo(plain.TORCH[dt]).max
    x[7, :32], x[8, 33] = big, -big
    xd = plain.f64(x)
    q, e = plain.encode(xd, dt)
    v = plain.decode(q, e)
    fin = np.isfinite(xd)
    assert np.array_equal(np.isnan(v), ~fin)
    back = torch.from_numpy(v).to(plain.TORCH[dt]).double().numpy()
    assert np.array_equal(back[fin], v[fin])
    k = np.repeat(e.astype(int), 32, axis=1)[:, :97] - 127
    bound = np.maximum(np.abs(xd) * 2.0 ** -4, np.ldexp(1.0, k - 10))
    assert np.all(np.abs(v - xd)[fin] <= bound[fin])
    assert e.min() >= 3 and e.max() <= 247


# ---- the header and the host side ---------------------------------------------------------

def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "zero_shard_grad.h"\n'
                   "int main(void) { return ZERO_ACT_BLOCK - 32 + ZERO_ACT_NONE + ZERO_I32; }\n")
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "t")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_fast_division_under_sanitizers(tmp_path):
    inc = "/opt/rocm/include"
    driver = os.path.join(ROOT, "tests", "sanitize", "fast_div_driver.cpp")
    if not os.path.exists(os.path.join(inc, "hip", "hip_runtime_api.h")) or \
            not os.path.exists(driver):
        pytest.skip("HIP headers or the driver not found")
    exe = tmp_path / "fast_div_driver"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=all", "-static-libasan", "-static-libubsan",
                        "-D__HIP_PLATFORM_AMD__", "-I", inc, "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "zero_sharded_mixed_shard_amd", "csrc"), driver,
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout, r.stderr[-2000:])
