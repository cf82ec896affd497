"""8-bit activation checkpoints on the GPU against their 64-bit definition.

Codes, exponents and values read back are compared bit for bit; the activation's
forward and backward results within the bounds derived in grad_plain.py.
"""
import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
ACTS = {"gelu": zs.ACT_GELU, "silu": zs.ACT_SILU}
FILL = {torch.float16: 7.5, torch.bfloat16: 7.5, torch.float32: 7.5, torch.uint8: 171}


class Framed:
    """A [rows, cols] device matrix of row stride ld inside a buffer of guard values,
    `lead` elements in; intact() checks everything outside the matrix."""

    def __init__(self, rows, cols, dtype, ld=None, lead=3):
        self.ld = cols if ld is None else ld
        self.rows, self.cols, self.lead = rows, cols, lead
        n = lead + rows * self.ld + 37
        self.buf = torch.full((n,), FILL[dtype], dtype=dtype, device=DEV)
        self.t = self.buf.as_strided((rows, cols), (self.ld, 1), lead)

    def intact(self) -> bool:
        mask = torch.ones_like(self.buf, dtype=torch.bool)
        mask.as_strided((self.rows, self.cols), (self.ld, 1), self.lead).fill_(False)
        return bool((self.buf[mask] == FILL[self.buf.dtype]).all())


def values(rows, cols, dt, seed, rare=True):
    """Wide-ranging values with every awkward one: zeros, blocks of zeros, ties, the
    format's ends, subnormals, infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.exp2(torch.randint(-12, 6, (rows, (cols + 31) // 32), generator=g).float()) \
        .repeat_interleave(32, 1)[:, :cols]
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0
    x = x.to(plain.TORCH[dt])
    if rare:
        big = torch.finfo(x.dtype).max
        tiny = torch.finfo(x.dtype).smallest_normal
        odd = [float("inf"), -float("inf"), float("nan"), big, -big, tiny, -tiny / 4, 448.0,
               449.0, 464.0, 0.0, -0.0, 2.0 ** -9, 1.0625, 1.1875]
        for i, v in enumerate(odd):
            x[(3 * i) % rows, (7 * i) % cols] = v
        if rows > 2:
            x[1] = 0
            x[2] = tiny * 0.25
    return x


def bits_equal(a, b) -> bool:
    """Equal values (NaN equal to NaN, zeros by sign)."""
    a, b = a.cpu().double().numpy(), np.asarray(b, dtype=np.float64)
    return bool(np.array_equal(a, b, equal_nan=True) and
                np.array_equal(np.signbit(a) | np.isnan(a), np.signbit(b) | np.isnan(b)))


# (rows, cols, ld - cols, lead): flat and strided, one element, odd widths, ends of blocks
SHAPES = [(1, 1, 0, 0), (1, 31, 0, 0), (3, 32, 0, 0), (5, 33, 0, 1), (7, 64, 0, 2),
          (2, 7, 0, 0), (16, 200, 8, 0), (33, 257, 3, 5), (64, 1024, 0, 0), (9, 2050, 1, 1),
          (300, 96, 0, 4), (1, 100_003, 0, 1), (1025, 5, 2, 0)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,gap,lead", SHAPES)
def test_checkpoint_matches_its_definition(rows, cols, gap, lead, dt):
    x = Framed(rows, cols, plain.TORCH[dt], cols + gap, lead)
    h = values(rows, cols, dt, rows * 7 + cols)
    x.t.copy_(h)
    q, e = Framed(rows, cols, torch.uint8, lead=lead), \
        Framed(rows, -(-cols // 32), torch.uint8, lead=lead)
    back = Framed(rows, cols, plain.TORCH[dt], cols + gap, lead)
    zs.zero_act_save(q.t, e.t, x.t)
    zs.zero_act_load(back.t, q.t, e.t)
    torch.cuda.synchronize()
    want_q, want_e = plain.encode(plain.f64(h), dt)
    got_q, got_e = q.t.cpu().numpy(), e.t.cpu().numpy()
    nan = (want_q & 127) == 127
    assert np.array_equal(got_e, want_e)
    assert np.array_equal(got_q[~nan], want_q[~nan]) and np.all((got_q[nan] & 127) == 127)
    assert bits_equal(back.t, plain.decode(want_q, want_e))
    for f in (x, q, e, back):
        assert f.intact()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_every_value_of_the_format(dt):
    # all 2^16 bit patterns, each alone in its block and all together in order
    allv = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(plain.TORCH[dt])
    for x in (allv.view(2048, 32), torch.cat([allv.view(-1, 1),
                                              torch.zeros(65536, 31, dtype=allv.dtype)], 1)):
        d = x.to(DEV)
        q = torch.empty(d.shape, dtype=torch.uint8, device=DEV)
        e = torch.empty((d.shape[0], 1), dtype=torch.uint8, device=DEV)
        back = torch.empty_like(d)
        zs.zero_act_save(q, e, d)
        zs.zero_act_load(back, q, e)
        want_q, want_e = plain.encode(plain.f64(x), dt)
        nan = (want_q & 127) == 127
        assert np.array_equal(e.cpu().numpy(), want_e)
        assert np.array_equal(q.cpu().numpy()[~nan], want_q[~nan])
        assert bits_equal(back, plain.decode(want_q, want_e))


def test_reading_into_another_format_rounds_once():
    x = values(40, 96, "f32", 9, rare=False)
    x[0, :32] *= 2.0 ** 20          # past FP16's range
    x[1, :32] *= 2.0 ** -30         # FP16 subnormals
    q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    e = torch.empty((40, 3), dtype=torch.uint8, device=DEV)
    zs.zero_act_save(q, e, x.to(DEV))
    v = torch.from_numpy(plain.decode(q.cpu().numpy(), e.cpu().numpy()))
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        out = torch.empty(x.shape, dtype=dt, device=DEV)
        zs.zero_act_load(out, q, e)
        assert torch.equal(out.cpu(), v.to(dt))


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols,gap,lead", [(1, 1, 0, 0), (3, 32, 0, 0), (5, 33, 0, 1),
                                                (16, 200, 8, 3), (64, 1024, 0, 0),
                                                (9, 2050, 1, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_activation_forward_and_backward(rows, cols, gap, lead, dt, act, in_place):
    td = plain.TORCH[dt]
    h = values(rows, cols, dt, rows + cols, rare=False)
    h[0, 0] = 11.0
    h[-1, -1] = -60.0
    x = Framed(rows, cols, td, cols + gap, lead)
    x.t.copy_(h)
    y = x if in_place else Framed(rows, cols, td, cols + 2 * gap, lead)
    q = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    e = torch.empty((rows, -(-cols // 32)), dtype=torch.uint8, device=DEV)
    zs.zero_act_save(q, e, x.t, act=ACTS[act], y=y.t)
    want_q, want_e = plain.encode(plain.f64(h), dt)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(e.cpu().numpy(), want_e)
    val, bound = plain.act(plain.f64(h), act)
    err = np.abs(plain.f64(y.t) - val)
    tol = plain.rounded(val, bound, dt)
    assert np.all(err <= tol), (err / tol).max()

    g = torch.Generator().manual_seed(rows)
    hdy = torch.randn(rows, cols, generator=g).to(td)
    dy = Framed(rows, cols, td, cols + gap, lead)
    dy.t.copy_(hdy)
    dx = dy if in_place else Framed(rows, cols, td, cols, lead + 1)
    zs.zero_act_backward(dx.t, dy.t, q, e, ACTS[act])
    slope, sb = plain.act_slope(plain.decode(want_q, want_e), act)
    d = plain.f64(hdy)
    err = np.abs(plain.f64(dx.t) - d * slope)
    tol = plain.rounded(d * slope, np.abs(d) * sb * (1 + 2 * plain.U) +
                        np.abs(d * slope) * plain.U, dt)
    assert np.all(err <= tol), (err / tol).max()
    log(f"  {act} {dt} {rows}x{cols}: worst {float((err / tol).max()):.2f} of the bound")
    for f in (x, y, dy, dx):
        assert f.intact()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_slope_against_differences(act):
    # the backward pass at the checkpoint's own values against differences of the forward
    # definition (FP64): second order in h, so h^2 times a third derivative below 2
    x = torch.linspace(-9, 9, 4096).view(64, 64)
    q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    e = torch.empty((64, 2), dtype=torch.uint8, device=DEV)
    zs.zero_act_save(q, e, x.to(DEV))
    dx = torch.empty(64, 64, device=DEV)
    zs.zero_act_backward(dx, torch.ones(64, 64, device=DEV), q, e, ACTS[act])
    v = plain.decode(q.cpu().numpy(), e.cpu().numpy())
    h = 1e-4
    diff = (plain.act(v + h, act)[0] - plain.act(v - h, act)[0]) / (2 * h)
    _, bound = plain.act_slope(v, act)
    assert np.all(np.abs(plain.f64(dx) - diff) <= bound + 2 * h * h + 1e-11)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_infinite_and_nan_activations_stay_visible(act):
    x = torch.zeros(2, 64)
    x[0, 3], x[0, 40], x[1, 5] = float("inf"), float("nan"), -float("inf")
    x[1, 40] = 3e38
    d = x.to(DEV)
    q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    e = torch.empty((2, 2), dtype=torch.uint8, device=DEV)
    y, dx = torch.empty_like(d), torch.empty_like(d)
    zs.zero_act_save(q, e, d, act=ACTS[act], y=y)
    zs.zero_act_backward(dx, torch.ones_like(d), q, e, ACTS[act])
    bad = ~torch.isfinite(x)
    assert torch.equal(~torch.isfinite(y.cpu()), bad)
    assert torch.equal(torch.isnan(dx.cpu()), bad)      # kept as NaN in 8 bits
    assert y[1, 40].item() == float(np.float32(3e38)) and dx[1, 40].item() == 1.0


def test_views_of_one_buffer_may_interleave():
    # gate and up halves of one buffer: x the left columns, y the right ones
    buf = torch.randn(17, 128, device=DEV)
    x, y = buf[:, :64], buf[:, 64:]
    h = x.cpu().clone()
    q = torch.empty(17, 64, dtype=torch.uint8, device=DEV)
    e = torch.empty(17, 2, dtype=torch.uint8, device=DEV)
    zs.zero_act_save(q, e, x, act=zs.ACT_SILU, y=y)
    val, bound = plain.act(plain.f64(h), "silu")
    assert np.all(np.abs(plain.f64(y) - val) <= plain.rounded(val, bound, "f32"))
    assert torch.equal(x.cpu(), h)
    with pytest.raises(zs.ZeroError):
        zs.zero_act_save(q, e, x, act=zs.ACT_SILU, y=buf[:, 63:127])


@pytest.mark.parametrize("cap", [1, 3])
def test_grid_loops_under_a_lowered_cap(cap):
    h = values(200, 777, "bf16", 4, rare=False)
    d = h.to(DEV)
    q = torch.empty(h.shape, dtype=torch.uint8, device=DEV)
    e = torch.empty((200, 25), dtype=torch.uint8, device=DEV)
    back = torch.empty_like(d)
    zs.zero_set_grid_cap(cap)
    try:
        zs.zero_act_save(q, e, d)
        zs.zero_act_load(back, q, e)
    finally:
        zs.zero_set_grid_cap(0)
    wq, we = plain.encode(plain.f64(h), "bf16")
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(e.cpu().numpy(), we)
    assert bits_equal(back, plain.decode(wq, we))


def test_a_matrix_past_4_gib():
    # element and byte offsets past 2^32: the last rows of a 9 GiB FP32 matrix
    rows, cols = 36_000, 65_536 + 32
    x = torch.empty(rows, cols, device=DEV)
    x[:-2] = 0.5
    tail = values(2, cols, "f32", 77, rare=False)
    x[-2:] = tail.to(DEV)
    q = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    e = torch.empty((rows, cols // 32), dtype=torch.uint8, device=DEV)
    zs.zero_act_save(q, e, x)
    wq, we = plain.encode(plain.f64(tail), "f32")
    assert np.array_equal(q[-2:].cpu().numpy(), wq) and np.array_equal(e[-2:].cpu().numpy(), we)
    assert bool((q[:-2] == q[0, 0]).all()) and bool((e[:-2] == e[0, 0]).all())
    zs.zero_act_load(x, q, e)
    assert bits_equal(x[-2:], plain.decode(wq, we)) and bool((x[:-2] == 0.5).all())
