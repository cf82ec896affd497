"""Matrices in 8-bit codes with a power of two for each block of 128, on the GPU: codes,
exponents and the values read back equal the 64-bit definition exactly; the product is
within its derived bound."""
import numpy as np
import pytest
import torch

import block_plain as plain
import grad_plain
import zero_sharded_mixed_shard_amd as zs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TORCH = grad_plain.TORCH


def place(t, ld=0, off=1):
    """t on the device at an odd place of a larger buffer, with row stride t.shape[1] + ld;
    the gaps hold a value that must stay."""
    rows, cols = t.shape
    w = cols + ld
    buf = torch.full((off + rows * w + 3,), 77, dtype=t.dtype, device=DEV)
    v = buf[off:off + rows * w].view(rows, w)[:, :cols]
    v.copy_(t)
    return buf, v


def untouched(buf, view, off=1):
    rest = buf.clone()
    rows, cols = view.shape
    if rows and cols:
        rest[off:off + rows * view.stride(0)].view(rows, -1)[:, :cols] = 77
    return bool((rest == 77).all())


def hidden(rows, cols, dt, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(
        torch.randint(-8, 4, (rows, 1), generator=g) * spread / 3)
    return x.to(TORCH[dt])


def u8(*shape, fill=171):
    return torch.full(shape, fill, dtype=torch.uint8, device=DEV)


SHAPES = [(1, 1), (1, 128), (3, 7), (2, 127), (5, 129), (127, 1601), (128, 128), (129, 256),
          (300, 260), (64, 1000)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("square", [False, True])
def test_codes_exact(dt, rows, cols, square):
    x = hidden(rows, cols, dt, rows * 7 + cols)
    flat = x.view(-1)
    if rows * cols > 300:               # what a code cannot hold, and the ends of the formats
        big = torch.finfo(TORCH[dt]).max
        for i, v in enumerate((float("inf"), float("-inf"), float("nan"), big, -big,
                               torch.finfo(TORCH[dt]).smallest_normal, 0.0, -0.0)):
            flat[(i * 61 + 5) % flat.numel()] = v
    for ld, off in ((0, 0), (3, 1)):
        buf, v = place(x, ld, off)
        tall = 128 if square else 1
        q, e = u8(rows, cols), u8(-(-rows // tall), -(-cols // 128))
        extra = {}
        if square:
            extra = dict(qt=u8(cols, rows), et=u8(-(-cols // 128), -(-rows // 128)))
        zs.zero_block_quant(q, e, v, square=square, **extra)
        wq, we = plain.encode(grad_plain.f64(x), dt, tall)
        nan = (wq & 127) == 127
        got = q.cpu().numpy()
        assert np.array_equal(got[~nan], wq[~nan]) and np.all((got[nan] & 127) == 127)
        assert np.array_equal(e.cpu().numpy(), we)
        if square:
            assert torch.equal(extra["qt"], q.t()) and torch.equal(extra["et"], e.t())
            q2, e2 = u8(rows, cols), u8(*e.shape)
            zs.zero_block_quant(q2, e2, v, square=True)
            assert torch.equal(q2, q) and torch.equal(e2, e)
        obuf, back = place(torch.zeros_like(x), ld, off)
        zs.zero_block_load(back, q, e, square=square)
        want = torch.from_numpy(plain.decode(wq, we, tall)).to(TORCH[dt])
        assert torch.equal(back.cpu().nan_to_num(7.0), want.nan_to_num(7.0))
        assert torch.equal(back.cpu().isnan(), want.isnan())
        assert untouched(obuf, back, off) and untouched(buf, v, off)


def test_every_code_border_rounds_to_even():
    # one block whose scale is 1, with all codes' values and the borders between them
    v = np.concatenate([plain.CODE_VALUES[:127], plain._MID])
    v = np.concatenate([v, -v])
    x = np.zeros((len(v), 128))
    x[:, 3], x[:, 0] = v, 448.0
    t = torch.from_numpy(x).to(DEV, torch.float32)
    q, e = u8(*t.shape), u8(len(v), 1)
    zs.zero_block_quant(q, e, t)
    wq, we = plain.encode(x, "f32")
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(e.cpu().numpy(), we)


def test_many_blocks_with_a_small_grid():
    x = hidden(700, 900, "bf16", 3)
    tens = x.to(DEV)
    want = [u8(700, 900), u8(700, 8), u8(700, 900), u8(6, 8), u8(900, 700), u8(8, 6)]
    got = [t.clone() for t in want]
    for out, cap in ((want, 0), (got, 3)):
        zs.zero_set_grid_cap(cap)
        try:
            zs.zero_block_quant(out[0], out[1], tens)
            zs.zero_block_quant(out[2], out[3], tens, square=True, qt=out[4], et=out[5])
            back = torch.zeros_like(tens)
            zs.zero_block_load(back, out[2], out[3], square=True)
        finally:
            zs.zero_set_grid_cap(0)
        out.append(back)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


# ---- the product ---------------------------------------------------------------------------

def coded(rows, cols, dt, seed, tall, block=128):
    x = hidden(rows, cols, dt, seed).double().numpy()
    q, e = plain.encode(x, dt, tall, block)
    return (torch.from_numpy(q).to(DEV), torch.from_numpy(e).to(DEV),
            plain.decode(q, e, tall, block))


def multiply(m, n, k, dt, a_block, seed=1, ld=0, off=1):
    src = "bf16" if dt == "f32" else dt
    qa, ea, a = coded(m, k, src, seed, 1, a_block)
    qb, eb, b = coded(n, k, src, seed + 1, 128)
    buf, y = place(torch.zeros(m, n, dtype=TORCH[dt]), ld, off)
    ws = u8(zs.zero_block_product_workspace(m, n, k))
    zs.zero_block_product(y, qa, ea, qb, eb, workspace=ws)
    want, bound = plain.product(a, b, dt)
    assert np.all(np.abs(grad_plain.f64(y) - want) <= bound)
    assert untouched(buf, y, off)
    return y


# one row to many; rows, columns and lengths around every tile's and wave's edge; lengths
# below, at and past a block; odd lengths, whose rows start at any byte
PRODUCTS = [(1, 1, 1), (1, 5, 3), (3, 2, 15), (1, 17, 16), (2, 33, 17), (1, 64, 128),
            (1, 130, 257), (5, 129, 129), (15, 200, 300), (16, 256, 511), (17, 100, 512),
            (31, 65, 640), (32, 128, 768), (33, 129, 769), (48, 300, 1000), (63, 127, 128),
            (64, 64, 2048), (65, 63, 1025), (100, 400, 96), (127, 255, 384), (128, 128, 128),
            (129, 257, 255), (200, 50, 3333), (255, 256, 130), (256, 256, 512), (257, 300, 769),
            (300, 520, 1100), (512, 512, 256), (700, 33, 48)]


@pytest.mark.parametrize("dt,a_block", [("f16", 128), ("bf16", 32), ("f32", 128), ("f32", 32)])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k, dt, a_block):
    multiply(m, n, k, dt, a_block, ld=(m + n) % 3 * 5, off=m % 2)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_product_of_large_extents(dt):
    multiply(1023, 1537, 768, dt, 32)
    multiply(2050, 770, 1664, dt, 128)


def test_product_repeats_bit_for_bit():
    for m, n, k in ((7, 2000, 4096), (300, 300, 4000), (600, 900, 700)):
        a, b = (multiply(m, n, k, "bf16", 128) for _ in range(2))
        assert torch.equal(a, b)


def test_product_of_a_checkpoint():
    # the layer's input as zero_act_save keeps it for the weight gradient
    x = hidden(130, 300, "bf16", 5).to(DEV)
    q, e = u8(130, 300), u8(130, 10)
    zs.zero_act_save(q, e, x)
    w = hidden(70, 300, "bf16", 6).to(DEV)
    qw, ew = u8(70, 300), u8(1, 3)
    zs.zero_block_quant(qw, ew, w, square=True)
    y = torch.zeros(130, 70, device=DEV)
    ws = u8(zs.zero_block_product_workspace(130, 70, 300))
    zs.zero_block_product(y, q, e, qw, ew, workspace=ws)
    a = plain.decode(q.cpu().numpy(), e.cpu().numpy(), 1, 32)
    b = plain.decode(qw.cpu().numpy(), ew.cpu().numpy(), 128)
    want, bound = plain.product(a, b, "f32")
    assert np.all(np.abs(grad_plain.f64(y) - want) <= bound)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(3, 40, 200), (40, 140, 200), (300, 300, 200)])
def test_product_nan_stays_in_its_row_and_column(m, n, k, dt):
    qa, ea, _ = coded(m, k, "bf16", 1, 1)
    qb, eb, _ = coded(n, k, "bf16", 2, 128)
    qa[m - 1, 5] = 127
    qb[n - 2, k - 1] = 255
    y = torch.zeros(m, n, dtype=TORCH[dt], device=DEV)
    zs.zero_block_product(y, qa, ea, qb, eb,
                          workspace=u8(zs.zero_block_product_workspace(m, n, k)))
    nan = torch.zeros(m, n, dtype=torch.bool)
    nan[m - 1, :] = True
    nan[:, n - 2] = True
    assert torch.equal(y.isnan().cpu(), nan)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m", [2, 40, 300])
def test_product_scales_of_the_whole_range(m, dt):
    # exponent bytes 3 and 247 in one row: huge times tiny is an ordinary number
    n, k = 150, 384
    qa, ea, _ = coded(m, k, "bf16", 3, 1)
    qb, eb, _ = coded(n, k, "bf16", 4, 128)
    ea[:, 0], ea[:, 1], ea[:, 2] = 247, 3, 127
    eb[:, 0], eb[:, 1], eb[:, 2] = 7, 247, 127
    a = plain.decode(qa.cpu().numpy(), ea.cpu().numpy())
    b = plain.decode(qb.cpu().numpy(), eb.cpu().numpy(), 128)
    y = torch.zeros(m, n, dtype=TORCH[dt], device=DEV)
    zs.zero_block_product(y, qa, ea, qb, eb,
                          workspace=u8(zs.zero_block_product_workspace(m, n, k)))
    want, bound = plain.product(a, b, dt)
    assert np.all(np.abs(grad_plain.f64(y) - want) <= bound)


def test_product_overflows_to_infinity_in_fp16():
    q = torch.full((40, 256), 0x7e, dtype=torch.uint8, device=DEV)     # 448
    e = u8(40, 2, fill=127)
    y = torch.zeros(40, 40, dtype=torch.float16, device=DEV)
    zs.zero_block_product(y, q, e, q, u8(1, 2, fill=127),
                          workspace=u8(zs.zero_block_product_workspace(40, 40, 256)))
    assert bool(torch.isposinf(y).all())


def test_product_of_no_columns_is_zero():
    for dt in ("f16", "f32"):
        buf, y = place(torch.ones(5, 9, dtype=TORCH[dt]), 4)
        zs.zero_block_product(y, u8(5, 0), u8(5, 0), u8(9, 0), u8(1, 0))
        assert bool((y == 0).all()) and untouched(buf, y)


def test_binding_refusals_on_the_device():
    y = torch.zeros(4, 6, device=DEV)
    qa, ea, qb, eb = u8(4, 300), u8(4, 3), u8(6, 300), u8(1, 3)
    for bad in (dict(qa=u8(5, 300)), dict(ea=u8(4, 4)), dict(qb=u8(7, 300)), dict(eb=u8(6, 3)),
                dict(qa=u8(300, 4).t()), dict(y=torch.zeros(6, 4, device=DEV).t())):
        a = dict(y=y, qa=qa, ea=ea, qb=qb, eb=eb)
        a.update(bad)
        with pytest.raises(ValueError):
            zs.zero_block_product(**a)
    x = torch.zeros(4, 300, device=DEV)
    with pytest.raises(ValueError):
        zs.zero_block_quant(u8(4, 300), u8(4, 3), x, qt=u8(300, 4), et=u8(3, 1))
    with pytest.raises(ValueError):
        zs.zero_block_quant(u8(4, 300), u8(1, 3), x, square=True, qt=u8(300, 4))
    with pytest.raises(ValueError):
        zs.zero_block_quant(u8(4, 301), u8(4, 3), x)
    with pytest.raises(ValueError):
        zs.zero_block_load(x, u8(4, 300), u8(4, 3), square=True)
