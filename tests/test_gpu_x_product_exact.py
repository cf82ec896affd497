"""The product's FP32 results where the exact sum is known to be a number of FP32: codes that
are small whole numbers, scales that change along a row in opposite directions on both sides,
so that every product is a whole number of one quantum, and sums of magnitudes below 2^24
quanta.  Whatever the order of its additions, an FP32 sum of exact products is then exact, and
results have to equal the FP64 product bit for bit: operands rounded anywhere, or parts of a
group of products dropped, would show."""
import pytest
import torch

import zero_sharded_mixed_shard_amd as zs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def u8(*shape, fill=171):
    return torch.full(shape, fill, dtype=torch.uint8, device=DEV)


def as_codes(x):
    """Codes of values that e4m3 holds."""
    q = x.to(torch.float8_e4m3fn)
    assert torch.equal(q.double(), x.double())
    return q.view(torch.uint8)


def values(q, e, block, tall):
    rows, cols = q.shape
    k = (e.double() - 127.0).repeat_interleave(block, 1)[:, :cols]
    k = k.repeat_interleave(tall, 0)[:rows]
    return q.view(torch.float8_e4m3fn).double() * torch.exp2(k)


def check(qa, ea, qb, eb, a_block, quantum):
    """The FP32 product equals the FP64 one, which is exact, bit for bit."""
    (m, k), n = qa.shape, qb.shape[0]
    a, b = values(qa, ea, a_block, 1), values(qb, eb, 128, 128)
    want, mag = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    assert float(mag.max()) < 2.0 ** 24 * quantum
    for cap in (0, 5):                  # 5: a workgroup's tiles one after another
        y = torch.full((m, n), 99.0, device=DEV)
        zs.zero_set_grid_cap(cap)
        try:
            zs.zero_block_product(y, qa, ea, qb, eb,
                                  workspace=u8(zs.zero_block_product_workspace(m, n, k)))
        finally:
            zs.zero_set_grid_cap(0)
        assert torch.equal(y.double(), want)


# 64 x 64 tiles, whole and in splits (the third, fourth and fifth), 128 x 128 ones, whole and
# in splits (the eighth), 256 x 256 ones; too short for tiles; whole blocks and ragged ends
SHAPES = [(3, 5, 11), (5, 40, 300), (7, 200, 4096), (65, 150, 4097), (130, 70, 1000),
          (1000, 1030, 2100), (2300, 2300, 300), (1024, 1024, 8192), (2048, 2048, 1024),
          (4096, 4096, 512), (3000, 4096, 1000)]


@pytest.mark.parametrize("a_block", [128, 32])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_sums_of_whole_numbers_are_exact(m, n, k, a_block):
    g = torch.Generator(device="cuda").manual_seed(m + n + k + a_block)
    pick = lambda shape, *v: torch.tensor(v, device=DEV)[
        torch.randint(len(v), shape, generator=g, device=DEV)]
    # one column of sixteen holds products of up to 2^14, the others of up to 6: a part below
    # 2^-13 of the largest
    a, b = pick((m, k), -2.0, -1.0, 0.0, 1.0, 2.0), pick((n, k), -3.0, -1.0, 1.0, 3.0)
    turn = torch.arange(k, device=DEV)
    large = turn % 16 == torch.randint(16, (1,), generator=g, device=DEV)
    few = large & (turn // 16 % 2 == 0)
    a = torch.where(large, pick((m, k), -120.0, 120.0, 104.0), a)
    b = torch.where(large, pick((n, k), 120.0, -104.0, 56.0), b)
    a = torch.where(few, pick((m, k), 448.0, -288.0, 256.0), a)      # past half the range
    b = torch.where(few, pick((n, k), 36.0, -32.0, 1.0), b)
    d = torch.randint(-122, 123, (-(-k // 128),), generator=g, device=DEV)
    d[0], d[-1] = 122, -122                                          # both ends on both sides
    ea = (125 + d).expand(m, -1)
    if a_block == 32:
        ea = ea.repeat_interleave(4, 1)[:, :-(-k // 32)]
    eb = (125 - d).expand(-(-n // 128), -1)
    check(as_codes(a), ea.to(torch.uint8).contiguous(), as_codes(b),
          eb.to(torch.uint8).contiguous(), a_block, 2.0 ** -4)


@pytest.mark.parametrize("a_block", [128, 32])
@pytest.mark.parametrize("m,n,k", [(2, 3, 12), (5, 40, 300), (65, 150, 4097), (2300, 2300, 300),
                                   (3000, 4096, 640)])
def test_the_smallest_numbers_against_the_largest(m, n, k, a_block):
    # blocks whose exponent byte is 3 and whose codes are below the format's normal numbers (whole
    # numbers of 2^-133), against blocks of byte 247 and codes up to 448; even blocks have the
    # small side in a, odd ones in b
    g = torch.Generator(device="cuda").manual_seed(m + n + k + a_block)
    sign = lambda shape: (torch.randint(2, shape, generator=g, device=DEV) * 128).to(torch.uint8)
    small = lambda rows: (torch.randint(8, (rows, k), generator=g, device=DEV) * 2 +
                          1).to(torch.uint8) | sign((rows, k))
    big = lambda rows: as_codes(torch.tensor(
        [1.0, -3.0, 7.0, 30.0, 448.0, -256.0], device=DEV)[torch.randint(
            6, (rows, k), generator=g, device=DEV)])
    nb = -(-k // 128)
    even = torch.arange(nb, device=DEV) % 2 == 0
    cols = even.repeat_interleave(128)[:k]
    qa = torch.where(cols, small(m), big(m))
    qb = torch.where(cols, big(n), small(n))
    ea = torch.where(even, 3, 247).to(torch.uint8).expand(m, -1).clone()
    eb = torch.where(even, 247, 3).to(torch.uint8).expand(-(-n // 128), -1).clone()
    # rows of a whose first block has the largest scale as well: its only code that is not zero
    # meets zeros of b, so that the block adds nothing (and no infinity)
    qa[1::3, :128] = 0
    qa[1::3, 1] = 0x7e
    qb[:, 1] = 0
    ea[1::3, 0] = 247
    if a_block == 32:
        ea = ea.repeat_interleave(4, 1)[:, :-(-k // 32)].contiguous()
    check(qa, ea, qb, eb, a_block, 2.0 ** -13)


def test_rows_of_the_largest_scale_on_both_sides():
    # byte 247 on either side and on both (there a's codes are zeros: an infinity made of b's
    # would give NaN), in some rows of a tile and not in others
    m, n, k = 70, 260, 640
    g = torch.Generator(device="cuda").manual_seed(9)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g, device=DEV).float()
    a, b = whole(m, k), whole(n, k)
    a[:, ::32], b[:, 5::32] = 448.0, 288.0
    a[:, 512:] = 0.0
    ea = torch.tensor([247, 10, 127, 247, 247], device=DEV).expand(m, -1).clone()
    eb = torch.tensor([10, 247, 130, 10, 247], device=DEV).expand(3, -1).clone()
    ea[::2, 3], ea[::4, 0] = 246, 245
    check(as_codes(a), ea.to(torch.uint8), as_codes(b), eb.to(torch.uint8), 128, 8.0 / 4)


def test_more_columns_than_fp32_counts():
    # 2^24 + 2^21 + 1 products of 1: adding them to one FP32 number stops at 2^24
    k = 2 ** 24 + 2 ** 21 + 1
    q = u8(2, k, fill=0x38)
    e = u8(2, -(-k // 128), fill=127)
    for dt in (torch.float32, torch.bfloat16):
        y = torch.zeros(1, 1, dtype=dt, device=DEV)
        zs.zero_block_product(y, q[:1], e[:1], q[1:], e[1:])
        assert float(y) == float(torch.tensor(float(k)).to(dt))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("a_block", [128, 32])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_16_bit_results_lose_nothing_of_products_of_like_size(m, n, k, a_block, dt):
    # whole products of 1 to 2^12: none has a part below 2^-13 of another, so that the 8-bit
    # instruction's sums are exact as well and the one rounding is all that is left
    g = torch.Generator(device="cuda").manual_seed(m + n + k + a_block)
    pick = lambda shape, *v: torch.tensor(v, device=DEV)[
        torch.randint(len(v), shape, generator=g, device=DEV)]
    a = pick((m, k), -3.0, -2.0, -1.0, 1.0, 5.0, 13.0, 64.0, -60.0, 0.0)
    b = pick((n, k), -7.0, -3.0, -1.0, 1.0, 2.0, 15.0, -64.0, 48.0)
    d = torch.randint(-110, 111, (-(-k // 128),), generator=g, device=DEV)
    ea = (121 + d).expand(m, -1)        # quanta of 2^-12, results within FP16's range
    if a_block == 32:
        ea = ea.repeat_interleave(4, 1)[:, :-(-k // 32)]
    ea = ea.to(torch.uint8).contiguous()
    eb = (121 - d).expand(-(-n // 128), -1).to(torch.uint8).contiguous()
    qa, qb = as_codes(a), as_codes(b)
    av, bv = values(qa, ea, a_block, 1), values(qb, eb, 128, 128)
    want, mag = av @ bv.t().contiguous(), av.abs() @ bv.abs().t().contiguous()
    assert float(mag.max()) < 2.0 ** 24 * 2.0 ** -12
    y = torch.full((m, n), 99.0, device=DEV, dtype=dt)
    zs.zero_block_product(y, qa, ea, qb, eb,
                          workspace=u8(zs.zero_block_product_workspace(m, n, k)))
    assert torch.equal(y, want.float().to(dt))
