"""The product in its largest tiles: extents for which 256 x 256 tiles are chosen (sixteen by
sixteen of them and many steps), whole and ragged, both blocks of a, a workgroup's tiles one
after another, against FP64 on the device."""
import pytest
import torch

import zero_sharded_mixed_shard_amd as zs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device=DEV)


def values(q, e, block, tall):
    rows, cols = q.shape
    k = (e.double() - 127.0).repeat_interleave(block, 1)[:, :cols]
    k = k.repeat_interleave(tall, 0)[:rows]
    return q.view(torch.float8_e4m3fn).double() * torch.exp2(k)


def operands(m, n, k, a_block, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn(m, k, generator=g, device=DEV)
    a *= torch.exp2(torch.randint(-6, 6, (m, 1), generator=g, device=DEV).float())
    b = torch.randn(n, k, generator=g, device=DEV)
    qa, ea = u8(m, k), u8(m, -(-k // a_block))
    if a_block == 32:
        zs.zero_act_save(qa, ea, a.bfloat16())
    else:
        zs.zero_block_quant(qa, ea, a)
    qb, eb = u8(n, k), u8(-(-n // 128), -(-k // 128))
    zs.zero_block_quant(qb, eb, b, square=True)
    return qa, ea, qb, eb


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 4096), (4090, 4081, 4090), (4083, 4096, 4161)])
@pytest.mark.parametrize("dt,a_block", [("bf16", 128), ("f16", 32), ("f32", 128), ("f32", 32)])
def test_large_tiles(m, n, k, dt, a_block):
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dt]
    ops = operands(m, n, k, a_block, m + k)
    if dt == "f16":
        ops[1].clamp_(max=118)          # within FP16's range
    a, b = values(ops[0], ops[1], a_block, 1), values(ops[2], ops[3], 128, 128)
    want, mag = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    # as for the small products: k FP32 additions in any order, each off by a step at most, and
    # for 16-bit results 2^-10 of the magnitudes and one rounding
    bound = mag * (k * 2.0 ** -23)
    if dt != "f32":
        bound = bound + mag * 2.0 ** -10
        half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -11
        bound = bound + (want.abs() + bound) * half + 2.0 ** -25
    else:
        bound = bound + want.abs() * 2.0 ** -24 + 2.0 ** -126
    buf = torch.full((m * (n + 5) + 1,), 77.0, device=DEV).to(dtype)
    y = buf[1:].view(m, n + 5)[:, :n]
    ws = u8(zs.zero_block_product_workspace(m, n, k))
    zs.zero_block_product(y, *ops, workspace=ws)
    assert bool(((y.double() - want).abs() <= bound).all())
    assert bool((buf[1:].view(m, n + 5)[:, n:] == 77).all()) and float(buf[0]) == 77
    again = torch.empty(m, n, dtype=dtype, device=DEV)
    zs.zero_set_grid_cap(7)             # some forty tiles a workgroup
    try:
        zs.zero_block_product(again, *ops, workspace=ws)
    finally:
        zs.zero_set_grid_cap(0)
    assert torch.equal(again, y)
