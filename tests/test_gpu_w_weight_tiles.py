"""Every tile of the weight gradient, through its whole loop, on the GPU.

The extents are such that the launcher takes each tile with and without split tokens, in every
grouping of tiles, over even and odd numbers of steps past the loop's steady part, with ragged
tokens, rows and columns (test_weight_plan_cpu.py checks that they still do).  Whole numbers:
every product and partial sum is exact in FP32, so results equal the FP64 product to the bit.
"""
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs
from test_gpu_o_act import Framed
from test_gpu_p_weight_grad import space

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

# tokens, n_out, n_in
SHAPES = [
    # 256 x 256 tiles: ungrouped, grouped four and eight and one wide, split tokens, whole tiles
    (335, 8922, 1306), (266, 1419, 8702), (323, 5934, 5046), (261, 5982, 4857), (329, 7957, 1834),
    (311, 8025, 1863), (779, 4082, 3902), (513, 8192, 4096), (640, 8192, 4096), (387, 65_327, 141),
    (701, 5414, 2346), (2194, 6582, 599),
    # 128 x 128 tiles
    (342, 3742, 561), (264, 780, 2987), (501, 5854, 1222), (317, 4772, 1453), (484, 4081, 970),
    (404, 899, 3971), (279, 60_983, 67), (384, 2048, 1152), (835, 8030, 4101), (1506, 709, 1436),
    # 64 x 64 tiles
    (721, 615, 558), (593, 541, 517), (927, 2907, 632), (792, 2431, 755), (786, 504, 2005),
    (2582, 609, 505), (517, 30_915, 20), (512, 2048, 1024)]


def whole(rows, cols, top, g):
    return torch.randint(-top, top + 1, (rows, cols), generator=g, device=DEV).float()


def checkpoint(x):
    q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
    e = torch.empty((x.shape[0], -(-x.shape[1] // 32)), dtype=torch.uint8, device=DEV)
    zs.zero_act_save(q, e, x)
    return q, e


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,n_out,n_in", SHAPES)
def test_whole_numbers_through_every_tile(tokens, n_out, n_in, dt):
    td = plain.TORCH[dt]
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens + n_out)
    hdy = whole(tokens, n_out, 4, g)
    dy = Framed(tokens, n_out, td, n_out + n_out % 3, lead=n_in % 5)
    dy.t.copy_(hdy)
    # blocks of several scales, each whole times a power of two: four bits, so held exactly
    scale = torch.exp2(torch.randint(0, 4, (tokens, -(-n_in // 32)), generator=g,
                                     device=DEV).float()).repeat_interleave(32, 1)[:, :n_in]
    x = whole(tokens, n_in, 4, g) * scale
    q, e = checkpoint(x.to(td))
    want = hdy.double().t().contiguous() @ x.double()
    ws = space(tokens, n_out, n_in)
    for out_dt in (td, torch.float32):
        dw = Framed(n_out, n_in, out_dt, lead=n_in % 7)
        zs.zero_weight_grad(dw.t, dy.t, q, e, workspace=ws)
        assert torch.equal(dw.t, want.float().to(out_dt))
        if out_dt == torch.float32:
            base = whole(n_out, n_in, 1000, g)
            dw.t.copy_(base)
            zs.zero_weight_grad(dw.t, dy.t, q, e, first=False, workspace=ws)
            assert torch.equal(dw.t.double(), base.double() + want)
        assert dw.intact()
    assert dy.intact()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,n_out,n_in", [(779, 4082, 3902), (2194, 6582, 599),
                                               (501, 5854, 1222)])
def test_the_three_results_are_one_sum(tokens, n_out, n_in, dt):
    # random inputs: the same FP32 sums whatever the result's form, repeated bit for bit, and
    # within the bound of one addition a token
    td = plain.TORCH[dt]
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    dy = torch.randn(tokens, n_out, generator=g, device=DEV).to(td)
    x = torch.randn(tokens, n_in, generator=g, device=DEV).to(td)
    q, e = checkpoint(x)
    v = torch.empty(tokens, n_in, device=DEV)
    zs.zero_act_load(v, q, e)
    ws = space(tokens, n_out, n_in)
    d32, again = torch.empty(n_out, n_in, device=DEV), torch.empty(n_out, n_in, device=DEV)
    d16 = torch.empty(n_out, n_in, dtype=td, device=DEV)
    zs.zero_weight_grad(d32, dy, q, e, workspace=ws)
    ws.fill_(1)
    zs.zero_weight_grad(again, dy, q, e, workspace=ws)
    zs.zero_weight_grad(d16, dy, q, e, workspace=ws)
    assert torch.equal(d32, again) and torch.equal(d16, d32.to(td))
    base = torch.randn(n_out, n_in, generator=g, device=DEV)
    acc = base.clone()
    zs.zero_weight_grad(acc, dy, q, e, first=False, workspace=ws)
    assert torch.equal(acc, base + d32)
    dyt, vd = dy.double().t().contiguous(), v.double()
    bound = (dyt.abs() @ vd.abs()) * (tokens * 2 * plain.U)
    assert bool(((d32.double() - dyt @ vd).abs() <= bound).all())
