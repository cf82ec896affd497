"""The weight gradient from an 8-bit checkpoint on the GPU.

With small whole numbers every product and partial sum is exact in FP32, so the
result must equal the 64-bit one to the bit whatever the order of the sums; random
inputs are held to the bound of T FP32 additions.
"""
import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs
from gpu_util import log
from test_gpu_o_act import Framed

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def checkpoint(x, dt):
    q, e = plain.encode(plain.f64(x), dt)
    return torch.from_numpy(q).to(DEV), torch.from_numpy(e).to(DEV)


def whole(rows, cols, seed, top=4):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-top, top + 1, (rows, cols), generator=g).float()


def space(tokens, n_out, n_in):
    return torch.full((zs.zero_weight_grad_workspace(tokens, n_out, n_in) + 16,), 255,
                      dtype=torch.uint8, device=DEV)


# tokens, n_out, n_in: single elements, ragged edges of tiles and steps, split tokens
SHAPES = [(1, 1, 1), (1, 5, 33), (2, 64, 32), (63, 17, 100), (64, 128, 128), (65, 129, 127),
          (130, 256, 256), (200, 300, 520), (777, 96, 31), (1000, 130, 258), (2048, 64, 64),
          (5000, 33, 40), (128, 4100, 4097), (70, 4096, 4224), (4096, 2000, 700),
          (9001, 1030, 770), (12_345, 2304, 768), (300, 9, 8), (300, 8, 1000), (129, 2050, 7)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,n_out,n_in", SHAPES)
def test_whole_numbers_are_exact(tokens, n_out, n_in, dt):
    td = plain.TORCH[dt]
    dy = Framed(tokens, n_out, td, n_out + (n_out % 3), lead=n_in % 5)
    hdy = whole(tokens, n_out, 1)
    dy.t.copy_(hdy)
    # blocks of several scales: whole numbers times a power of two by column block and token
    g = torch.Generator().manual_seed(3)
    hx = whole(tokens, n_in, 2) * torch.exp2(
        torch.randint(0, 4, (tokens, (n_in + 31) // 32), generator=g).float()
    ).repeat_interleave(32, 1)[:, :n_in]
    q, e = checkpoint(hx.to(td), dt)
    want = (hdy.double().t() @ hx.double()).numpy()
    ws = space(tokens, n_out, n_in)
    for out_dt in (td, torch.float32):
        dw = Framed(n_out, n_in, out_dt, lead=n_in % 7)
        zs.zero_weight_grad(dw.t, dy.t, q, e, workspace=ws)
        exp = torch.from_numpy(want).float().to(out_dt)
        assert torch.equal(dw.t.cpu(), exp)
        if out_dt == torch.float32:
            zs.zero_weight_grad(dw.t, dy.t, q, e, first=False, workspace=ws)
            assert np.array_equal(plain.f64(dw.t), 2 * want)
        assert dw.intact()
    assert dy.intact()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,n_out,n_in", [(300, 200, 170), (4099, 70, 200), (513, 700, 900)])
def test_random_inputs_within_the_sum_bound(tokens, n_out, n_in, dt):
    td = plain.TORCH[dt]
    g = torch.Generator().manual_seed(tokens)
    hdy = torch.randn(tokens, n_out, generator=g).to(td)
    hx = (torch.randn(tokens, n_in, generator=g) *
          torch.exp2(torch.randint(-9, 5, (tokens, 1), generator=g).float())).to(td)
    q, e = checkpoint(hx, dt)
    v = plain.decode(*plain.encode(plain.f64(hx), dt))
    want, bound = plain.weight_grad(plain.f64(hdy), v)
    base = torch.randn(n_out, n_in, generator=g)
    dy, ws = hdy.to(DEV), space(tokens, n_out, n_in)
    dw = torch.empty(n_out, n_in, device=DEV)
    zs.zero_weight_grad(dw, dy, q, e, workspace=ws)
    err = np.abs(plain.f64(dw) - want)
    assert np.all(err <= bound), (err / bound).max()
    again = torch.empty_like(dw)
    ws.fill_(1)
    zs.zero_weight_grad(again, dy, q, e, workspace=ws)
    assert torch.equal(dw, again)                      # repeatable, whatever the workspace held
    acc = base.to(DEV)
    zs.zero_weight_grad(acc, dy, q, e, first=False, workspace=ws)
    assert torch.equal(acc.cpu(), base + dw.cpu())     # one FP32 addition
    d16 = torch.empty(n_out, n_in, dtype=td, device=DEV)
    zs.zero_weight_grad(d16, dy, q, e, workspace=ws)
    assert torch.equal(d16.cpu(), dw.cpu().to(td))     # the same sum, rounded once
    log(f"  weight grad {dt} {tokens}x{n_out}x{n_in}: worst {float((err / bound).max()):.3f}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_ends_of_the_formats_range(dt):
    # values read back at the format's largest and smallest magnitudes, products exact
    td = plain.TORCH[dt]
    big, small = plain.TOP[dt], 2.0 ** (-24 if dt == "f16" else -133)
    x = torch.zeros(64, 64, dtype=torch.float64)
    x[0, 0], x[1, 40], x[2, 7] = big, small, -small * 3
    dy = torch.zeros(64, 32, dtype=torch.float64)
    dy[0, 0], dy[1, 1], dy[2, 2] = 2.0 ** -10, 1.0, 2.0 ** 3
    q, e = checkpoint(x.to(td), dt)
    dw = torch.empty(32, 64, device=DEV)
    ws = space(64, 32, 64)
    zs.zero_weight_grad(dw, dy.to(td).to(DEV), q, e, workspace=ws)
    want = torch.zeros(32, 64, dtype=torch.float64)
    want[0, 0], want[1, 40], want[2, 7] = big * 2.0 ** -10, small, -small * 24
    if dt == "f16":
        assert torch.equal(dw.cpu().double(), want)
    else:   # BF16 subnormals: the matrix unit may take them as zero (absolute 2^-126)
        assert float((dw.cpu().double() - want).abs().max()) <= 2.0 ** -126 * 8


def test_nan_codes_reach_every_gradient_they_touch():
    x = torch.ones(70, 64, dtype=torch.bfloat16)
    x[66, 33] = float("inf")
    q, e = checkpoint(x, "bf16")
    dy = torch.ones(70, 40, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty(40, 64, device=DEV)
    zs.zero_weight_grad(dw, dy, q, e, workspace=space(70, 40, 64))
    bad = torch.isnan(dw.cpu())
    assert bool(bad[:, 33].all()) and int(bad.sum()) == 40
    assert bool((dw.cpu()[:, :33] == 70).all())


def test_no_tokens():
    for dtype in (torch.bfloat16, torch.float32):
        dw = Framed(5, 40, dtype)
        q = torch.empty(0, 40, dtype=torch.uint8, device=DEV)
        e = torch.empty(0, 2, dtype=torch.uint8, device=DEV)
        dy = torch.empty(0, 5, dtype=torch.bfloat16, device=DEV)
        if dtype == torch.float32:
            zs.zero_weight_grad(dw.t, dy, q, e, first=False)
            assert bool((dw.t == 7.5).all())
        zs.zero_weight_grad(dw.t, dy, q, e)
        assert bool((dw.t == 0).all()) and dw.intact()


def test_grid_loop_under_a_lowered_cap():
    hdy, hx = whole(100, 600, 5), whole(100, 700, 6)
    q, e = checkpoint(hx, "bf16")
    dw = torch.empty(600, 700, device=DEV)
    ws = space(100, 600, 700)
    zs.zero_set_grid_cap(3)
    try:
        zs.zero_weight_grad(dw, hdy.bfloat16().to(DEV), q, e, workspace=ws)
    finally:
        zs.zero_set_grid_cap(0)
    assert torch.equal(dw.cpu().double(), hdy.double().t() @ hx.double())


def test_gradient_against_differences():
    # loss = sum(c * (v W^T)): its gradient in W, exactly linear, by FP64 differences
    g = torch.Generator().manual_seed(8)
    c = torch.randn(50, 24, generator=g).bfloat16()
    q, e = checkpoint(torch.randn(50, 37, generator=g).bfloat16(), "bf16")
    v = plain.decode(q.cpu().numpy(), e.cpu().numpy())
    dw = torch.empty(24, 37, device=DEV)
    zs.zero_weight_grad(dw, c.to(DEV), q, e, workspace=space(50, 24, 37))
    W = torch.randn(24, 37, generator=g, dtype=torch.float64).numpy()
    cd = plain.f64(c)
    loss = lambda w: float((cd * (v @ w.T)).sum())
    _, bound = plain.weight_grad(cd, v)
    for o, i in ((0, 0), (5, 36), (23, 12), (11, 32)):
        up, dn = W.copy(), W.copy()
        up[o, i] += 0.5
        dn[o, i] -= 0.5
        assert abs(loss(up) - loss(dn) - float(dw[o, i])) <= bound[o, i] + 1e-10


def test_row_strides_past_the_offsets_range():
    # rows 2^24 + 16 elements apart (2.2 GB): the element-by-element form takes over
    ld, tokens = (1 << 24) + 16, 70
    buf = torch.zeros(ld * tokens, dtype=torch.bfloat16, device=DEV)
    dy = buf.as_strided((tokens, 40), (ld, 1))
    hdy, hx = whole(tokens, 40, 1), whole(tokens, 100, 2)
    dy.copy_(hdy)
    q, e = checkpoint(hx, "bf16")
    dw = Framed(40, 100, torch.float32)
    zs.zero_weight_grad(dw.t, dy, q, e, workspace=space(tokens, 40, 100))
    assert torch.equal(dw.t.cpu().double(), hdy.double().t() @ hx.double()) and dw.intact()


def test_a_checkpoint_wider_than_the_offsets_range():
    n_in, tokens, n_out = (1 << 24) + 37, 3, 9
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    x = torch.randint(-4, 5, (tokens, n_in), generator=g, device=DEV).bfloat16()
    q = torch.empty(tokens, n_in, dtype=torch.uint8, device=DEV)
    e = torch.empty(tokens, -(-n_in // 32), dtype=torch.uint8, device=DEV)
    zs.zero_act_save(q, e, x)
    dy = whole(tokens, n_out, 3).bfloat16().to(DEV)
    dw = torch.empty(n_out, n_in, device=DEV)
    zs.zero_weight_grad(dw, dy, q, e, workspace=space(tokens, n_out, n_in))
    want = sum(dy[t].float()[:, None] * x[t].float()[None, :] for t in range(tokens))
    assert torch.equal(dw, want)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gradients_past_4_gib(dt):
    # dw of 5.2 GB of FP32: offsets past 2^32 in its last rows
    td = plain.TORCH[dt]
    n_out, n_in, tokens = 40_003, 32_800, 5
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    dy = torch.randint(-4, 5, (tokens, n_out), generator=g, device=DEV).to(td)
    x = torch.randint(-4, 5, (tokens, n_in), generator=g, device=DEV).to(td)
    q = torch.empty(tokens, n_in, dtype=torch.uint8, device=DEV)
    e = torch.empty(tokens, -(-n_in // 32), dtype=torch.uint8, device=DEV)
    zs.zero_act_save(q, e, x)
    dw = torch.empty(n_out, n_in, device=DEV)
    zs.zero_weight_grad(dw, dy, q, e, workspace=space(tokens, n_out, n_in))
    for r in (slice(0, 300), slice(n_out // 2, n_out // 2 + 300), slice(n_out - 300, n_out)):
        want = sum(dy[t, r].float()[:, None] * x[t].float()[None, :] for t in range(tokens))
        assert torch.equal(dw[r], want)
