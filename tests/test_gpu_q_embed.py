"""The embedding lookup and its gradient by sorted tokens on the GPU."""
import numpy as np
import pytest
import torch

import grad_plain as plain
import zero_sharded_mixed_shard_amd as zs
from gpu_util import log
from test_gpu_o_act import Framed

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def ids_of(tokens, vocab, seed, kind="mixed", dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens,), generator=g)
    if kind == "same":
        ids.fill_(vocab // 2)
    elif kind == "mixed":          # a third one id, some outside the table
        ids[torch.rand(tokens, generator=g) < 0.33] = vocab - 1
        ids[torch.rand(tokens, generator=g) < 0.1] = -1
        ids[torch.rand(tokens, generator=g) < 0.05] = vocab
        if tokens > 3 and dtype == torch.int64:
            ids[1], ids[2] = -2 ** 62, 2 ** 40 + 3
    elif kind == "outside":
        ids.fill_(-100)
    elif kind == "distinct":
        ids = torch.randperm(vocab, generator=g)[:tokens]
    return ids.to(dtype)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,vocab,width,gap,scale", [
    (1, 1, 1, 0, 1.0), (1, 100, 768, 0, 1.0), (7, 50, 33, 0, 0.5), (130, 1000, 64, 8, 27.7),
    (1000, 77, 255, 1, -1.3), (3, 5, 8192, 0, 1.0), (513, 300, 7, 2, 2.0),
    (37, 90, 2051, 3, 0.3), (5, 9, 4099, 0, 3.0), (200, 40, 513, 1, 1.0), (11, 6, 259, 0, 1.7)])
def test_lookup_is_exact(tokens, vocab, width, gap, scale, itype, dt):
    g = torch.Generator().manual_seed(width)
    h = torch.randn(vocab, width, generator=g).to(plain.TORCH[dt])
    table = Framed(vocab, width, h.dtype, lead=width % 3)
    table.t.copy_(h)
    ids = ids_of(tokens, vocab, tokens, dtype=itype)
    out = Framed(tokens, width, h.dtype, width + gap, lead=1)
    zs.zero_embed_lookup(out.t, table.t, ids.to(DEV), scale=scale)
    want = torch.from_numpy(plain.lookup(plain.f64(h), ids.numpy(), scale)).to(h.dtype)
    assert torch.equal(out.t.cpu(), want)
    assert out.intact() and table.intact()


def test_lookup_of_an_empty_table_and_far_rows():
    out = torch.full((4, 9), 3.0, device=DEV)
    zs.zero_embed_lookup(out, torch.empty(0, 9, device=DEV),
                         torch.zeros(4, dtype=torch.int64, device=DEV))
    assert bool((out == 0).all())
    table = torch.zeros(600_000, 4096, dtype=torch.bfloat16, device=DEV)   # 4.9 GB
    table[-1] = 1.5
    out = torch.empty(2, 4096, dtype=torch.bfloat16, device=DEV)
    zs.zero_embed_lookup(out, table, torch.tensor([599_999, 0], device=DEV), scale=2.0)
    assert bool((out[0] == 3).all()) and bool((out[1] == 0).all())


def grad_case(tokens, vocab, width, dt, kind, scale, itype=torch.int64, seed=1, gap=0):
    td = plain.TORCH[dt]
    g = torch.Generator().manual_seed(seed)
    ids = ids_of(tokens, vocab, seed + 1, kind, itype)
    h = torch.randint(-8, 9, (tokens, width), generator=g).float()
    dy = Framed(tokens, width, td, width + gap, lead=width % 5)
    dy.t.copy_(h)
    skip = (ids < 0) | (ids >= vocab)
    dy.t[skip.to(DEV)] = float("nan")            # never read
    want, _ = plain.embed_grad(h.double().numpy(), ids.numpy(), vocab, scale)
    ws = torch.full((zs.zero_embed_grad_workspace(tokens, vocab, width),), 255,
                    dtype=torch.uint8, device=DEV)
    return ids, dy, want, ws


# whole numbers: sums are exact in FP32, so results must match to the bit
GRADS = [(1, 1, 1, "distinct"), (1, 50257, 64, "mixed"), (5, 3, 9, "mixed"),
         (31, 7, 16, "same"), (32, 7, 16, "same"), (33, 9, 513, "same"), (64, 100, 40, "mixed"),
         (65, 64, 768, "mixed"), (1000, 333, 520, "mixed"), (1024, 2048, 24, "distinct"),
         (1500, 40, 33, "same"), (4000, 513, 2049, "mixed"), (8192, 1000, 16, "mixed"),
         (8193, 1000, 16, "mixed"), (20000, 511, 40, "mixed"), (20000, 512, 8, "mixed"),
         (16385, 300_000, 8, "mixed"), (70_001, 5, 24, "mixed"), (300_000, 1000, 8, "mixed"),
         (9000, 17, 8, "outside"), (12_345, 20_000, 8, "distinct"), (40_000, 1, 8, "same")]


@pytest.mark.parametrize("tokens,vocab,width,kind", GRADS)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gradient_of_whole_numbers_is_exact(tokens, vocab, width, kind, dt):
    itype = torch.int32 if tokens % 2 else torch.int64
    ids, dy, want, ws = grad_case(tokens, vocab, width, dt, kind, 0.5, itype,
                                  gap=tokens % 3)
    d_ids = ids.to(DEV)
    td = plain.TORCH[dt]
    for out_dt in (td, torch.float32):
        dw = Framed(vocab, width, out_dt, lead=3)
        zs.zero_embed_grad(dw.t, dy.t, d_ids, scale=0.5, workspace=ws)
        assert torch.equal(dw.t.cpu(), torch.from_numpy(want).float().to(out_dt))
        assert dw.intact()
    # accumulation touches only the rows that occur
    acc = Framed(vocab, width, torch.float32, lead=1)
    acc.t[:] = 2.0
    seen = torch.zeros(vocab, dtype=torch.bool)
    seen[ids[(ids >= 0) & (ids < vocab)].long()] = True
    acc.t[~seen.to(DEV)] = float("nan")
    zs.zero_embed_grad(acc.t, dy.t, d_ids, scale=0.5, first=False, workspace=ws)
    got = acc.t.cpu().double()
    assert bool(torch.isnan(got[~seen]).all())
    assert np.array_equal(got[seen].numpy(), 2.0 + want[seen.numpy()])
    assert acc.intact() and torch.equal(d_ids.cpu(), ids)


# few tokens in a large table: ids that crowd into one group of rows, runs on both sides of
# 16 tokens, tables that end inside a group of 64 rows
FEW = [(1024, 16_384, 48, "mixed"), (1024, 16_383, 48, "mixed"), (1025, 16_384, 48, "mixed"),
       (1024, 262_144, 8, "mixed"), (1024, 262_145, 8, "mixed"), (1, 16_385, 1, "same"),
       (1024, 20_000, 1030, "same"), (1023, 16_447, 520, "crowd"), (1000, 20_001, 512, "runs"),
       (700, 17_000, 2051, "runs"), (512, 50_257, 768, "distinct"), (300, 16_400, 9, "outside"),
       (65, 16_385, 777, "last")]


@pytest.mark.parametrize("tokens,vocab,width,kind", FEW)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gradient_of_few_tokens_is_exact(tokens, vocab, width, kind, dt, monkeypatch):
    special = {"crowd": lambda t: 64 * 7 + t % 64,            # 16 tokens a row, interleaved
               "runs": lambda t: 63 + 5 * (t * (t + 1) % 33 % 11),   # rows of uneven counts
               "last": lambda t: vocab - 1 - t % 3}
    if kind in special:
        make = special[kind]
        monkeypatch.setitem(globals(), "ids_of", lambda n, v, s, k, dtype=torch.int64:
                            torch.tensor([make(t) for t in range(n)]).to(dtype))
    test_gradient_of_whole_numbers_is_exact(tokens, vocab, width, kind, dt)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,vocab,width",
                         [(700, 50, 130), (30_000, 2000, 64), (1000, 20_000, 130)])
def test_random_gradients_within_the_sum_bound_and_repeatable(tokens, vocab, width, dt):
    g = torch.Generator().manual_seed(3)
    h = torch.randn(tokens, width, generator=g).to(plain.TORCH[dt])
    ids = ids_of(tokens, vocab, 4)
    want, bound = plain.embed_grad(plain.f64(h), ids.numpy(), vocab, 27.7)
    ws = torch.empty(zs.zero_embed_grad_workspace(tokens, vocab, width), dtype=torch.uint8,
                     device=DEV)
    dw = torch.empty(vocab, width, device=DEV)
    zs.zero_embed_grad(dw, h.to(DEV), ids.to(DEV), scale=27.7, workspace=ws)
    err = np.abs(plain.f64(dw) - want)
    assert np.all(err <= bound + 1e-30), (err / (bound + 1e-30)).max()
    again = torch.empty_like(dw)
    zs.zero_embed_grad(again, h.to(DEV), ids.to(DEV), scale=27.7, workspace=ws)
    assert torch.equal(dw, again)
    d16 = torch.empty(vocab, width, dtype=h.dtype, device=DEV)
    zs.zero_embed_grad(d16, h.to(DEV), ids.to(DEV), scale=27.7, workspace=ws)
    assert torch.equal(d16.cpu(), dw.cpu().to(h.dtype))
    log(f"  embed grad {dt} {tokens}: worst {float((err / (bound + 1e-30)).max()):.3f}")


def test_no_tokens():
    dw = Framed(6, 10, torch.bfloat16)
    dy = torch.empty(0, 10, dtype=torch.bfloat16, device=DEV)
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    zs.zero_embed_grad(dw.t, dy, ids)
    assert bool((dw.t == 0).all()) and dw.intact()
    acc = torch.ones(6, 10, device=DEV)
    zs.zero_embed_grad(acc, dy, ids, first=False)
    assert bool((acc == 1).all())


@pytest.mark.parametrize("cap", [1, 3])
@pytest.mark.parametrize("tokens", [500, 9000])
def test_grid_loops_under_a_lowered_cap(tokens, cap):
    ids, dy, want, ws = grad_case(tokens, 100, 700, "bf16", "mixed", 1.0)
    dw = torch.empty(100, 700, device=DEV)
    out = torch.empty(tokens, 700, dtype=torch.bfloat16, device=DEV)
    table = torch.randn(100, 700, device=DEV).bfloat16()
    zs.zero_set_grid_cap(cap)
    try:
        zs.zero_embed_grad(dw, dy.t, ids.to(DEV), workspace=ws)
        zs.zero_embed_lookup(out, table, ids.to(DEV))
    finally:
        zs.zero_set_grid_cap(0)
    assert np.array_equal(plain.f64(dw), want)
    look = torch.from_numpy(plain.lookup(plain.f64(table), ids.numpy(), 1.0)).bfloat16()
    assert torch.equal(out.cpu(), look)


def test_lookup_and_gradient_are_adjoint():
    # <lookup(W), dy> = <W, grad(dy)> for whole numbers, exactly
    ids, dy, want, ws = grad_case(900, 40, 24, "bf16", "mixed", 2.0)
    W = torch.randint(-8, 9, (40, 24)).float()
    out = torch.empty(900, 24, dtype=torch.bfloat16, device=DEV)
    zs.zero_embed_lookup(out, W.bfloat16().to(DEV), ids.to(DEV), scale=2.0)
    dw = torch.empty(40, 24, device=DEV)
    zs.zero_embed_grad(dw, dy.t, ids.to(DEV), scale=2.0, workspace=ws)
    left = (out.double() * dy.t.double().nan_to_num(0.0)).sum().item()
    assert left == (W.double() * dw.cpu().double()).sum().item()


def test_gradient_rows_past_4_gib():
    # a table gradient of 5.4 GB and dy of 4.4 GB: offsets past 2^32 on both sides
    vocab, width, tokens = 330_000, 4096, 540_000
    ids = torch.full((tokens,), vocab - 2, dtype=torch.int32, device=DEV)
    ids[::1000] = vocab - 1
    ids[1::1000] = 0
    dy = torch.zeros(tokens, width, dtype=torch.bfloat16, device=DEV)
    dy[-1], dy[-1000], dy[-999] = 1.0, 2.0, 4.0     # ids vocab - 2, vocab - 1 and 0
    ws = torch.empty(zs.zero_embed_grad_workspace(tokens, vocab, width), dtype=torch.uint8,
                     device=DEV)
    dw = torch.full((vocab, width), 3.0, device=DEV)
    zs.zero_embed_grad(dw, dy, ids, workspace=ws)
    assert bool((dw[vocab - 2] == 1).all()) and bool((dw[vocab - 1] == 2).all())
    assert bool((dw[0] == 4).all()) and not bool(dw[1:vocab - 2].any())
