"""Dropout on the GPU: equal to the definition bit for bit."""
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


def expected(x, p, seed, offset):
    y = plain.dropout(x.float().numpy(), p, seed, offset)
    return torch.from_numpy(y).to(x.dtype)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (61, 769), (5, 4099), (400, 64)])
@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 0.1, 0.5, 0.99999, 1.0])
def test_exact(dt, rows, cols, p):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g).to(TORCH[dt])
    seed, offset = 0x9abcdef012345678, (rows << 33) + cols
    want = expected(x, p, seed, offset)
    for ld, off in ((0, 0), (5, 1)):
        _, v = place(x, ld, off)
        buf, y = place(torch.zeros_like(x), ld, off)
        zs.zero_dropout(y, v, p, seed, offset)
        assert torch.equal(y.cpu(), want) and untouched(buf, y, off)
        zs.zero_dropout(v, v, p, seed, offset)            # in place
        assert torch.equal(v.cpu(), want)


def test_what_is_dropped_is_zero_whatever_it_was():
    x = torch.full((64, 64), float("nan"), device=DEV)
    x[::2] = float("inf")
    y = torch.empty_like(x)
    zs.zero_dropout(y, x, 0.5, 1, 2)
    keep, _ = plain.mask(64, 64, 0.5, 1, 2)
    keep = torch.from_numpy(keep)
    y = y.cpu()
    assert bool((y[~keep] == 0).all()) and bool(y[::2][keep[::2]].isinf().all())
    assert bool(y[1::2][keep[1::2]].isnan().all())


def test_mask_depends_on_the_place_and_not_on_the_matrix():
    ones = torch.ones(50, 200, device=DEV)
    whole, part = torch.empty_like(ones), torch.empty(30, 77, device=DEV)
    zs.zero_dropout(whole, ones, 0.3, 5, 6)
    zs.zero_dropout(part, ones[:30, :77], 0.3, 5, 6)
    assert torch.equal(part, whole[:30, :77])


def test_offset_from_the_device():
    x = torch.ones(40, 333, device=DEV)
    a, b = torch.empty_like(x), torch.empty_like(x)
    for held, offset in ((0, 7), (5, 7), (2 ** 40, 2 ** 35), (-3, 2)):     # wraps at 2^64
        d = torch.tensor([held], dtype=torch.int64, device=DEV)
        zs.zero_dropout(a, x, 0.4, 9, offset, d_offset=d)
        want = expected(x.cpu(), 0.4, 9, (offset + held) % 2 ** 64)
        assert torch.equal(a.cpu(), want)
        zs.zero_dropout(b, x, 0.4, 9, (offset + held) % 2 ** 64)
        assert torch.equal(a, b)


def test_a_captured_graph_draws_a_new_mask_each_replay():
    x = torch.ones(64, 1000, device=DEV)
    y, step = torch.empty_like(x), torch.zeros(1, dtype=torch.int64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        zs.zero_dropout(y, x, 0.25, 3, 100, d_offset=step)
    for k in range(4):
        step.fill_(k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), expected(x.cpu(), 0.25, 3, 100 + k))
    del graph


def test_small_grid():
    x = torch.randn(333, 517, generator=torch.Generator().manual_seed(1)).to(DEV)
    y = torch.empty_like(x)
    zs.zero_set_grid_cap(2)
    try:
        zs.zero_dropout(y, x, 0.1, 1, 1)
    finally:
        zs.zero_set_grid_cap(0)
    assert torch.equal(y.cpu(), expected(x.cpu(), 0.1, 1, 1))


def test_refusals():
    x = torch.zeros(4, 8, device=DEV)
    for bad in (torch.zeros(4, 9, device=DEV), torch.zeros(4, 8, device=DEV).bfloat16(),
                torch.zeros(8, 4, device=DEV).t(), torch.zeros(4, 8)):
        with pytest.raises((ValueError, TypeError)):
            zs.zero_dropout(bad, x, 0.1, 1)
    with pytest.raises(TypeError):
        zs.zero_dropout(x, x, 0.1, 1, 0, d_offset=torch.zeros(1, device=DEV))
    with pytest.raises(ValueError):
        zs.zero_dropout(x, x, 0.1, 1, 0, d_offset=torch.zeros(2, dtype=torch.int64, device=DEV))
    for p in (-0.01, 1.01, float("nan")):
        with pytest.raises(zs.ZeroError):
            zs.zero_dropout(x, x, p, 1)
