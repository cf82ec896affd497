"""That the weight gradient's tests reach every tile, split and grouping (host only)."""
import random

import pytest

import zero_sharded_mixed_shard_amd as zs
from test_gpu_w_weight_tiles import SHAPES
from weight_plan import STEP, UNIT, costs, plan


def test_the_plan_is_the_librarys():
    # the workspace tells the library's splits: 4 bytes a result and split, none for one
    rng, table = random.Random(7), costs()
    size = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    shapes = SHAPES + [(size(1, 40_000), size(8, 60_000), size(8, 60_000)) for _ in range(2000)]
    split = 0
    for s in shapes:
        p = plan(*s, table)
        want = 0 if p.splits == 1 else 4 * s[1] * s[2] * p.splits
        assert zs.zero_weight_grad_workspace(*s) == want, s
        split += p.splits > 1
    assert split > 200


@pytest.mark.parametrize("tile", [256, 128, 64])
def test_every_tile_is_run_through_its_loop(tile):
    # past four steps (the steady part), even and odd; one split and several; whole and ragged
    # last steps; grouped and not
    got = [(s, p) for s, p in ((s, plan(*s)) for s in SHAPES) if p.tile == tile]
    for odd in (0, 1):
        for grouped in (False, True):
            assert any(p.splits == 1 and p.steps > 4 and p.steps % 2 == odd and
                       (p.group_i > 0) == grouped for _, p in got), (odd, grouped)
    assert any(p.splits > 1 and p.steps > 4 for _, p in got)
    assert any(p.splits > 1 and s[0] % UNIT for s, p in got)
    assert any(s[0] % STEP[tile] for s, p in got if p.splits == 1)
    assert any(s[1] % 8 and s[2] % 8 for s, p in got if p.splits == 1)
    assert {p.group_i for _, p in got} >= {0, 1, 8}


def test_every_grouping_is_run():
    assert {p.group_i for p in (plan(*s) for s in SHAPES)} == {0, 1, 2, 4, 8}
