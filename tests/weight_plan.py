"""How a weight gradient's extents choose tile, splits and tile groups, for the tests: the same
arithmetic as the launcher's, with its measured costs read from the source."""
from __future__ import annotations

import os
import re
from dataclasses import dataclass

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "zero_sharded_mixed_shard_amd", "csrc", "wgrad_kernels.hip")
UNIT = 128            # tokens: splits are whole units
FILL = 256            # compute units
STEP = {256: 64, 128: 64, 64: 128}   # tokens a step of each tile


def costs() -> list:
    """(tile, ns of 64 tokens, ns of start and end) of each tile, from the source."""
    with open(SOURCE) as f:
        table = re.search(r"TileCost kTiles\[3\] = \{(.*)\};", f.read()).group(1)
    return [tuple(int(v) for v in m) for m in re.findall(r"\{(\d+), (\d+), (\d+)\}", table)]


@dataclass
class Plan:
    tile: int
    splits: int
    per_split: int
    steps: int         # of the first split
    group_i: int


def _up(a, b):
    return -(-a // b)


def plan(tokens, n_out, n_in, table=None) -> Plan:
    units, plane_ns = _up(tokens, UNIT), n_out * n_in // 1000
    best_ns, best = None, None
    for tile, step, ends in table or costs():
        n = _up(n_out, tile) * _up(n_in, tile)
        for s in range(1, min(64, units) + 1):
            if s > 1 and n * s > 2 * FILL:
                break
            per = _up(units, s)
            if _up(units, per) != s:
                continue
            ns = _up(n * s, FILL) * (per * (UNIT // 64) * step + ends)
            if s > 1:
                ns += 5000 + s * (plane_ns + 150)
            if best_ns is None or ns < best_ns:
                best_ns, best = ns, (tile, s, per * UNIT)
    tile, splits, per_split = best
    to, ti = _up(n_out, tile), _up(n_in, tile)
    group = 0
    for gi in (8, 4, 2, 1):
        if to * ti < FILL:
            break
        places = _up(_up(to, 32 // gi) * _up(ti, gi), 8) * 8 * 32
        if places * 8 <= to * ti * 9:
            group = gi
            break
    return Plan(tile, splits, per_split, _up(min(per_split, tokens), STEP[tile]), group)
