"""The step between two blocks in place (u over r, df over dh, dr over du) on rows that are no
multiple of eight columns.  The lanes of a row's last, short group, and lanes past the row's
end, read the row's last eight columns, some of which another lane, or another wave, writes
over; what they keep must be their own columns' alone, so that results equal those of separate
matrices bit for bit.  Widths put the short group first in a wave, first in a workgroup's second
round of columns, or behind whole groups; without norms no barrier stands between a row's
reads and its writes."""
import pytest
import torch

import zero_sharded_mixed_shard_amd as zs
from test_gpu_y_residual import Case, DEV

pytestmark = pytest.mark.gpu


def run(c, in_place):
    d = lambda t: t.to(DEV)
    told, pre = c.told(), c.P["pre"] != "none"
    r, f, dh, du = d(c.r), d(c.f), d(c.dh) if pre else None, d(c.du)
    new = lambda t: t if in_place else torch.zeros_like(t)
    u, h = new(r), torch.zeros_like(f) if pre else None
    stats = torch.zeros(c.rows, 4, device=DEV)
    zs.zero_residual_norm(u, h, stats, r, f, **told)
    out = [u.clone(), h, stats]
    df, dr = new(dh) if pre else torch.zeros_like(f), new(du)
    ws = torch.empty(zs.zero_residual_norm_workspace(c.rows, c.cols), dtype=torch.uint8,
                     device=DEV)
    grad = lambda k: None if c.par[k] is None else torch.zeros(c.cols, device=DEV)
    grads = {"d_post_weight": grad("w1"), "d_post_bias": grad("b1"), "d_gate": grad("gate"),
             "d_pre_weight": grad("w2"), "d_pre_bias": grad("b2")}
    zs.zero_residual_norm_backward(df, dr, dh, du, f, u, stats, workspace=ws, **grads, **told)
    return out + [df, dr] + list(grads.values())


@pytest.mark.parametrize("rows,cols", [(3000, 9), (5000, 65), (2100, 513), (1500, 1025),
                                       (1030, 2049), (600, 4099), (600, 8191), (600, 8193),
                                       (300, 12553), (300, 16383), (300, 16385)])
@pytest.mark.parametrize("dt,res", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("post,pre,bias", [("none", "none", False), ("rms", "rms", False),
                                           ("none", "layer", True), ("layer", "none", True)])
def test_rows_of_odd_length_in_place(rows, cols, dt, res, post, pre, bias):
    c = Case(rows, cols, dt, res, post, pre, bias=bias)
    want = run(c, False)
    for _ in range(3):
        for a, b in zip(want, run(c, True)):
            assert a is None or torch.equal(a, b)
    if rows * cols < 200000:            # and they are the definition's
        c.check_forward(in_place=True)
        c.check_backward(in_place=True)
