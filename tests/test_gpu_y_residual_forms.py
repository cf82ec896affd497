"""The backward step between two blocks without biases, whose parameters' gradients come from
two sums over the rows instead of four: every way in which rows are held, from one wave a row
to the longest rows on chip, and rows walked over in memory."""
import pytest
import torch

import zero_sharded_mixed_shard_amd as zs
from test_gpu_y_residual import Case

pytestmark = pytest.mark.gpu

# rows of one wave with one group a lane and with two, of several waves, the last widths on
# chip for each format and the first past them; whole and odd lengths
WIDTHS = [(9, 512), (9, 520), (6, 1024), (6, 1025), (5, 1600), (4, 4104), (4, 5120), (3, 8191),
          (3, 8192), (3, 8193), (3, 9216), (2, 12288), (2, 12555), (2, 16383), (2, 16384),
          (2, 16392)]


@pytest.mark.parametrize("rows,cols", WIDTHS)
@pytest.mark.parametrize("dt,res", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"),
                                    ("f32", "f32")])
@pytest.mark.parametrize("post,pre,p", [("rms", "rms", 0.0), ("layer", "layer", 0.1)])
def test_two_sums(rows, cols, dt, res, post, pre, p):
    c = Case(rows, cols, dt, res, post, pre, bias=False, p=p)
    c.check_backward(ld=cols % 3, off=cols % 2)


# more rows than workgroups, so that a workgroup adds several rows to its sums
@pytest.mark.parametrize("rows,cols", [(2100, 512), (2500, 700), (530, 1600), (300, 5120),
                                       (520, 8192), (300, 8193), (600, 12288), (270, 16383)])
@pytest.mark.parametrize("dt,res,post,pre,p", [("bf16", "bf16", "rms", "rms", 0.0),
                                               ("f16", "f16", "none", "layer", 0.1),
                                               ("bf16", "f32", "layer", "rms", 0.1)])
def test_two_sums_of_many_rows(rows, cols, dt, res, post, pre, p):
    c = Case(rows, cols, dt, res, post, pre, bias=False, p=p)
    c.check_backward(out=dt)
    c.check_backward(first=False, du=False)


@pytest.mark.parametrize("cols", [700, 5120, 8200, 12555, 16384])
@pytest.mark.parametrize("dt,res", [("bf16", "bf16"), ("f16", "f32")])
def test_two_sums_in_place_and_in_small_grids(cols, dt, res):
    c = Case(40, cols, dt, res, "rms", "layer", bias=False)
    a = c.check_backward()
    zs.zero_set_grid_cap(3)
    try:
        b = c.check_backward(in_place=True)
    finally:
        zs.zero_set_grid_cap(0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for k, t in a[2].items():
        assert t is None or torch.equal(t, b[2][k]), k
