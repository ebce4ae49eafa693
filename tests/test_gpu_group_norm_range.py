"""svdq_group_norm on values whose squares, or whose sums, pass fp32's range while the squares
about the group's mean do not: the statistics stay finite, in one launch and in two, for every way
a vector lies in the groups, with row lanes, tiles and lanes of the joins that have no values.

A constant group has a mean of exactly its value (every join adds a difference of zero) and a
variance of zero, so out is exactly the rounded offset D.  Groups with a spread keep the bound of
the element errors in test_gpu_group_norm."""
import pytest
import torch

from test_gpu_group_norm import BF, F32, Case

pytestmark = pytest.mark.gpu

# B, rows, C, groups: one row (all other row lanes empty), a ragged chunk, one launch of four rows a
# thread, two launches with a last tile of few rows, a wide group in parts (its last one narrower)
SHAPES = {
    "one row": (2, 1, 64, 8), "ragged chunk": (1, 37, 64, 8), "two groups a vector": (1, 45, 80, 8),
    "any groups": (1, 100, 48, 16), "single elements": (1, 77, 33, 3), "four rows": (1, 2000, 64, 4),
    "two launches": (1, 20003, 64, 8), "two launches, two groups": (1, 20003, 80, 8),
    "two launches, any groups": (1, 20003, 48, 16), "two launches, single elements": (1, 9003, 33, 3),
    "wide group in parts": (1, 700, 1544, 1),
}


@pytest.mark.parametrize("xd", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_constant_groups(shape, xd):
    B, rows, C, G = SHAPES[shape]
    c = Case(5, B, rows, C, G, xd=xd, od=F32, act=0)
    want = c.b.float().expand(B * rows, C)
    for value in (1e20, -1e20, 1e30 / 3, -3e38, 1234.567):
        print("constant", shape, xd, value, flush=True)
        c.wx.fill_(value)
        got = c.call()
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), want), value


# a spread of `step` about `offset`, both far from zero: squares of the offset overflow, those
# about the mean (at most 1.5 million of them) do not
@pytest.mark.parametrize("offset,step,xd", [(1e20, 1e15, F32), (-1e20, 1e15, F32), (1e22, 1e16, F32), (1e5, 0.5, F32)])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_small_spread_about_a_large_offset(shape, offset, step, xd):
    B, rows, C, G = SHAPES[shape]
    print("spread", shape, offset, flush=True)
    c = Case(6, B, rows, C, G, xd=xd, od=F32, act=0, affine=False, eps=1e-5)
    g = torch.Generator().manual_seed(9)
    c.x = (offset + step * torch.randn(B * rows, C, generator=g, dtype=torch.float64)).to(xd)
    c.wx.copy_(c.x)
    got = c.call()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(got).all())
    c.check(got)


@pytest.mark.parametrize("shape", list(SHAPES))
def test_few_outliers_about_a_large_offset_bf16(shape):
    """2^66 with 32 values one bf16 step (2^59) higher: 32 x 2^118 = 2^123 in squares."""
    B, rows, C, G = SHAPES[shape]
    c = Case(7, B, rows, C, G, od=F32, act=0)
    c.x.fill_(2.0 ** 66)
    flat = c.x.view(-1)
    flat[torch.randperm(flat.numel(), generator=torch.Generator().manual_seed(3))[:32]] = 2.0 ** 66 + 2.0 ** 59
    c.wx.copy_(c.x)
    got = c.call()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(got).all())
    c.check(got)


def test_infinities_still_spoil_their_group_alone():
    for rows in (100, 30000):
        c, ref = Case(8, 1, rows, 64, 8), Case(8, 1, rows, 64, 8)
        c.wx[3, 17] = float("inf")
        c.wx[rows - 1, 42] = float("-inf")
        got, want = c.call().clone(), ref.call()
        torch.cuda.synchronize()
        assert bool(torch.isnan(got[:, 16:24]).all()) and bool(torch.isnan(got[:, 40:48]).all())
        for lo in (16, 40):
            got[:, lo:lo + 8] = want[:, lo:lo + 8]
        assert torch.equal(got, want)
