"""GPU parity of the adapters and the group norm at sizes that take the kernels which the other
tests' sizes do not, and on both sides of the limits between them, against the same binary64 forms
and element bounds.  test_launches shows that every kernel is among the launches of these cases."""
import pytest
import torch

from test_gpu_group_norm import BF, DEV, F32
from test_gpu_group_norm import Case as Norm
from test_gpu_lora_batch import Case as Lora
from test_gpu_lora_batch import cuts

pytestmark = pytest.mark.gpu


def ones(n):
    return dict(M=n, starts=list(range(n + 1)), ids=[i % 4 - 1 for i in range(n)])


LORA = {
    # 32 rows a workgroup, 64 columns a wave, and 32 columns
    "32 rows, whole lines, rank 32": dict(M=8200, K=64, N=2060, R=32, starts=cuts(4000, 33, 4167), ids=[0, 1, 2], act=1),
    "32 rows, rank 16": dict(M=8200, K=64, N=1030, R=16, starts=cuts(4000, 33, 4160), ids=[0, 1, 2]),
    "32 rows, rank 64": dict(M=8200, K=64, N=1030, R=64, starts=cuts(4000, 33, 4160), ids=[0, 1, 2], ranks=[64, 5, 33]),
    # 16 rows, 64 columns
    "whole lines of single rows, rank 16": dict(K=64, N=2100, R=16, **ones(300)),
    "whole lines of single rows, rank 32": dict(K=64, N=2100, R=32, ranks=[32, 1, 17], **ones(300)),
    "whole lines of single rows, rank 64": dict(K=64, N=2100, R=64, act=2, **ones(300)),
    # 16 rows, 32 columns
    "few rows, many columns, rank 16": dict(M=300, K=192, N=4400, R=16, starts=cuts(130, 0, 170), ids=[0, 1, 2], act=2),
    "few rows, many columns, rank 16, fp32": dict(M=300, K=192, N=4400, R=16, starts=cuts(130, 0, 160), ids=[0, 1, 2], bf=False),
    "few rows, many columns, rank 32, fp32": dict(M=300, K=192, N=4401, R=32, starts=cuts(130, 170), ids=[0, 1], bf=False, act=1),
    "few rows, many columns, rank 32": dict(M=300, K=192, N=4400, R=32, starts=cuts(130, 170), ids=[2, 1], ranks=[32, 3, 20]),
    # eight column blocks a workgroup, the last one not whole
    "32 rows, rank 128, eight blocks": dict(M=8200, K=64, N=4100, R=128, starts=cuts(4000, 4200), ids=[0, 1], ranks=[128, 100, 1]),
    "32 rows, rank 128, eight blocks of low ranks": dict(M=8200, K=64, N=4100, R=128, starts=cuts(4000, 4200), ids=[0, 1], ranks=[64, 7, 1]),
}


@pytest.mark.parametrize("name", list(LORA))
def test_lora_batch(name):
    print("lora_batch", name, flush=True)
    c = Lora(len(name) * 13 + 5, **LORA[name])
    if c.ranks is not None:
        for s, r in enumerate(c.ranks):
            c.ddown[s, r:] = float("nan")
            c.dup[s, :, r:] = float("inf")
    got = c.call()
    torch.cuda.synchronize()
    c.check(got)
    first = got.clone()
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(got, first)


NORM = {
    # x of 32 MB and more: out past the caches
    "large, bf16": dict(B=1, rows=70001, C=256, G=32, mod=F32),
    "large, fp32": dict(B=1, rows=70001, C=128, G=8, xd=F32),
    "large, fp32 out": dict(B=2, rows=40003, C=256, G=16, od=F32, act=1),
    "large, two groups a vector": dict(B=1, rows=60003, C=320, G=32, mod=BF),
    "large, two groups a vector, fp32": dict(B=1, rows=30003, C=320, G=32, xd=F32, od=F32, act=0),
    "large, padded rows": dict(B=1, rows=70001, C=256, G=32, xpad=8, opad=24),
    "large, single elements": dict(B=1, rows=140001, C=125, G=5),
    "large, single elements, fp32": dict(B=1, rows=70001, C=125, G=25, xd=F32, od=F32),
    "the last below 32 MB": dict(B=1, rows=65535, C=256, G=32),
    "the first of 32 MB": dict(B=1, rows=65536, C=256, G=32),
    # two launches, ways a vector lies in the groups
    "two launches, groups of 10, fp32": dict(B=2, rows=4099, C=320, G=32, xd=F32, od=F32, act=1),
    "two launches, groups of 6, bf16": dict(B=1, rows=9001, C=192, G=32),
    "two launches, groups of 4, bf16": dict(B=2, rows=9001, C=64, G=16, mod=F32),
    "two launches, groups of 3, fp32": dict(B=1, rows=9001, C=96, G=32, xd=F32, od=F32),
    "two launches, groups of 2, fp32": dict(B=1, rows=9001, C=64, G=32, xd=F32),
    "two launches, single elements, bf16": dict(B=1, rows=20001, C=33, G=3),
    # one launch, four rows a thread
    "four rows, fp32": dict(B=3, rows=1999, C=64, G=4, xd=F32, od=F32),
    "four rows, groups of 10, fp32": dict(B=2, rows=800, C=320, G=32, xd=F32, od=F32, mod=F32),
    "four rows, groups of 3, fp32": dict(B=8, rows=500, C=96, G=32, xd=F32, od=F32),
    "four rows, groups of 4, bf16": dict(B=20, rows=500, C=64, G=16),
    "four rows, single elements, fp32": dict(B=7, rows=150, C=66, G=6, xd=F32, od=F32, xpad=1, opad=3),
    "four rows, single elements, bf16": dict(B=7, rows=150, C=66, G=6),
    # one row a thread
    "one row, groups of 3, fp32": dict(B=1, rows=20, C=96, G=32, xd=F32),
    "one row, groups of 6, bf16": dict(B=1, rows=20, C=96, G=16),
    "one row, groups of 10, fp32": dict(B=1, rows=20, C=320, G=32, xd=F32, act=1),
    # the limits: vectors of a slab, vectors read in all, one row or four
    "fp32, the one launch's last": dict(B=1, rows=2048, C=64, G=4, xd=F32, od=F32),
    "fp32, the two launches' first": dict(B=1, rows=2049, C=64, G=4, xd=F32, od=F32),
    "reads, the one launch's last": dict(B=32, rows=1024, C=64, G=4),
    "reads, the two launches' first": dict(B=33, rows=1024, C=64, G=4),
    "one row, the last": dict(B=127, rows=64, C=64, G=4),
    "four rows, the first": dict(B=127, rows=65, C=64, G=4),
}


@pytest.mark.parametrize("name", list(NORM))
def test_group_norm(name):
    print("group_norm", name, flush=True)
    c = Norm(len(name) * 19 + 1, **NORM[name])
    got = c.call().clone()
    torch.cuda.synchronize()
    c.check(got)
    if c.os > c.C:
        w = c.wo.clone()
        w[:, c.shift:c.shift + c.C] = 9.0
        assert bool((w == 9.0).all())
    again = c.call()
    torch.cuda.synchronize()
    assert torch.equal(got, again)


@pytest.mark.parametrize("rows,C,G,xd", [(70001, 256, 32, BF), (70001, 128, 8, F32), (60003, 320, 32, BF), (70001, 125, 5, F32)])
def test_group_norm_of_large_images_in_place(rows, C, G, xd):
    c = Norm(11, 1, rows, C, G, xd=xd, od=xd, mod=F32)
    buf = c.x.to(DEV)
    c.call(x=buf, out=buf)
    torch.cuda.synchronize()
    c.check(buf)
