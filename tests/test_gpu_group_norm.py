"""GPU parity of svdq_group_norm against its fp64 form: types, group widths that are and are
not whole vectors, image sizes on both sides of every choice the launcher makes, strides,
modulation, activations, offsets far from zero, in place, captured graphs, other streams.

Bound of one element (u = 2^-24, L the longest chain of additions on the way to a mean or a
sum of squares, 256 here: chunks, joins, lanes and tiles together): the mean is off by L u of
the group's largest |x|; the deviation's square sum by a relative 2 (L + 8) u plus the square
of the mean's error over the deviation, both halved by the root; (x - mean) A + D takes 8
roundings.  Both activations have slope <= 1.13 and 32 roundings of their own."""
import numpy as np
import pytest
import torch

import bit_diffusion_amd as bd
from oracle import batch

pytestmark = pytest.mark.gpu
U, L, DEV = 2.0 ** -24, 256, "cuda:0"
DT = {torch.float32: bd.SVDQ_DT_F32, torch.bfloat16: bd.SVDQ_DT_BF16}
F32, BF = torch.float32, torch.bfloat16


class Case:
    def __init__(self, seed, B, rows, C, G, xd=BF, od=BF, act=2, affine=True, mod=None, offset=1.0, spread=1.0, xpad=0,
                 opad=0, shift=0, eps=1e-5):
        g = torch.Generator().manual_seed(seed)
        self.B, self.rows, self.C, self.G, self.act, self.eps = B, rows, C, G, act, eps
        self.xd, self.od, self.md = xd, od, mod or F32
        self.x = (torch.randn(B * rows, C, generator=g) * (spread * (0.3 + torch.rand(C, generator=g))) + offset).to(xd)
        self.w = (1 + 0.3 * torch.randn(C, generator=g)).to(BF) if affine else None
        self.b = (0.3 * torch.randn(C, generator=g)).to(BF) if affine else None
        self.mod = (0.4 * torch.randn(B, 2 * C + 3, generator=g)).to(mod) if mod else None
        self.xs, self.os, self.shift = C + xpad, C + opad, shift
        self.wx = torch.full((B * rows, self.xs), float("nan"), dtype=xd)
        self.wx[:, shift:shift + C] = self.x
        self.wx = self.wx.to(DEV)
        self.wo = torch.full((B * rows, self.os), 9.0, dtype=od, device=DEV)
        self.dw, self.db = (None, None) if not affine else (self.w.to(DEV), self.b.to(DEV))
        self.dmod = None if mod is None else self.mod.to(DEV)
        self.nb = bd.svdq_group_norm_workspace_bytes(B, rows, C, G)
        self.ws = torch.full((max(self.nb, 16),), 0xFF, dtype=torch.uint8, device=DEV)

    def call(self, stream=None, x=None, out=None):
        x = self.wx[:, self.shift:] if x is None else x
        out = self.wo[:, self.shift:] if out is None else out
        ms = None if self.dmod is None else self.dmod[:, :self.C]
        mt = None if self.dmod is None else self.dmod[:, self.C + 3:]
        bd.svdq_group_norm(self.B, self.rows, self.C, self.G, self.eps, DT[self.xd], x, self.xs, self.dw, self.db,
                           DT[self.md], ms, mt, 2 * self.C + 3, self.act, DT[self.od], out, self.os, self.ws, self.nb,
                           stream=stream)
        return self.wo[:, self.shift:self.shift + self.C]

    def check(self, got):
        f = lambda t: None if t is None else t.double().numpy()   # noqa: E731
        x = f(self.x).reshape(self.B, self.rows, self.C)
        ms = None if self.mod is None else f(self.mod[:, :self.C])
        mt = None if self.mod is None else f(self.mod[:, self.C + 3:])
        ref, p = batch.group_norm(x, self.G, self.eps, f(self.w), f(self.b), ms, mt, self.act)
        got = got.double().cpu().numpy().reshape(ref.shape)
        dm = L * U * p["big"] * p["rstd"]                      # the mean's error, in deviations
        e = np.abs(p["F"]) * (dm + np.abs(p["xhat"]) * ((L + 8) * U + dm * dm)) \
            + 8 * U * (np.abs(p["xhat"] * p["F"]) + np.abs(p["D"]))
        if self.act:
            e = 1.13 * e + 32 * U * np.abs(p["y"])
        half = 2.0 ** -8 if self.od == BF else U
        tol = e + half * (np.abs(ref) + e) + 1e-37
        bad = np.abs(got - ref) > tol
        assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / tol).max()), np.argwhere(bad)[:5])


CASES = {
    "one position": dict(B=1, rows=1, C=64, G=8),
    "one value a group": dict(B=2, rows=1, C=40, G=40, act=1),
    "one channel": dict(B=1, rows=7, C=1, G=1, xd=F32, od=F32),
    "one group": dict(B=2, rows=50, C=264, G=1, act=0),
    "two positions": dict(B=3, rows=2, C=320, G=32, mod=F32),
    "8x8": dict(B=2, rows=64, C=1280, G=32),
    "9x7, groups of 10": dict(B=2, rows=63, C=320, G=32, xd=F32, od=F32, mod=BF),
    "groups of 4": dict(B=1, rows=333, C=128, G=32, act=1),
    "groups of 1": dict(B=1, rows=500, C=96, G=96, affine=False),
    "groups of 20": dict(B=2, rows=1024, C=640, G=32, mod=F32),
    "groups of 11, odd": dict(B=2, rows=513, C=330, G=30, xd=F32, od=F32, act=1, mod=BF),
    "groups of 11, odd, bf16": dict(B=1, rows=2100, C=33, G=3),
    "wide odd group": dict(B=1, rows=130, C=501, G=3, xd=F32, od=BF),
    "wide group": dict(B=2, rows=77, C=2080, G=2, act=1),
    "wide group, many rows": dict(B=1, rows=700, C=1544, G=1, xd=F32, od=F32, mod=F32),
    "prime width": dict(B=1, rows=90, C=127, G=127, act=0),
    "16 rows a thread": dict(B=1, rows=2000, C=64, G=4),
    "the resident form's last": dict(B=1, rows=2048, C=64, G=4, act=0),
    "the split form's first": dict(B=1, rows=2049, C=64, G=4, act=0),
    "fp32, resident's last": dict(B=1, rows=1024, C=64, G=4, xd=F32, od=F32),
    "fp32, split's first": dict(B=1, rows=1025, C=64, G=4, xd=F32, od=F32),
    "64x64": dict(B=1, rows=4096, C=320, G=32),
    "many tiles": dict(B=1, rows=70001, C=64, G=8, od=F32, mod=F32),
    "many images": dict(B=40, rows=31, C=96, G=12),
    "padded rows": dict(B=2, rows=300, C=128, G=16, xpad=8, opad=24),
    "unaligned": dict(B=2, rows=300, C=128, G=16, xpad=5, opad=3, shift=3),
    "unaligned, split": dict(B=1, rows=9001, C=24, G=6, xpad=5, opad=3, shift=3, xd=F32),
    "far from zero": dict(B=1, rows=900, C=64, G=8, xd=F32, od=F32, offset=1000.0, act=0),
    "far from zero, split": dict(B=1, rows=20000, C=64, G=8, xd=F32, od=F32, offset=1000.0, act=0),
    "tiny values": dict(B=1, rows=200, C=64, G=8, xd=F32, od=F32, offset=0.0, spread=1e-4, act=0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_fp64(name):
    print("group_norm", name, flush=True)
    c = Case(len(name) * 17 + 3, **CASES[name])
    got = c.call().clone()
    torch.cuda.synchronize()
    c.check(got)
    w = c.wo.clone()
    w[:, c.shift:c.shift + c.C] = 9.0
    assert bool((w == 9.0).all()), "wrote beside the columns"
    again = c.call()
    torch.cuda.synchronize()
    assert torch.equal(got, again), "another run gives other bits"


@pytest.mark.parametrize("rows", [200, 30000])
def test_constant_images_and_single_outliers(rows):
    """A constant group has variance 0: the result is the offset.  One huge value in a row is
    no reason for the others' squares to be lost."""
    c = Case(5, 1, rows, 64, 8, xd=F32, od=F32, act=0)
    c.x[:] = 3.25
    c.x[0, 8] = 30000.0
    c.wx.copy_(c.x)
    got = c.call()
    torch.cuda.synchronize()
    c.check(got)
    assert torch.equal(got[:, 16:].cpu(), c.b[16:].float().expand(rows, 48))


@pytest.mark.parametrize("rows", [100, 30000])
def test_nan_stays_in_its_group(rows):
    c = Case(6, 2, rows, 64, 8)
    ref = Case(6, 2, rows, 64, 8)
    c.wx[rows + 3, 17] = float("nan")            # image 1, group 2
    got, want = c.call().clone(), ref.call()
    torch.cuda.synchronize()
    assert bool(torch.isnan(got[rows:, 16:24]).all())
    got[rows:, 16:24] = want[rows:, 16:24]
    assert torch.equal(got, want)


# in place, rows that other workgroups still read must stay: more workgroups than run at a time,
# in images that out of place take one launch
@pytest.mark.parametrize("B,rows,C,G,xd", [(1, 150, 64, 8, BF), (1, 150, 64, 8, F32), (1, 40000, 64, 8, BF), (2, 16, 64, 8, F32),
                                           (40, 1024, 320, 32, BF), (40, 1000, 96, 12, F32), (64, 64, 640, 32, BF),
                                           (300, 256, 64, 2, BF), (8, 300, 50, 5, F32)])
def test_in_place(B, rows, C, G, xd):
    c = Case(7, B, rows, C, G, xd=xd, od=xd, mod=F32)
    buf = c.x.to(DEV)
    c.call(x=buf, out=buf)
    torch.cuda.synchronize()
    c.check(buf)


@pytest.mark.parametrize("rows", [100, 50000])
def test_graph_replays(rows):
    c = Case(8, 1, rows, 64, 8, mod=BF)
    c.call()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            c.call(stream=side)
    torch.cuda.synchronize()
    for k in range(3):
        c.x = (c.x.float() * 1.5 + k).to(BF)
        c.wx.copy_(c.x)
        c.wo.fill_(9.0)
        c.ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = c.wo.clone()
        c.check(got)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(c.wo, got), k


def test_two_streams_with_their_own_workspaces():
    cs = [Case(50 + i, 1, 20000, 64, 8) for i in range(2)]
    want = [c.call().clone() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for c in cs:
            c.wo.zero_()
        torch.cuda.synchronize()
        for c, st in zip(cs, streams):
            c.call(stream=st)
        torch.cuda.synchronize()
        for c, w in zip(cs, want):
            assert torch.equal(c.wo, w)


def test_zero_sizes():
    t = torch.full((64,), 5.0, device=DEV)
    for B, rows in ((0, 4), (3, 0)):
        bd.svdq_group_norm(B, rows, 64, 8, 1e-5, 0, t, 64, None, None, 0, None, None, 64, 0, 0, t, 64, None, 0)
    torch.cuda.synchronize()
    assert bool((t == 5.0).all())


# positions whose offsets pass 2^31 elements: one launch, two, and single elements
@pytest.mark.parametrize("B,rows,C,G", [(1, 40, 64, 8), (1, 20000, 64, 8), (2, 3000, 33, 3)])
def test_offsets_past_32_bits(B, rows, C, G):
    c = Case(70, B, rows, C, G, mod=F32)
    c.xs = c.os = ((1 << 31) // (B * rows - 1) // 8 + 1) * 8
    n = (B * rows - 1) * c.xs + C
    assert n > 1 << 31
    x, out = (torch.empty(n, dtype=BF, device=DEV).as_strided((B * rows, C), (c.xs, 1)) for _ in range(2))
    x.copy_(c.x)
    c.call(x=x, out=out)
    torch.cuda.synchronize()
    c.check(out)
