"""GPU parity of svdq_layer_norm against its fp64 form: types, widths on both sides of every choice
the launcher makes, cuts with empty and single-row segments and rows of none, strides, optional
operands, in place, captured graphs, other streams.

Bound of one element (u = 2^-24, L = 80 the longest chain of additions on the way to a row's sum: 32
values of a thread, 6 of a wave, 16 waves, rounded up): h is off by 2 u of its summands.  The mean's
own rounding is taken off again with the mean of the differences d = h - mean, whose sum is off by L u
of the largest |d|.  The variance is off by a relative 2 (L + 8) u, and as the mean's error squared;
half of that passes the root.  d rstd A + D takes 10 roundings, A and D 3 of their summands."""
import pytest
import torch

import bit_diffusion_amd as bd
from oracle import packed

pytestmark = pytest.mark.gpu
U, L, DEV = 2.0 ** -24, 80, "cuda:0"
F32, BF = torch.float32, torch.bfloat16
DT = {F32: bd.SVDQ_DT_F32, BF: bd.SVDQ_DT_BF16}
HALF = {F32: U, BF: 2.0 ** -8}


class Case:
    def __init__(self, seed, starts, C, tail=0, xd=BF, yd=BF, od=BF, md=F32, residual=True, gate=True, affine=False, mod=True,
                 keep=True, xpad=0, ypad=0, opad=0, shift=0, offset=1.0, spread=1.0, eps=1e-6, no_starts=False):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        self.starts, self.C, self.M, self.n = starts, C, starts[-1] + tail, len(starts) - 1
        self.xd, self.yd, self.od, self.md, self.eps, self.shift, self.no_starts = xd, yd, od, md, eps, shift, no_starts
        M, n = self.M, self.n
        self.xs, self.ys, self.os = C + xpad, C + ypad, C + opad
        wide = lambda t, s, dt: torch.cat([torch.full((M, shift), 7.0), t, torch.full((M, s - C - shift), 7.0)], 1).to(dt).to(DEV)   # noqa: E731
        self.wx = wide(rnd(M, C) * spread * (0.3 + torch.rand(C, generator=g)) + offset, self.xs, xd)
        self.wy = wide(rnd(M, C), self.ys, yd) if residual else None
        self.w = (1 + 0.3 * rnd(C)).to(BF).to(DEV) if affine else None
        self.b = (0.3 * rnd(C)).to(BF).to(DEV) if affine else None
        # a stride that takes what C takes
        self.ms = 3 * C + (4 if C % 4 == 0 else 2 - C % 2)
        self.mod = (0.4 * rnd(n, self.ms)).to(md).to(DEV)
        self.gate = self.mod[:, :C] if gate and residual else None
        self.scale, self.mshift = (self.mod[:, C:2 * C], self.mod[:, 2 * C:3 * C]) if mod else (None, None)
        self.start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.wo = torch.full((M, self.os), 9.0, dtype=od, device=DEV)
        self.wh = torch.full((M, self.xs), 9.0, dtype=xd, device=DEV) if residual and keep else None

    def view(self, t):
        return None if t is None else t[:, self.shift:self.shift + self.C]

    def call(self, stream=None, x=None, y=None, out=None, xo=None):
        p = lambda t: None if t is None else t[:, self.shift:]   # noqa: E731
        bd.svdq_layer_norm(self.M, self.C, self.n, self.eps, DT[self.xd], p(self.wx if x is None else x), self.xs, DT[self.yd],
                           p(self.wy if y is None else y), self.ys, self.w, self.b, None if self.no_starts else self.start,
                           DT[self.md], self.gate, self.scale, self.mshift, self.ms, p(self.wh if xo is None else xo), self.xs,
                           DT[self.od], p(self.wo if out is None else out), self.os, stream=stream)

    def expect(self):
        f = lambda t: None if t is None else t.double().cpu()   # noqa: E731
        self.seg = packed.segment_of(self.starts, self.M)
        if self.no_starts:
            self.seg[:] = 0
        return packed.layer_norm(f(self.view(self.wx)), f(self.view(self.wy)), f(self.w), f(self.b), self.seg, f(self.gate),
                                 f(self.scale), f(self.mshift), self.eps)

    def check(self, want, out=None, xo=None):
        h, ref, p = want
        inside = self.seg >= 0
        out = self.view(self.wo if out is None else out).double().cpu()
        # h: one rounding of the product and one of the sum at most, then the result's
        eh = 2 * U * p["hin"] * (self.wy is not None)
        dmax, hmax = p["d"].abs().amax(1, keepdim=True), p["hin"].amax(1, keepdim=True)
        first = L * U * hmax                                    # the first mean's error
        dm = eh + eh.amax(1, keepdim=True) + (L + 4) * U * (dmax + first)
        var = 2 * (L + 8) * U * (1 + (first * p["rstd"]) ** 2) + 2 * (dm * p["rstd"]).amax(1, keepdim=True)
        z = (p["d"] * p["rstd"] * p["A"]).abs()
        e = dm * p["rstd"] * p["A"].abs() + z * (0.5 * var + 10 * U) + 8 * U * (p["Dabs"] + ref.abs())
        tol = e + HALF[self.od] * (ref.abs() + e) + 1e-37
        bad = ((out - ref).abs() > tol) & inside[:, None]
        assert not bad.any(), (int(bad.sum()), float(((out - ref).abs() / tol)[inside].max()), bad.nonzero()[:5])
        assert bool((out[~inside] == 9.0).all()), "rows of no segment were written"
        xo = self.wh if xo is None else xo
        if xo is not None:
            got = self.view(xo).double().cpu()
            tol = eh + HALF[self.xd] * (h.abs() + eh)
            assert bool(((got - h).abs() <= tol)[inside].all())
            assert bool((got[~inside] == 9.0).all())


def cut(*lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


CASES = {
    "one row": dict(starts=cut(1), C=64),
    "one value": dict(starts=cut(3), C=1, xd=F32, od=F32),
    "four values": dict(starts=cut(2, 1), C=4),
    "odd width": dict(starts=cut(5, 0, 1, 9), C=333, tail=3, xd=F32, od=F32),
    "up to one wave": dict(starts=cut(30, 34), C=256, md=BF),
    "the first of two vectors": dict(starts=cut(30, 34), C=260, md=BF, affine=True),
    "up to two vectors": dict(starts=cut(7, 1, 1, 8), C=2048, tail=5),
    "the first of four": dict(starts=cut(7, 1, 1, 8), C=2052, xd=F32, yd=F32, od=F32),
    "the metric's width": dict(starts=cut(100, 0, 37), C=3072, tail=1),
    "up to four vectors": dict(starts=cut(9), C=4096, yd=F32, od=F32),
    "the first of eight": dict(starts=cut(9, 2), C=4100, xd=F32, md=BF),
    "widest": dict(starts=cut(2, 3), C=16384, affine=True),
    "pairs, one": dict(starts=cut(6, 5), C=126),
    "pairs, two": dict(starts=cut(6, 5), C=1170, tail=3, xd=F32, md=BF, affine=True),
    "pairs, four": dict(starts=cut(6, 5), C=2050, od=F32),
    "pairs, eight": dict(starts=cut(3, 5), C=4098, yd=F32),
    "pairs, widest": dict(starts=cut(3, 2), C=8190, xd=F32, od=F32),
    "pairs by a stride": dict(starts=cut(30, 20), C=320, xpad=2),
    "pairs by an address": dict(starts=cut(30, 20), C=320, xpad=4, ypad=4, opad=4, shift=2),
    "single elements, one": dict(starts=cut(6, 6), C=63, yd=F32),
    "single elements, two": dict(starts=cut(6, 7), C=511, od=F32),
    "single elements, four": dict(starts=cut(6, 0, 0, 7), C=1023, xd=F32, md=BF, affine=True),
    "single elements, eight": dict(starts=cut(3, 4), C=1025),
    "single elements, widest": dict(starts=cut(3, 2), C=8191, xd=F32, yd=F32),
    "no residual": dict(starts=cut(50, 14), C=320, residual=False, affine=True),
    "no gate": dict(starts=cut(50, 14), C=320, gate=False, mod=False),
    "only the norm": dict(starts=cut(64), C=640, residual=False, mod=False, no_starts=True),
    "h not kept": dict(starts=cut(50, 14), C=320, keep=False),
    "no offsets": dict(starts=cut(77), C=128, no_starts=True),
    "single rows": dict(starts=list(range(101)), C=192),
    "many segments": dict(starts=sorted([0] + [(i * 7919) % 5000 for i in range(4200)] + [5000]), C=24, tail=4),
    "starts late": dict(starts=[13, 13, 40, 41], C=96, tail=9),
    "several rounds of a workgroup": dict(starts=cut(4000, 3001, 1, 2500), C=40),
    "padded rows": dict(starts=cut(40, 33), C=128, xpad=8, ypad=4, opad=16),
    "unaligned rows": dict(starts=cut(40, 33), C=128, xpad=5, ypad=6, opad=7, shift=3),
    "far from zero": dict(starts=cut(20), C=320, xd=F32, od=F32, offset=3000.0, residual=False),
    "tiny": dict(starts=cut(20), C=320, xd=F32, od=F32, offset=0.0, spread=1e-5, residual=False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_fp64(name):
    print("layer_norm", name, flush=True)
    c = Case(len(name) * 31 + 5, **CASES[name])
    c.call()
    torch.cuda.synchronize()
    c.check(c.expect())
    w = c.wo.clone()
    c.view(w).fill_(9.0)
    assert bool((w == 9.0).all()), "wrote beside the columns"
    first = [t.clone() for t in (c.wo, c.wh) if t is not None]
    c.call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, [t for t in (c.wo, c.wh) if t is not None])), "another run gives other bits"


@pytest.mark.parametrize("xd", [BF, F32])
@pytest.mark.parametrize("yd", [BF, F32])
@pytest.mark.parametrize("od", [BF, F32])
@pytest.mark.parametrize("C", [200, 1200, 3072, 5000, 9000, 122, 1170, 2050, 4102, 63, 333, 2001, 3001])
def test_types(xd, yd, od, C):
    c = Case(C, cut(11, 0, 6), C, tail=2, xd=xd, yd=yd, od=od, md=BF, affine=True)
    c.call()
    torch.cuda.synchronize()
    c.check(c.expect())


def test_constant_rows_give_the_offset():
    c = Case(3, cut(9, 8), 331, xd=F32, od=F32, residual=False)
    c.wx[:] = torch.linspace(-1000.1, 5e6, c.M, device=DEV)[:, None]
    c.call()
    torch.cuda.synchronize()
    want = c.mshift[packed.segment_of(c.starts, c.M).to(DEV)]
    assert torch.equal(c.view(c.wo), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_rows_spoil_no_other(bad):
    c, ref = (Case(4, cut(30, 35), 384) for _ in range(2))
    c.wx[17, 5] = bad
    c.call()
    ref.call()
    torch.cuda.synchronize()
    assert bool(torch.isnan(c.wo[17]).all())
    keep = torch.arange(c.M, device=DEV) != 17
    assert torch.equal(c.wo[keep], ref.wo[keep]) and torch.equal(c.wh[keep], ref.wh[keep])


@pytest.mark.parametrize("C", [384, 3072, 6000, 77])
@pytest.mark.parametrize("which", ["x_out is x", "out is y", "x_out is y", "out is x"])
def test_in_place(which, C):
    c, ref = (Case(9, cut(300, 1, 0, 220), C, tail=3) for _ in range(2))
    ref.call()
    torch.cuda.synchronize()
    x, y = c.wx.clone(), c.wy.clone()
    out, xo = {"x_out is x": (c.wo, x), "out is y": (y, c.wh), "x_out is y": (c.wo, y), "out is x": (x, c.wh)}[which]
    c.call(x=x, y=y, out=out, xo=xo)
    torch.cuda.synchronize()
    assert torch.equal(out[:521], ref.wo[:521]) and torch.equal(xo[:521], ref.wh[:521])


def test_graph_replays_with_other_offsets():
    c = Case(8, cut(40, 50, 10), 320)
    c.call()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            c.call(stream=side)
    torch.cuda.synchronize()
    for starts in ([0, 0, 99, 100], [0, 1, 2, 3], [5, 70, 70, 90], [0, 40, 90, 100]):
        c.starts = starts
        c.start.copy_(torch.tensor(starts, dtype=torch.int32))
        c.wo.fill_(9.0)
        c.wh.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.check(c.expect())
        got = c.wo.clone(), c.wh.clone()
        c.wo.fill_(9.0)
        c.wh.fill_(9.0)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], c.wo) and torch.equal(got[1], c.wh)


def test_two_streams():
    cs = [Case(50 + i, cut(2000, 1, 900), 640) for i in range(2)]
    want = []
    for c in cs:
        c.call()
        torch.cuda.synchronize()
        want.append((c.wo.clone(), c.wh.clone()))
        c.wo.zero_()
        c.wh.zero_()
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, s in zip(cs, streams):
        c.call(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert torch.equal(c.wo, w[0]) and torch.equal(c.wh, w[1])


def test_offsets_that_decrease_stay_inside():
    """Nothing beside the rows is written, whatever the offsets hold."""
    c = Case(60, cut(40, 40, 20), 64, tail=5)
    big = 2 ** 31 - 1
    for starts in ([50, 10, 80, 3], [-5, 200, -9, 30], [big, -big - 1, big, 7], [9, 9, 1000000, 0]):
        pad = torch.full((c.M + 64, c.C), 9.0, dtype=BF, device=DEV)
        c.start.copy_(torch.tensor(starts, dtype=torch.int32))
        c.call(out=pad[32:32 + c.M])
        torch.cuda.synchronize()
        assert bool((pad[:32] == 9.0).all()) and bool((pad[32 + c.M:] == 9.0).all()), starts


def test_zero_sizes_and_offsets_past_32_bits():
    t = torch.full((64,), 5.0, device=DEV)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    for M, n in ((0, 1), (3, 0)):
        bd.svdq_layer_norm(M, 8, n, 1e-6, 0, t, 8, 0, None, 0, None, None, st, 0, None, None, None, 8, None, 0, 0, t[32:], 8)
    torch.cuda.synchronize()
    assert bool((t == 5.0).all())
    c = Case(70, cut(30, 11), 64, residual=False)
    s = ((1 << 31) // (c.M - 1) // 8 + 1) * 8
    n = (c.M - 1) * s + c.C
    assert n > 1 << 31
    x, out = (torch.empty(n, dtype=BF, device=DEV).as_strided((c.M, c.C), (s, 1)) for _ in range(2))
    x.copy_(c.wx)
    c.xs = c.os = s
    c.call(x=x, out=out)
    torch.cuda.synchronize()
    c.xs = c.os = c.C
    c.check(c.expect(), out=out)
