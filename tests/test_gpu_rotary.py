"""GPU parity of svdq_rotary against its fp64 form: both pairings, one to four axes, head widths that
are and are not whole vectors, types, norms of either, strides, far positions, in place, graphs.

Bound of one element (u = 2^-24): cos and sin are off by 8 u (the reduced angle's rounding to fp32,
pi u at most, and the library function's 4) and by the binary64 product's 2^-50 |angle|; the normed
pair by 44 u (a sum of at most 16 products a lane and 6 over lanes, halved by the root, and 32 for the
root, the factors and what is left); the turn takes 4.  Then the result's rounding."""
import pytest
import torch

import bit_diffusion_amd as bd
from oracle import packed

pytestmark = pytest.mark.gpu
U, DEV = 2.0 ** -24, "cuda:0"
F32, BF = torch.float32, torch.bfloat16
DT = {F32: bd.SVDQ_DT_F32, BF: bd.SVDQ_DT_BF16}
HALF = {F32: U, BF: 2.0 ** -8}


class Case:
    def __init__(self, seed, M, H, G, pairs, halves=False, xd=BF, od=BF, norm="qk", pad=0, opad=0, shift=0, far=1.0, eps=1e-6,
                 ppad=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        self.M, self.H, self.G, self.pairs, self.halves, self.xd, self.od, self.eps = M, H, G, pairs, halves, xd, od, eps
        self.D = D = 2 * sum(pairs)
        self.width = (H + 2 * G) * D + pad
        self.x = (rnd(M, self.width) * (0.2 + 2 * torch.rand(self.width, generator=g))).to(xd).to(DEV)
        self.shift = shift
        self.qs, self.ks = self.width, self.width
        self.pos = torch.randint(-40, 40, (M, len(pairs) + ppad), generator=g).float() * far + 0.25 * rnd(M, len(pairs) + ppad)
        self.pos = self.pos.to(DEV)
        self.freqs = torch.cat([10000.0 ** (-torch.arange(p, dtype=torch.float64) / p) for p in pairs if p]).to(DEV)
        self.qw = (1 + 0.2 * rnd(D)).to(BF).to(DEV) if "q" in norm else None
        self.kw = (1 + 0.2 * rnd(D)).to(BF).to(DEV) if "k" in norm else None
        self.os = (H * D + opad, G * D + opad)
        self.o = [torch.full((M, s + shift), 9.0, dtype=od, device=DEV) for s in self.os]

    def call(self, stream=None, x=None, outs=None, os=None):
        x = self.x if x is None else x
        s, D = self.shift, self.D
        qo, ko = outs or [o[:, s:] for o in self.o]
        os = os or [v + s for v in self.os]
        bd.svdq_rotary(self.M, self.H, self.G, D, self.pairs, bd.SVDQ_ROTARY_HALVES if self.halves else bd.SVDQ_ROTARY_INTERLEAVED,
                       self.pos, self.pos.shape[1], self.freqs, self.eps, self.qw, self.kw, DT[self.xd], x[:, s:], self.qs,
                       x[:, s + self.H * D:], self.ks, DT[self.od], qo, os[0], ko, os[1], stream=stream)

    def check(self, outs=None, x=None):
        f = lambda t: None if t is None else t.double().cpu()   # noqa: E731
        x = f(self.x if x is None else x)[:, self.shift:]
        axis = torch.tensor([a for a, p in enumerate(self.pairs) for _ in range(p)])
        at = 0
        for heads, w, o, i in ((self.H, self.qw, None if outs is None else outs[0], 0), (self.G, self.kw, None if outs is None else outs[1], 1)):
            n = heads * self.D
            if n == 0:
                continue
            ref, size, ang = packed.rotary(x[:, at:at + n], heads, axis, f(self.pos), f(self.freqs), f(w), self.eps, self.halves)
            at += n
            wide = self.o[i] if o is None else o
            got = f(wide[:, self.shift:self.shift + n] if o is None else o[:, :n])
            e = size * ((44 * U if w is not None else 0) + 12 * U + ang * 2.0 ** -50)
            tol = e + HALF[self.od] * (ref.abs() + e) + 1e-37
            bad = (got - ref).abs() > tol
            assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / tol).max()), bad.nonzero()[:5])
            if o is None:
                rest = wide.clone()
                rest[:, self.shift:self.shift + n] = 9.0
                assert bool((rest == 9.0).all()), "wrote beside the columns"


CASES = {
    "one pair": dict(M=3, H=1, G=1, pairs=[1]),
    "one row": dict(M=1, H=24, G=24, pairs=[64], norm=""),
    "image": dict(M=130, H=24, G=24, pairs=[8, 28, 28]),
    "image, fp32": dict(M=33, H=3, G=3, pairs=[8, 28, 28], xd=F32, od=F32),
    "video, halves": dict(M=77, H=16, G=4, pairs=[16, 16, 16], halves=True, xd=F32, far=100000.0),
    "halves of 64": dict(M=515, H=4, G=2, pairs=[32], halves=True),
    "halves of 128": dict(M=9, H=4, G=2, pairs=[30, 34], halves=True, od=F32),
    "halves of 144": dict(M=9, H=4, G=2, pairs=[30, 42], halves=True),
    "halves of 256": dict(M=9, H=2, G=2, pairs=[100, 28], halves=True, xd=F32, od=F32),
    "halves of 256, bf16": dict(M=2050, H=2, G=1, pairs=[100, 28], halves=True, od=F32),
    "halves of 160, fp32": dict(M=12, H=2, G=1, pairs=[80], halves=True, xd=F32),
    "halves of 16, fp32": dict(M=12, H=2, G=1, pairs=[8], halves=True, xd=F32, od=F32),
    "four axes": dict(M=21, H=5, G=1, pairs=[4, 9, 3, 20]),
    "an axis without pairs": dict(M=21, H=5, G=1, pairs=[0, 9, 0, 11]),
    "heads of 72": dict(M=600, H=16, G=16, pairs=[12, 12, 12]),
    "heads of 200": dict(M=40, H=3, G=1, pairs=[50, 50], xd=F32),
    "heads of 256": dict(M=40, H=3, G=1, pairs=[128]),
    "heads of 248, fp32": dict(M=40, H=3, G=1, pairs=[124], xd=F32, od=F32),
    "heads of 216": dict(M=40, H=3, G=1, pairs=[108], od=F32),
    "heads of 8": dict(M=40, H=3, G=1, pairs=[4], od=F32),
    "heads of 56, fp32": dict(M=40, H=3, G=1, pairs=[20, 8], xd=F32, od=F32),
    "heads of 56": dict(M=40, H=3, G=1, pairs=[20, 8], xd=F32),
    "heads of 104": dict(M=40, H=3, G=1, pairs=[20, 32], od=F32),
    "heads of 104, fp32": dict(M=40, H=3, G=1, pairs=[20, 32], xd=F32),
    "heads of 30": dict(M=70, H=3, G=3, pairs=[5, 5, 5]),
    "heads of 30, halves": dict(M=70, H=3, G=3, pairs=[5, 5, 5], halves=True, xd=F32, od=F32),
    "halves of 24": dict(M=70, H=3, G=3, pairs=[12], halves=True, od=F32),
    "heads of 254": dict(M=11, H=3, G=2, pairs=[127], xd=F32),
    "unaligned rows": dict(M=50, H=3, G=3, pairs=[16, 16], pad=9, opad=3, shift=1),
    "padded rows": dict(M=50, H=3, G=3, pairs=[16, 16], pad=16, opad=8, ppad=3),
    "norm of q": dict(M=50, H=3, G=5, pairs=[16, 16], norm="q"),
    "norm of k": dict(M=50, H=3, G=5, pairs=[16, 16], norm="k", halves=True),
    "q alone": dict(M=50, H=7, G=0, pairs=[16, 16]),
    "k alone": dict(M=50, H=0, G=7, pairs=[16, 16]),
    "rows of several workgroups": dict(M=5003, H=2, G=1, pairs=[20, 20]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_fp64(name):
    print("rotary", name, flush=True)
    c = Case(len(name) * 13 + 1, **CASES[name])
    c.call()
    torch.cuda.synchronize()
    c.check()
    first = [o.clone() for o in c.o]
    c.call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, c.o)), "another run gives other bits"


TYPES = [dict(M=37, H=4, G=2, pairs=pairs, halves=halves, xd=xd, od=od)
         for pairs, halves in (([20, 8], False), ([32, 32], False), ([124], False), ([20, 12], True), ([80], True),
                               ([5, 10], False), ([45], False), ([100, 27], False), ([15], True), ([30, 15], True), ([127], True))
         for xd in (BF, F32) for od in (BF, F32)]


@pytest.mark.parametrize("kw", TYPES)
def test_types(kw):
    c = Case(11, **kw)
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("pairs,halves,xd", [([8, 28, 28], False, BF), ([16, 16], True, F32), ([5, 6], False, BF)])
def test_in_place(pairs, halves, xd):
    c = Case(7, 300, 6, 2, pairs, halves=halves, xd=xd, od=xd)
    buf = c.x.clone()
    n = 6 * c.D
    c.call(x=buf, outs=[buf, buf[:, n:]], os=[c.width, c.width])
    torch.cuda.synchronize()
    c.check(outs=[buf, buf[:, n:]])
    assert torch.equal(buf[:, 8 * c.D:], c.x[:, 8 * c.D:]), "v was written"


def test_far_positions_keep_their_angle():
    """Positions of 2^24: an angle held in fp32 would be off by a radian."""
    c = Case(8, 64, 2, 2, [64], xd=F32, od=F32, norm="")
    c.pos.copy_((torch.arange(64, device=DEV) + (1 << 24) - 100).float()[:, None])
    c.call()
    torch.cuda.synchronize()
    c.check()


def test_positions_that_are_not_numbers_stay_in_their_row():
    c, ref = (Case(9, 40, 3, 3, [16, 16]) for _ in range(2))
    c.pos[7, 1] = float("nan")
    c.pos[9, 0] = float("inf")
    c.call()
    ref.call()
    torch.cuda.synchronize()
    for a, b in zip(c.o, ref.o):
        v = a.reshape(40, 3, 64)
        assert bool(torch.isnan(v[7, :, 32:]).all()) and bool(torch.isnan(v[9, :, :32]).all())
        a[7], a[9] = b[7], b[9]
        assert torch.equal(a, b)


def test_graph_replays():
    c = Case(10, 200, 4, 2, [8, 12, 12])
    c.call()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            c.call(stream=side)
    torch.cuda.synchronize()
    for i in range(3):
        c.x.mul_(1.25)
        c.pos.add_(float(i) + 0.5)
        [o.fill_(9.0) for o in c.o]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.check()


def test_two_streams():
    cs = [Case(20 + i, 2000, 8, 8, [8, 12, 12]) for i in range(2)]
    want = []
    for c in cs:
        c.call()
        torch.cuda.synchronize()
        want.append([o.clone() for o in c.o])
        [o.fill_(9.0) for o in c.o]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, s in zip(cs, streams):
        c.call(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert all(torch.equal(a, b) for a, b in zip(c.o, w))


def test_no_rows_and_offsets_past_32_bits():
    t = torch.full((64,), 5.0, device=DEV)
    f = torch.ones(4, dtype=torch.float64, device=DEV)
    bd.svdq_rotary(0, 1, 1, 8, [4], 0, None, 1, f, 0.0, None, None, 0, None, 8, None, 8, 0, None, 8, None, 8)
    bd.svdq_rotary(3, 0, 0, 8, [4], 0, t, 1, f, 0.0, None, None, 0, None, 0, None, 0, 0, None, 0, None, 0)
    torch.cuda.synchronize()
    assert bool((t == 5.0).all())
    c = Case(30, 40, 2, 1, [16, 16], halves=True)
    s = ((1 << 31) // 39 // 8 + 1) * 8
    n = 39 * s + c.width
    assert n > 1 << 31
    x, qo, ko = (torch.empty(n, dtype=BF, device=DEV).as_strided((40, c.width), (s, 1)) for _ in range(3))
    x.copy_(c.x)
    c.qs = c.ks = s
    c.call(x=x, outs=[qo, ko], os=[s, s])
    torch.cuda.synchronize()
    c.check(outs=[qo, ko])
