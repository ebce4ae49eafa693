"""GPU parity of svdq_attention against its fp64 form: head widths on both sides of every choice,
grouped heads, cuts with empty segments and rows of none, keys from none to thousands, masks that
leave rows empty, caps, biases, values that are not finite where nobody looks, splits, graphs.

Bound of one element (u = 2^-24, w the softmax weights).  A score is off by 2 D u of sum |q k| scale
(D products in fp32), 4 u of the cap or of its own size, 4 u of its bias, and 4 u of its distance to
the maximum, at most 200 where the weight is not 0 in fp32: with e all that, each weight is off by a
relative 2 e + 4 u in the sum and its normalisation.  Each weight is rounded to bf16, by at most 2^-8
of it; the sum over keys of such roundings times v is at most 2^-8 sum w |v|, and as they are as often
up as down, past 7 2^-8 sqrt(sum (w v)^2) with a probability below 2 exp(-7^2 / 2) = 5e-11 (Hoeffding).
Sums over n keys take (n + 16) u of sum w |v|, a rescaled maximum 2 u for every tile.  Then the result's
rounding to bf16."""
import pytest
import torch

import bit_diffusion_amd as bd
from oracle import packed

pytestmark = pytest.mark.gpu
U, DEV = 2.0 ** -24, "cuda:0"
BF = torch.bfloat16


def cut(*lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


class Case:
    def __init__(self, seed, qs, H, G, D, ks=None, causal=False, prefix=None, cap=0.0, bias=False, tail=0, scale=None, sharp=1.0,
                 pad=0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        self.qs, self.ks, self.H, self.G, self.D = qs, qs if ks is None else ks, H, G, D
        self.Mq, self.Mk = qs[-1] + tail, self.ks[-1] + (tail if ks is None else 0)
        self.n, self.causal, self.cap, self.scale = len(qs) - 1, causal, cap, D ** -0.5 if scale is None else scale
        self.qw, self.kw = H * D + pad, G * D + pad
        self.q = (rnd(self.Mq, self.qw) * sharp).to(BF).to(DEV)
        self.k, self.v = (rnd(max(self.Mk, 1), self.kw).to(BF).to(DEV) for _ in range(2))
        self.start, self.kstart = (torch.tensor(s, dtype=torch.int32, device=DEV) for s in (self.qs, self.ks))
        self.prefix = prefix
        self.dprefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV)
        self.slopes = (torch.exp2(-8.0 * torch.arange(1, H + 1) / H)).to(DEV) if bias else None
        self.out = torch.full((self.Mq, self.qw), 9.0, dtype=BF, device=DEV)
        self.nb = bd.svdq_attention_workspace_bytes(self.Mq, self.Mk, H, G, D, self.n)
        self.ws = torch.full((max(self.nb, 16),), 0xFF, dtype=torch.uint8, device=DEV)

    def call(self, stream=None, out=None):
        bd.svdq_attention(self.Mq, self.Mk, self.H, self.G, self.D, self.n, self.scale, self.cap,
                          bd.SVDQ_MASK_CAUSAL if self.causal else bd.SVDQ_MASK_NONE, self.start, self.kstart, self.dprefix,
                          self.slopes, self.q, self.qw, self.k, self.kw, self.v, self.kw, self.out if out is None else out,
                          self.qw, self.ws, self.nb, stream=stream)

    def parts(self):
        """Row range, key range, head, fp64 form of every segment and head."""
        rep, D = self.H // self.G, self.D
        for i in range(self.n):
            a, b, c, d = self.qs[i], self.qs[i + 1], self.ks[i], self.ks[i + 1]
            if b == a:
                continue
            for h in range(self.H):
                kv = slice(h // rep * D, h // rep * D + D)
                yield a, b, h, packed.attention(self.q[a:b, h * D:h * D + D].double(), self.k[c:d, kv].double(),
                                                self.v[c:d, kv].double(), self.scale, self.cap, self.causal,
                                                0 if self.prefix is None else self.prefix[i],
                                                None if self.slopes is None else float(self.slopes[h])), d - c

    def check(self, out=None):
        out = self.out if out is None else out
        D = self.D
        touched = torch.zeros(self.Mq, self.qw, dtype=torch.bool, device=DEV)
        for a, b, h, (ref, wabs, wroot, size, bias), n in self.parts():
            got = out[a:b, h * D:h * D + D].double()
            touched[a:b, h * D:h * D + D] = True
            e = 2 * D * U * size + 4 * U * torch.maximum(size, torch.full_like(size, self.cap)) + 4 * U * bias + 4 * U * 200
            tol = wabs * (2 * e + 4 * U + (n + 16) * U + 2 * U * (n // 64 + 1)) + torch.minimum(2.0 ** -8 * wabs, 7 * 2.0 ** -8 * wroot)
            tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 1e-37
            bad = ~((got - ref).abs() <= tol)
            assert not bad.any(), (a, b, h, int(bad.sum()), float(((got - ref).abs() / tol).max()), bad.nonzero()[:5])
        assert bool((out[~touched] == 9.0).all()), "wrote beside the rows"


CASES = {
    "one row, one key": dict(qs=cut(1), H=1, G=1, D=8),
    "one row, no key": dict(qs=cut(1), ks=cut(0), H=2, G=1, D=16),
    "a tile": dict(qs=cut(128), ks=cut(64), H=2, G=2, D=128),
    "a tile and one": dict(qs=cut(129), ks=cut(65), H=2, G=2, D=128),
    "joint": dict(qs=cut(700), H=3, G=3, D=128),
    "packed": dict(qs=cut(101, 0, 37, 250, 64, 1, 91), H=4, G=4, D=72, tail=29),
    "packed, 64": dict(qs=cut(101, 0, 37, 250, 64, 1, 91), H=4, G=2, D=64, tail=3),
    "packed, 96": dict(qs=cut(300, 300), H=4, G=1, D=96),
    "packed, 80": dict(qs=cut(150, 150, 1), H=4, G=1, D=80),
    "packed, 32": dict(qs=cut(33, 31, 200), H=4, G=1, D=32),
    "packed, 8": dict(qs=cut(33, 31, 200), H=4, G=1, D=8),
    "packed, 24": dict(qs=cut(33, 31, 200), H=2, G=1, D=24, bias=True),
    "packed, 40": dict(qs=cut(33, 31, 200), H=2, G=1, D=40, cap=5.0),
    "packed, 104": dict(qs=cut(33, 31, 200), H=2, G=1, D=104),
    "packed, 120": dict(qs=cut(33, 31, 200), H=2, G=1, D=120, cap=8.0, bias=True),
    "cross": dict(qs=cut(256, 256, 256, 256), ks=cut(77, 300, 0, 128), H=8, G=8, D=64, cap=30.0),
    "cross, long": dict(qs=cut(500), ks=cut(3000), H=2, G=2, D=128),
    "causal": dict(qs=cut(400, 63, 64, 65, 1), H=2, G=2, D=128, causal=True),
    "causal, grouped": dict(qs=cut(300, 129), H=8, G=2, D=64, causal=True),
    "causal, groups of 5": dict(qs=cut(300, 129), H=5, G=1, D=72, causal=True, bias=True),
    "causal, more rows than keys": dict(qs=cut(200, 3, 90), ks=cut(70, 0, 89), H=2, G=1, D=128, causal=True),
    "causal, more keys than rows": dict(qs=cut(200, 3, 90), ks=cut(300, 700, 91), H=2, G=1, D=128, causal=True),
    "prefix": dict(qs=cut(400, 200, 100), H=4, G=2, D=128, causal=True, prefix=[100, 200, 0]),
    "prefix past the keys": dict(qs=cut(100, 90, 80), H=2, G=2, D=64, causal=True, prefix=[1000, -5, 79]),
    "prefix, rows without own keys": dict(qs=cut(200, 150), ks=cut(70, 0), H=2, G=1, D=96, causal=True, prefix=[33, 10]),
    "capped": dict(qs=cut(300), H=2, G=2, D=128, cap=2.0, sharp=4.0),
    "biased": dict(qs=cut(300, 40), H=4, G=2, D=128, bias=True),
    "capped, biased, causal, prefix": dict(qs=cut(300, 40), H=4, G=2, D=128, bias=True, cap=10.0, causal=True, prefix=[70, 5]),
    "capped, biased, 72": dict(qs=cut(300, 40), H=4, G=2, D=72, bias=True, cap=10.0),
    "capped, 96": dict(qs=cut(130), H=2, G=2, D=96, cap=10.0),
    "biased, 64": dict(qs=cut(130), H=2, G=2, D=64, bias=True),
    "biased, 16, capped": dict(qs=cut(130), H=2, G=2, D=16, bias=True, cap=3.0),
    "capped, 32": dict(qs=cut(130), H=2, G=2, D=32, cap=3.0),
    "capped, biased, 64": dict(qs=cut(130), H=2, G=2, D=64, cap=3.0, bias=True),
    "single rows": dict(qs=list(range(9)), ks=cut(800, 311, 2096, 1, 277, 0, 600, 503), H=8, G=2, D=128, bias=True),
    "single rows, one head": dict(qs=list(range(4)), ks=cut(5000, 64, 3), H=1, G=1, D=64),
    "single rows, causal": dict(qs=list(range(4)), ks=cut(5000, 64, 0), H=2, G=1, D=72, causal=True),
    "few rows, many keys": dict(qs=cut(40, 2), ks=cut(4000, 1000), H=2, G=1, D=128, cap=20.0),
    "few rows, many keys, 32": dict(qs=cut(40, 2), ks=cut(4000, 1000), H=2, G=1, D=32),
    "many rows, split": dict(qs=cut(590, 10), ks=cut(2000, 900), H=8, G=8, D=64),
    "many rows, split, causal": dict(qs=cut(590, 10), ks=cut(2000, 900), H=8, G=8, D=72, causal=True, prefix=[100, 3], tail=5),
    "eight heads, several lengths": dict(qs=cut(140, 300, 20, 0, 10), ks=cut(500, 30, 0, 7, 129), H=16, G=8, D=64, cap=9.0),
    "sixteen heads in step": dict(qs=cut(140, 300), H=16, G=16, D=32),
    "split, one long of many": dict(qs=list(range(9)), ks=cut(22, 11, 14, 529, 199, 14, 3630, 49), H=24, G=24, D=128, cap=50.0),
    "split, short ones whole": dict(qs=cut(66, 315, 493, 20, 60, 91), H=2, G=2, D=80, cap=15.0, tail=13),
    "split, causal": dict(qs=cut(1300), H=4, G=1, D=128, causal=True, tail=40),
    "split, more segments than lanes": dict(qs=list(range(71)), ks=[60 * i if i < 70 else 60 * 69 + 3000 for i in range(71)], H=2, G=2, D=32),
    "parts last, in step": dict(qs=cut(0, 700, 30, 64, 0, 200), ks=cut(100, 2500, 3000, 64, 700, 0), H=8, G=8, D=64, tail=3),
    "parts last, causal": dict(qs=cut(0, 700, 30, 64, 0, 200), ks=cut(100, 2500, 3000, 64, 700, 500), H=6, G=3, D=104, causal=True,
                               prefix=[5, 2000, 0, 7, 1, 100]),
    "parts last, none cut": dict(qs=cut(512, 512, 500, 512), H=4, G=4, D=128, tail=9),
    "parts last, none cut, more rows": dict(qs=cut(1024, 1024, 1000, 1024), H=4, G=4, D=128, tail=9),
    "many segments": dict(qs=sorted([0] + [i * 37 % 900 for i in range(150)] + [900]), H=2, G=1, D=64),
    "more heads than a tile's rows": dict(qs=cut(3, 1), ks=cut(90, 200), H=300, G=2, D=64, causal=True),
    "sharp": dict(qs=cut(500), H=2, G=2, D=128, sharp=60.0),
    "growing scores": dict(qs=cut(130), ks=cut(1000), H=2, G=2, D=64, sharp=30.0),
    "padded rows": dict(qs=cut(130, 20), H=2, G=2, D=72, pad=24),
    "scale of its own": dict(qs=cut(130, 20), H=2, G=2, D=128, scale=1.0),
}


# every number of 16-channel steps, each with and without a cap and a bias, for few heads (two waves share
# rows) and for many
CASES.update({f"width {D}, cap {cap}, bias {bias}, {G} kv heads": dict(qs=cut(130, 20), ks=cut(200, 70), H=H, G=G, D=D, cap=cap, bias=bias)
              for D in (16, 32, 40, 48, 64, 72, 80, 96, 104, 112, 128) for cap in (0.0, 6.0) for bias in (False, True)
              for H, G in ((2, 1), (80, 80))})


@pytest.mark.parametrize("name", list(CASES))
def test_matches_fp64(name):
    print("attention", name, flush=True)
    c = Case(len(name) * 23 + 7, **CASES[name])
    if name == "growing scores":      # every tile has a larger maximum than the one before
        c.k.mul_(torch.linspace(0.01, 1.0, c.k.shape[0], device=DEV)[:, None].to(BF))
    c.call()
    torch.cuda.synchronize()
    c.check()
    first = c.out.clone()
    c.ws.fill_(0xFF)
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out), "another run gives other bits"


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("qlen,klen,H,G,D", [(4097, 4097, 1, 1, 128), (1000, 8191, 2, 1, 64), (1, 30000, 4, 1, 128), (9, 6001, 1, 1, 72),
                                             (5000, 333, 1, 1, 96)])
def test_every_key_counts_once(qlen, klen, H, G, D, causal):
    """q = 0 weighs all keys alike; v has a one in the column of its key's number modulo D, so the
    result is the number of such keys over their sum, exact but for two roundings."""
    c = Case(5, cut(qlen), H, G, D, ks=cut(klen), causal=causal)
    c.q.zero_()
    j = torch.arange(klen, device=DEV)
    c.v.zero_()
    for g in range(G):
        c.v[j, g * D + j % D] = 1.0
    c.call()
    torch.cuda.synchronize()
    n = packed.limits(qlen, klen, causal, 0).to(DEV)[:, None].double()
    count = torch.clamp((n - torch.arange(D, device=DEV) + D - 1) // D, min=0)
    want = torch.where(n > 0, count / n.clamp(min=1), 0 * n)
    for h in range(H):
        got = c.out[:, h * D:h * D + D].double()
        assert bool(((got - want).abs() <= (2.0 ** -8 + 4 * U) * want).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("G", [2, 80])
def test_what_is_not_seen_does_not_count(bad, causal, G):
    """Rows of k and v of other segments, behind the last and, with a causal mask, of later positions."""
    c, ref = (Case(6, cut(70, 90, 133), 2 * G, G, 72, causal=causal, prefix=[0, 3, 0] if causal else None, tail=40) for _ in range(2))
    ref.call()
    hit = torch.zeros(c.Mq, dtype=torch.bool, device=DEV)     # rows that see a bad key
    rows = {20: 70, 100: 160, 165: 293, 292: 293}             # bad row -> end of its segment
    for r, end in rows.items():
        c.k[r] = bad
        c.v[r] = bad
        start = 0 if r < 70 else 70 if r < 160 else 160
        hit[r if causal else start:end] = True
    c.k[300:], c.v[300:] = bad, bad
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out[~hit], ref.out[~hit])
    if bad != bad:
        assert bool(torch.isnan(c.out[hit]).all())


@pytest.mark.parametrize("kw", [dict(), dict(cap=9.0), dict(bias=True), dict(causal=True), dict(causal=True, bias=True, cap=5.0)])
@pytest.mark.parametrize("G", [2, 80])
def test_rows_do_not_depend_on_the_rows_beside_them(kw, G):
    """The same bits whether the other rows of a segment hold numbers, huge ones or none."""
    c = Case(12, cut(150, 90), 2 * G, G, 64, **kw)
    c.call()
    torch.cuda.synchronize()
    ref = c.out.clone()
    odd = torch.arange(240, device=DEV) % 3 == 1
    for v in (float("nan"), 3e4, -float("inf")):
        c.q[odd] = v
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(c.out[~odd], ref[~odd]), v


@pytest.mark.parametrize("D", [32, 64, 96, 128])
@pytest.mark.parametrize("G", [1, 80])
def test_infinite_values_where_seen(D, G):
    """An infinity of v gives its sign to the rows that see it, both signs or a NaN give NaN, in the
    columns that hold them and nowhere else."""
    c, ref = (Case(8, cut(100), 2 * G, G, D, causal=True) for _ in range(2))
    ref.call()
    c.v[50, 3], c.v[60, 4], c.v[70, 5] = float("inf"), -float("inf"), float("nan")
    c.v[52, 7], c.v[80, 7] = float("inf"), -float("inf")
    c.call()
    torch.cuda.synchronize()
    for h in range(2):
        o, r = c.out[:, h * D:h * D + D].float(), ref.out[:, h * D:h * D + D].float()
        assert bool((o[50:, 3] == float("inf")).all()) and bool((o[60:, 4] == -float("inf")).all()) and bool(torch.isnan(o[70:, 5]).all())
        assert bool((o[52:80, 7] == float("inf")).all()) and bool(torch.isnan(o[80:, 7]).all())
        for col, first in ((3, 50), (4, 60), (5, 70), (7, 52)):
            o[first:, col] = r[first:, col]
        assert torch.equal(o, r)


def test_scores_that_are_infinite():
    """A minus infinity among a row's scores is a weight of 0."""
    c = Case(9, cut(40), 1, 1, 64)
    c.q.fill_(1.0)
    c.k[7] = -float("inf")
    c.call()
    torch.cuda.synchronize()
    keep = [j for j in range(40) if j != 7]
    ref = packed.attention(c.q.double(), c.k[keep].double(), c.v[keep].double(), c.scale, 0.0, False, 0, None)[0]
    assert bool(((c.out.double() - ref).abs() <= 2.0 ** -6 * c.v.double().abs().amax()).all())


@pytest.mark.parametrize("kw", [dict(qs=cut(90, 60, 31), H=4, G=2, D=72, causal=True, prefix=[9, 0, 31]),
                                dict(qs=cut(90, 60, 31), H=160, G=80, D=72, causal=True, prefix=[9, 0, 31]),
                                dict(qs=[0, 1, 2, 3], ks=cut(2000, 100, 900), H=4, G=2, D=128)])
def test_graph_replays_with_other_offsets(kw):
    c = Case(10, **kw)
    c.call()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            c.call(stream=side)
    torch.cuda.synchronize()
    m, k = c.qs[-1], c.ks[-1]
    same = c.qs is c.ks
    for i in range(4):
        c.qs = [[0, 0, m - 1, m], [0, 1, 2, m], [1, 1, 1, m], kw["qs"]][i]
        c.ks = c.qs if same else [[0, 50, 51, k], [7, 7, k, k], [0, 1000, 1500, k - 1], kw["ks"]][i]
        c.start.copy_(torch.tensor(c.qs, dtype=torch.int32))
        c.kstart.copy_(torch.tensor(c.ks, dtype=torch.int32))
        c.q.copy_(torch.randn(c.q.shape, generator=torch.Generator().manual_seed(i)).to(BF))
        c.out.fill_(9.0)
        c.ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.check()
        got = c.out.clone()
        c.out.fill_(9.0)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(got, c.out)


@pytest.mark.parametrize("kw", [dict(qs=cut(900, 700), H=4, G=2, D=64), dict(qs=[0, 1, 2, 3], ks=cut(3000, 100, 900), H=4, G=2, D=128)])
def test_two_streams_with_their_own_workspaces(kw):
    cs = [Case(40 + i, **kw) for i in range(2)]
    want = []
    for c in cs:
        c.call()
        torch.cuda.synchronize()
        want.append(c.out.clone())
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for c in cs:
            c.out.fill_(9.0)
        torch.cuda.synchronize()
        for c, s in zip(cs, streams):
            c.call(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(c.out, w) for c, w in zip(cs, want))


@pytest.mark.parametrize("split", [False, True])
def test_offsets_that_decrease_stay_inside(split):
    c = Case(60, [0, 1, 2, 3], 2, 1, 64, ks=cut(2000, 30, 5)) if split else Case(61, cut(40, 40, 20), 2, 1, 64, tail=5)
    assert (c.nb > 0) == split
    big = 2 ** 31 - 1
    for qs, ks in (([50, 10, 80, 3], [60, 4, 90, 1]), ([-5, 200, -9, 30], [-7, 1 << 20, 3, -1]), ([big, -big - 1, big, 7], [0, big, -big - 1, big]),
                   ([0, 1, 2, 3], [9, 3, 2, 1])):
        pad = torch.full((c.Mq + 64, c.qw), 9.0, dtype=BF, device=DEV)
        c.start.copy_(torch.tensor(qs, dtype=torch.int32))
        c.kstart.copy_(torch.tensor(ks, dtype=torch.int32))
        c.call(out=pad[32:32 + c.Mq])
        torch.cuda.synchronize()
        assert bool((pad[:32] == 9.0).all()) and bool((pad[32 + c.Mq:] == 9.0).all()), (qs, ks)


def test_no_rows_and_no_segments():
    t = torch.full((64,), 5.0, device=DEV).to(BF)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    for Mq, n in ((0, 1), (1, 0)):
        bd.svdq_attention(Mq, 1, 1, 1, 8, n, 1.0, 0.0, 0, st, st, None, None, t, 8, t, 8, t, 8, t[32:], 8, None, 0)
    torch.cuda.synchronize()
    assert bool((t == 5.0).all())


def test_offsets_past_32_bits():
    """Keys whose offsets pass 2^31 elements, in every tile and at the last key."""
    c = Case(70, cut(150), 2, 1, 64, ks=cut(300))
    s = 1 << 23
    n = 299 * s + 64
    assert n > 1 << 31
    k = torch.empty(n, dtype=BF, device=DEV).as_strided((300, 64), (s, 1))
    k.copy_(c.k)
    bd.svdq_attention(150, 300, 2, 1, 64, 1, c.scale, 0.0, 0, c.start, c.kstart, None, None, c.q, c.qw, k, s, k, s, c.out, c.qw,
                      c.ws, c.nb)
    c.v.copy_(c.k)
    torch.cuda.synchronize()
    c.check()
