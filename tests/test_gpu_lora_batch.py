"""GPU parity of svdq_lora_batch against its fp64 form: types, ranks, strides, odd widths,
segments of every length, rows without adapter and rows of no segment, values in unused
places, in place, captured graphs, other streams.

Bound of one element (u = 2^-24, the fp32 half step; every sum counted twice for orders and
internal roundings of the matrix unit): t carries 2 (K + 16) u of its terms' absolute sum D
and is used to `split` (2^-16 with two bf16 terms, 2^-24 with three); the up-projection adds
up to 3 R + 4 products, then base.  Both activations have slope <= 1.13 and 32 roundings of
their own.  The output's rounding is half a step of its type."""
import numpy as np
import pytest
import torch

import bit_diffusion_amd as bd
import synth
from oracle import batch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DEV = "cuda:0"


def bf16(rng, shape, scale=1.0):
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)
    return t


def f64(t):
    return t.double().numpy()


class Case:
    def __init__(self, seed, M, K, N, R, starts, ids, ranks=None, bf=True, act=0, S=3, base=True, xpad=0, opad=0, shift=0):
        rng = np.random.default_rng(seed)
        self.M, self.K, self.N, self.R, self.S, self.act, self.bf = M, K, N, R, S, act, bf
        self.starts, self.ids = list(starts), list(ids)
        self.ranks = None if ranks is None else list(ranks)
        self.x, self.down, self.up = bf16(rng, (M, K)), bf16(rng, (S, R, K), K ** -0.5), bf16(rng, (S, N, R), 0.2)
        self.alphas = torch.from_numpy(rng.uniform(0.5, 1.5, S).astype(np.float32))
        dt = torch.bfloat16 if bf else torch.float32
        self.dt = dt
        self.base = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(dt) if base else None
        self.out = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(dt)
        self.xpad, self.opad, self.shift = xpad, opad, shift
        self.put()

    def wide(self, t, pad, fill):
        """t on the device as columns [shift, shift + n) of rows pad elements longer."""
        w = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype)
        w[:, self.shift:self.shift + t.shape[1]] = t
        w = w.to(DEV)
        return w, w[:, self.shift:self.shift + t.shape[1]]

    def put(self):
        self.dx = torch.full((self.M, self.K + self.xpad), float("nan"), dtype=torch.bfloat16)
        self.dx[:, :self.K] = self.x
        self.dx = self.dx.to(DEV)
        self.ddown, self.dup, self.dalphas = self.down.to(DEV), self.up.to(DEV), self.alphas.to(DEV)
        self.dstarts = torch.tensor(self.starts, dtype=torch.int32, device=DEV)
        self.dids = torch.tensor(self.ids, dtype=torch.int32, device=DEV)
        self.dranks = None if self.ranks is None else torch.tensor(self.ranks, dtype=torch.int32, device=DEV)
        self.wbase, self.dbase = (None, None) if self.base is None else self.wide(self.base, self.opad, 7.0)
        self.wout, self.dout = self.wide(self.out, self.opad, 9.0)
        self.nb = bd.svdq_lora_batch_workspace_bytes(self.M, self.K, self.N, self.R, len(self.ids))
        self.ws = torch.full((max(self.nb, 16),), 0xFF, dtype=torch.uint8, device=DEV)   # NaN words

    def call(self, out=None, base=None, stream=None, ws=None):
        out = self.dout if out is None else out
        base = self.dbase if base is None else base
        bd.svdq_lora_batch(self.M, self.K, self.N, self.R, self.S, len(self.ids), self.dx, self.K + self.xpad,
                           self.ddown, self.dup, self.dalphas, self.dranks, self.dstarts, self.dids, base,
                           self.N + self.opad, self.act, bd.SVDQ_DT_BF16 if self.bf else bd.SVDQ_DT_F32, out,
                           self.N + self.opad, self.ws if ws is None else ws, self.nb, stream=stream)
        return out

    def ref(self, out=None):
        down, up = f64(self.down), f64(self.up)
        ranks = [self.R] * self.S if self.ranks is None else [min(max(r, 0), self.R) for r in self.ranks]
        return batch.lora_batch(f64(self.x), down, up, f64(self.alphas), ranks, self.starts, self.ids,
                                None if self.base is None else f64(self.base), self.act,
                                f64(self.out if out is None else out))

    def check(self, got, ref=None):
        res, y, T, D = self.ref() if ref is None else ref
        got = f64(got.cpu())
        split, half = (2.0 ** -16, 2.0 ** -8) if self.bf else (2.0 ** -24, 2.0 ** -24)
        b = np.abs(f64(self.base)) if self.base is not None else 0.0
        e = 2 * (self.K + 16) * U * D + (split + 2 * (3 * self.R + 4) * U) * T + 4 * U * (b + np.abs(y))
        if self.act:
            e = 1.13 * e + 32 * U * np.abs(y)
        tol = e + half * (np.abs(res) + e) + 1e-37
        bad = np.abs(got - res) > tol
        assert not bad.any(), (int(bad.sum()), float((np.abs(got - res) / tol).max()), np.argwhere(bad)[:5])


def cuts(*lens, first=0):
    return list(np.cumsum([first] + list(lens)))


CASES = {
    "one row": dict(M=1, K=64, N=1, R=16, starts=[0, 1], ids=[1]),
    "one row, wide": dict(M=1, K=192, N=1000, R=16, starts=[0, 1], ids=[2], bf=False),
    "two rows, rank 128": dict(M=2, K=1024, N=513, R=128, starts=[0, 1, 2], ids=[2, 0]),
    "one row a segment": dict(M=70, K=320, N=130, R=32, starts=list(range(71)), ids=[i % 4 - 1 for i in range(70)], bf=False),
    "ragged, empty ones": dict(M=150, K=256, N=200, R=16, starts=cuts(0, 17, 0, 0, 33, 1, 64, 16, 0), ids=[0, 1, 2, 0, -1, 2, 1, 0, 1]),
    "rows before and behind": dict(M=90, K=128, N=96, R=16, starts=cuts(20, 30, first=13), ids=[0, 2], act=1),
    "no adapter at all": dict(M=40, K=64, N=72, R=16, starts=[0, 40], ids=[-1], act=2),
    "index past the pool": dict(M=40, K=64, N=72, R=16, starts=[0, 20, 40], ids=[3, 1 << 30]),
    "mixed ranks": dict(M=100, K=448, N=260, R=64, starts=cuts(30, 30, 20, 20), ids=[0, 1, 2, 1], ranks=[1, 64, 19], bf=False),
    "ranks out of range": dict(M=60, K=128, N=64, R=48, starts=cuts(20, 20, 20), ids=[0, 1, 2], ranks=[-5, 1000, 41]),
    "rank 0": dict(M=33, K=64, N=65, R=16, starts=[0, 33], ids=[0], ranks=[0, 0, 0], act=1),
    "rank 48": dict(M=77, K=576, N=300, R=48, starts=cuts(40, 37), ids=[1, 0]),
    "rank 112, fp32": dict(M=77, K=576, N=300, R=112, starts=cuts(40, 37), ids=[1, 0], bf=False, act=2),
    "delta alone": dict(M=50, K=256, N=136, R=16, starts=cuts(25, 25), ids=[0, 1], base=False),
    "delta alone, fp32": dict(M=50, K=256, N=131, R=16, starts=cuts(25, 25), ids=[0, 1], base=False, bf=False, act=1),
    "padded rows": dict(M=65, K=192, N=256, R=32, starts=cuts(33, 32), ids=[0, 1], xpad=64, opad=64),
    "columns of a wider matrix": dict(M=65, K=192, N=250, R=32, starts=cuts(33, 32), ids=[0, 1], xpad=8, opad=37, shift=5, bf=False),
    "odd columns, bf16": dict(M=65, K=192, N=251, R=16, starts=cuts(1, 64), ids=[2, 1], opad=6, shift=3, act=2),
    "more than 64 segments": dict(M=300, K=64, N=40, R=16, starts=cuts(*([3] * 99 + [3])), ids=[i % 3 for i in range(100)]),
    "64 rows exactly": dict(M=64, K=64, N=256, R=16, starts=[0, 64], ids=[0]),
    "tall tiles": dict(M=8300, K=128, N=1030, R=32, starts=cuts(4100, 1, 4190), ids=[0, 1, 2]),
    "tall tiles, rank 128, fp32": dict(M=8200, K=64, N=1100, R=128, starts=cuts(63, 65, 8000, 72), ids=[0, 1, 2, 0], bf=False, act=1),
    "wide, 32 rows": dict(M=4100, K=192, N=72, R=64, starts=cuts(2000, 33, 0, 2067), ids=[0, 1, 2, 2], ranks=[64, 3, 40], act=1),
    "wide, 32 rows, rank 128": dict(M=4200, K=320, N=40, R=128, starts=cuts(1, 4000, 150, first=9), ids=[0, 1, 2], ranks=[128, 64, 17], bf=False),
    "wide, 64 rows": dict(M=9000, K=448, N=56, R=64, starts=cuts(63, 65, 8000, 872), ids=[0, 1, 2, 0], ranks=[48, 64, 64]),
    "wide, 64 rows, rank 128": dict(M=9001, K=320, N=130, R=128, starts=cuts(4500, 4501), ids=[0, 1], ranks=[128, 100, 7]),
    "wide, 96 rows": dict(M=17000, K=128, N=48, R=64, starts=cuts(95, 97, 16000, 700), ids=[0, -1, 2, 0], bf=False),
    "wide, 96 rows, rank 128": dict(M=16600, K=256, N=40, R=128, starts=cuts(8000, 0, 8500, 90), ids=[0, 1, 2, 1], ranks=[128, 1, 64]),
    "wide, more than one round": dict(M=33000, K=64, N=33, R=48, starts=cuts(33000), ids=[1]),
    "many one-row segments, rank 64": dict(M=300, K=128, N=140, R=64, starts=list(range(301)), ids=[i % 4 - 1 for i in range(300)], ranks=[64, 12, 33]),
    "many one-row segments, rank 128, fp32": dict(M=300, K=256, N=270, R=128, starts=list(range(301)), ids=[i % 3 for i in range(300)], bf=False),
    "two rank blocks": dict(M=4500, K=128, N=80, R=32, starts=cuts(4500), ids=[1]),
    "whole lines, rank 16": dict(M=8200, K=64, N=2060, R=16, starts=cuts(4000, 4200), ids=[0, 1], act=2),
    "whole lines, rank 16, fp32": dict(M=8200, K=64, N=1028, R=16, starts=cuts(4000, 4200), ids=[0, 1], bf=False),
    "whole lines, rank 64": dict(M=8200, K=64, N=2060, R=64, starts=cuts(4000, 4200), ids=[0, 1], ranks=[64, 30, 1]),
    "whole lines, rank 32, fp32": dict(M=8200, K=64, N=1027, R=32, starts=cuts(4000, 4200), ids=[0, 1], bf=False, act=1),
    "whole lines, rank 64, fp32": dict(M=8200, K=64, N=1028, R=64, starts=cuts(8200), ids=[2], bf=False),
    "32 rows, rank 128": dict(M=8200, K=64, N=1100, R=128, starts=cuts(4000, 4200), ids=[0, 1], ranks=[128, 64, 1], act=1),
    "long K": dict(M=20, K=12288, N=64, R=16, starts=cuts(7, 13), ids=[0, 1], bf=False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_fp64(name):
    c = Case(len(name) * 31 + 7, **CASES[name])
    print("lora_batch", name, flush=True)
    if c.ranks is not None:      # whatever stands past an adapter's rank is not used
        for s, r in enumerate(c.ranks):
            r = min(max(r, 0), c.R)
            c.ddown[s, r:] = float("nan")
            c.dup[s, :, r:] = float("inf")
    got = c.call()
    torch.cuda.synchronize()
    c.check(got)
    if c.opad:                   # nothing beside the columns is written
        w = c.wout.clone()
        w[:, c.shift:c.shift + c.N] = 9.0
        assert bool((w == 9.0).all())
    first = got.clone()
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(got, first), "another run gives other bits"


def test_untouched_rows_and_unused_values():
    """NaN in rows of no segment, in adapters no segment uses and in rows without adapter stay
    where they are."""
    c = Case(3, 60, 128, 96, 16, cuts(10, 12, 20, first=5), [0, -1, 2])
    ref = c.ref()
    c.dx[:5] = float("nan")
    c.dx[47:] = float("inf")
    c.dx[15:27] = float("nan")          # rows without adapter
    c.ddown[1] = float("nan")
    c.dup[1] = float("inf")
    c.dalphas[1] = float("nan")
    got = c.call()
    torch.cuda.synchronize()
    c.check(got, ref)
    assert torch.equal(got[:5].cpu(), c.out[:5]) and torch.equal(got[47:].cpu(), c.out[47:])


@pytest.mark.parametrize("bf,act,N", [(True, 0, 264), (False, 1, 131)])
def test_in_place(bf, act, N):
    c = Case(11, 100, 256, N, 16, cuts(40, 30, 20, first=4), [0, -1, 1], bf=bf, act=act)
    want = c.call().clone()
    buf = c.base.to(DEV)
    bd.svdq_lora_batch(c.M, c.K, c.N, c.R, c.S, 3, c.dx, c.K, c.ddown, c.dup, c.dalphas, None, c.dstarts, c.dids,
                       buf, N, act, bd.SVDQ_DT_BF16 if bf else bd.SVDQ_DT_F32, buf, N, c.ws, c.nb)
    torch.cuda.synchronize()
    want[:4], want[94:] = c.base[:4].to(DEV), c.base[94:].to(DEV)
    assert torch.equal(buf, want)


def test_zero_sizes():
    c = Case(12, 8, 64, 40, 16, [0, 8], [0])
    before = c.dout.clone()
    bd.svdq_lora_batch(0, 64, 40, 16, 3, 1, c.dx, 64, c.ddown, c.dup, c.dalphas, None, c.dstarts, c.dids, c.dbase, 40,
                       0, 1, c.dout, 40, None, 0)
    bd.svdq_lora_batch(8, 64, 40, 16, 3, 0, c.dx, 64, c.ddown, c.dup, c.dalphas, None, c.dstarts, c.dids, c.dbase, 40,
                       0, 1, c.dout, 40, None, 0)
    torch.cuda.synchronize()
    assert torch.equal(c.dout, before)


def test_large_values_and_infinities():
    """t beyond bf16's largest value stays finite where the result is; an infinite x row is
    infinite or NaN in its own row alone."""
    c = Case(13, 32, 64, 48, 16, [0, 16, 32], [0, 1], bf=False)
    c.x[:, :] = 0
    c.x[:, 0] = 1.0
    c.down[:] = 0
    c.down[:, 0, 0] = 3.3895e38          # bf16's largest
    c.up[:] = 0
    c.up[:, :, 0] = 2.0 ** -120
    c.alphas[:] = torch.tensor([1.0009765, 0.999, 1.0])
    c.base[:] = 0
    c.put()
    got = c.call().cpu().double().numpy()
    ref = c.ref()[0]
    assert np.isfinite(got).all()
    assert np.abs(got - ref).max() <= 2.0 ** -20 * np.abs(ref).max()
    c2 = Case(14, 32, 64, 48, 16, [0, 16, 32], [0, 1], bf=True)
    ref2 = c2.ref()
    c2.dx[5, 3] = float("inf")
    got2 = c2.call()
    torch.cuda.synchronize()
    assert not bool(torch.isfinite(got2[5]).any())
    keep = [i for i in range(32) if i != 5]
    got2[5] = 0
    ref2[0][5] = 0
    c2.check(got2, ref2)
    assert bool(torch.isfinite(got2[keep]).all())


def test_graph_replays_with_new_segments():
    """A captured call replays with what the segment arrays, x and base hold then."""
    c = Case(20, 200, 256, 300, 32, cuts(50, 80, 40, 20), [0, 1, 2, 0])
    c.call()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            c.call(stream=side)
    torch.cuda.synchronize()
    for k, (starts, ids) in enumerate(((cuts(50, 80, 40, 20), [0, 1, 2, 0]), (cuts(0, 1, 190, 3), [1, 2, 0, -1]),
                                       (cuts(7, 7, 7, 7, first=60), [2, 2, -1, 1]))):
        c.starts, c.ids = starts, ids
        c.dstarts.copy_(torch.tensor(starts, dtype=torch.int32))
        c.dids.copy_(torch.tensor(ids, dtype=torch.int32))
        c.dout.copy_(c.out)
        c.ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = c.dout.clone()
        c.check(got)
        c.dout.copy_(c.out)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(c.dout, got), k


def test_two_streams_with_their_own_workspaces():
    cs = [Case(30 + i, 500, 256, 384, 16, cuts(200, 300), [i, 2]) for i in range(2)]
    want = [c.call().clone() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for c, st in zip(cs, streams):
            c.dout.copy_(c.out)
        torch.cuda.synchronize()
        for c, st in zip(cs, streams):
            c.call(stream=st)
        torch.cuda.synchronize()
        for c, w in zip(cs, want):
            assert torch.equal(c.dout, w)


@pytest.mark.parametrize("starts", [[0, 30, 10, 50], [-(1 << 31), (1 << 31) - 1, -7, 50], [90, 80, 70, 60], [0, 1 << 30, 1 << 30, 1 << 30]])
def test_offsets_that_break_the_rules_stay_inside(starts):
    """Offsets out of range or decreasing are clamped: only the rows the clamped segments name
    are written, and everything around the matrices keeps its value."""
    c = Case(40, 64, 64, 96, 16, [0, 16, 32, 64], [0, 1, -1], opad=8)
    c.dstarts.copy_(torch.tensor(starts, dtype=torch.int32))
    c.call()
    torch.cuda.synchronize()
    lim = [min(max(v, 0), 64) for v in starts]
    rows = set()
    for a, b in zip(lim, lim[1:]):
        rows |= set(range(a, b))
    rest = [r for r in range(64) if r not in rows]
    assert torch.equal(c.dout.cpu()[rest], c.out[rest])
    w = c.wout.clone()
    w[:, :96] = 9.0
    assert bool((w == 9.0).all())


def far(t, stride):
    """t's rows `stride` elements apart in a buffer of 2^31 elements or more."""
    buf = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype, device=DEV)
    assert buf.numel() > 1 << 31
    view = buf.as_strided(t.shape, (stride, 1))
    view.copy_(t)
    return view


# rows and pool entries whose offsets pass 2^31 elements give what near ones give, bit for bit
@pytest.mark.parametrize("M,K,N,R", [(40, 64, 72, 16), (600, 128, 130, 64), (4200, 64, 40, 64)])
def test_offsets_past_32_bits(M, K, N, R):
    c = Case(70 + R, M, K, N, R, cuts(M // 3, M - M // 3), [0, 2])
    want = c.call().clone()
    stride = ((1 << 31) // (M - 1) // 8 + 1) * 8
    x, base, out = (far(t.to(DEV), stride) for t in (c.x, c.base, c.out))
    bd.svdq_lora_batch(M, K, N, R, c.S, 2, x, x.stride(0), c.ddown, c.dup, c.dalphas, None, c.dstarts, c.dids, base,
                       stride, 0, bd.SVDQ_DT_BF16, out, stride, c.ws, c.nb)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_pools_past_32_bits():
    S, R, K, N = 4200, 128, 4096, 4096
    c = Case(71, 40, K, N, R, cuts(15, 25), [0, 1], S=2)
    want = c.call().clone()
    down = torch.empty(S, R, K, dtype=torch.bfloat16, device=DEV)
    up = torch.empty(S, N, R, dtype=torch.bfloat16, device=DEV)
    assert down.numel() > 1 << 31 and up.numel() > 1 << 31
    alphas = torch.empty(S, dtype=torch.float32, device=DEV)
    for i, s in ((0, S - 1), (1, S - 2)):
        down[s], up[s], alphas[s] = c.ddown[i], c.dup[i], c.dalphas[i]
    c.ddown, c.dup, c.dalphas, c.S = down, up, alphas, S
    c.dids = torch.tensor([S - 1, S - 2], dtype=torch.int32, device=DEV)
    got = c.call(out=c.out.to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(got, want)
