"""svdq_lora_batch as a server calls it, at sizes of two launches (narrow and wide down-projection, one
and several column blocks a workgroup) as well as one: in place, on a column range of a wider
matrix, both at once, captured and replayed with other segments, and two calls at a time."""
import pytest
import torch

import bit_diffusion_amd as bd
from test_gpu_lora_batch import DEV, Case, cuts

pytestmark = pytest.mark.gpu

# M, K, N, R, bf16 out: one launch; two; wide at ranks 64 and 128; several column blocks
SIZES = [(90, 192, 264, 16, True), (700, 128, 3000, 32, True), (700, 128, 1030, 64, False), (4300, 64, 520, 64, True),
         (8200, 64, 4100, 128, True), (8200, 64, 1028, 16, True), (5000, 64, 1028, 128, False)]


def case(M, K, N, R, bf, **kw):
    return Case(M + N + R, M, K, N, R, cuts(M // 4, M // 2, M - M // 4 - M // 2 - 3, first=2), [0, -1, 2], ranks=[R, 3, R - 5],
                bf=bf, **kw)


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("M,K,N,R,bf", SIZES)
def test_in_place_on_a_column_range(M, K, N, R, bf, act):
    """The middle third of a fused projection, updated in place, gives what a call beside it gives,
    bit for bit; the other two thirds and the rows of no segment stay."""
    print("in place", M, K, N, R, bf, act, flush=True)
    c = case(M, K, N, R, bf, act=act)
    want = c.call().clone()
    torch.cuda.synchronize()
    for left in (N, 3):          # aligned as the width is, and unaligned
        wide = torch.randn(M, 3 * N, generator=torch.Generator().manual_seed(1)).to(c.dt).to(DEV)
        wide[:, left:left + N] = c.base.to(DEV)
        before = wide.clone()
        mid = wide[:, left:]
        bd.svdq_lora_batch(M, K, N, R, c.S, 3, c.dx, K, c.ddown, c.dup, c.dalphas, c.dranks, c.dstarts, c.dids, mid, 3 * N, act,
                           bd.SVDQ_DT_BF16 if bf else bd.SVDQ_DT_F32, mid, 3 * N, c.ws, c.nb)
        torch.cuda.synchronize()
        lo, hi = c.starts[0], c.starts[-1]
        before[lo:hi, left:left + N] = want[lo:hi]
        assert torch.equal(wide, before)


@pytest.mark.parametrize("M,K,N,R,bf", SIZES)
def test_graph_replays_with_new_segments(M, K, N, R, bf):
    print("graph", M, K, N, R, bf, flush=True)
    c = case(M, K, N, R, bf)
    c.call()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            c.call(stream=side)
    torch.cuda.synchronize()
    for starts, ids in (([2, M // 3, M // 2, M], [0, 1, 2]), ([0, 0, M - 1, M - 1], [1, 2, 0]), ([5, 22, 23, M // 2], [-1, 0, 1])):
        c.dstarts.copy_(torch.tensor(starts, dtype=torch.int32))
        c.dids.copy_(torch.tensor(ids, dtype=torch.int32))
        c.dx.copy_(torch.randn(M, K, device=DEV).to(torch.bfloat16))
        c.dout.copy_(c.out)
        c.ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = c.dout.clone()
        c.x, c.starts, c.ids = c.dx.cpu(), starts, ids
        c.check(got)
        c.dout.copy_(c.out)
        c.ws.fill_(0xFF)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(c.dout, got)


@pytest.mark.parametrize("M,K,N,R,bf", SIZES)
def test_two_calls_at_a_time(M, K, N, R, bf):
    print("two calls", M, K, N, R, bf, flush=True)
    cs = [case(M, K, N, R, bf), case(M, K, N, R, bf, act=2)]
    cs[1].dx.mul_(2)
    want = [c.call().clone() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for c in cs:
            c.dout.copy_(c.out)
            c.ws.fill_(0xFF)
        torch.cuda.synchronize()
        for c, st in zip(cs, streams):
            c.call(stream=st)
        torch.cuda.synchronize()
        for c, w in zip(cs, want):
            assert torch.equal(c.dout, w)
