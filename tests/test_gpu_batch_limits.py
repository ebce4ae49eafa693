"""svdq_lora_batch and svdq_group_norm at the limits their documentation names, and with one of two
optional operands alone.  References in binary64 on the device, in plain two-dimensional products."""
import pytest
import torch

import bit_diffusion_amd as bd
from test_gpu_group_norm import BF, DEV, DT, F32
from test_gpu_group_norm import Case as Norm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("rows", [50, 12000])
@pytest.mark.parametrize("keep", ["weight", "bias", "scale", "shift"])
def test_one_optional_operand_alone(rows, keep):
    c = Norm(31, 2, rows, 64, 8, mod=BF, act=1)
    w, b, mod = c.dw, c.db, c.dmod
    bd.svdq_group_norm(c.B, rows, 64, 8, c.eps, DT[BF], c.wx, 64, w if keep == "weight" else None, b if keep == "bias" else None, DT[BF],
                       mod[:, :64] if keep == "scale" else None, mod[:, 67:] if keep == "shift" else None, 2 * 64 + 3, 1, DT[BF],
                       c.wo, 64, c.ws, c.nb)
    torch.cuda.synchronize()
    c.w = c.w if keep == "weight" else torch.ones_like(c.w)
    c.b = c.b if keep == "bias" else torch.zeros_like(c.b)
    c.mod = c.mod.clone()
    if keep != "scale":
        c.mod[:, :64] = 0
    if keep != "shift":
        c.mod[:, 67:] = 0
    c.check(c.wo)


# the most images: one launch, two launches, single elements
@pytest.mark.parametrize("rows,C,G,xd", [(1, 64, 8, BF), (3, 64, 8, BF), (1, 33, 3, F32), (5, 24, 3, F32)])
def test_most_images(rows, C, G, xd):
    c = Norm(32, 65535, rows, C, G, xd=xd, act=0)
    got = c.call()
    torch.cuda.synchronize()
    c.check(got)


def test_most_rows():
    """2^30 positions of one channel.  A thread's chain of joins is 2048 chunks long (2^30 rows over
    256 tiles of 256 threads, 8 rows a chunk), and the tiles' joins come on top: 2304 roundings of
    the mean and of the square sum, where the shorter cases count 256."""
    n, chain = 1 << 30, 2304
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.empty(n, dtype=BF, device=DEV)
    for part in x.split(1 << 27):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * 2 + 1)
    out = torch.empty_like(x)
    nb = bd.svdq_group_norm_workspace_bytes(1, n, 1, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    bd.svdq_group_norm(1, n, 1, 1, 1e-5, DT[BF], x, 1, None, None, 0, None, None, 1, 0, DT[BF], out, 1, ws, nb)
    torch.cuda.synchronize()
    parts = list(x.split(1 << 26))
    mean = sum(p.double().sum().item() for p in parts) / n
    var = sum(((p.double() - mean) ** 2).sum().item() for p in parts) / n
    big, rstd = max(p.abs().max().item() for p in parts), (var + 1e-5) ** -0.5
    dm = chain * U * big * rstd
    for p, o in zip(parts, out.split(1 << 26)):
        ref = (p.double() - mean) * rstd
        e = dm + ref.abs() * ((chain + 8) * U + dm * dm) + 8 * U * ref.abs()
        assert bool(((o.double() - ref).abs() <= e + 2.0 ** -8 * (ref.abs() + e)).all())


@pytest.mark.parametrize("n", [1, 3, 65536])
@pytest.mark.parametrize("R,bf", [(16, True), (64, False), (128, True)])
def test_most_rows_and_segments_of_adapters(n, R, bf):
    """M = 2^22 rows in one, few and the most segments."""
    print("adapters", n, R, bf, flush=True)
    M, K, N, S = 1 << 22, 64, 24, 2
    dt = BF if bf else F32
    g = torch.Generator(device=DEV).manual_seed(n + R)
    x = torch.randn(M, K, generator=g, device=DEV).to(BF)
    down, up = torch.randn(S, R, K, generator=g, device=DEV).to(BF) / 8, torch.randn(S, N, R, generator=g, device=DEV).to(BF) / 4
    alphas = torch.tensor([0.75, -1.25], device=DEV)
    base, out = (torch.randn(M, N, generator=g, device=DEV).to(dt) for _ in range(2))
    before = out.clone()
    starts = torch.linspace(5, M - 7, n + 1, device=DEV, dtype=torch.float64).round().to(torch.int32)
    ids = (torch.arange(n, device=DEV) % 3 - (1 if n > 1 else 0)).to(torch.int32)
    nb = bd.svdq_lora_batch_workspace_bytes(M, K, N, R, n)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    bd.svdq_lora_batch(M, K, N, R, S, n, x, K, down, up, alphas, None, starts, ids, base, N, 0, DT[dt], out, N, ws, nb)
    torch.cuda.synchronize()
    lens = (starts[1:] - starts[:-1]).long()
    row_id = torch.full((M,), -2, dtype=torch.long, device=DEV)
    row_id[5:M - 7] = torch.repeat_interleave(ids.long(), lens)
    for lo in range(0, M, 1 << 20):
        s = slice(lo, lo + (1 << 20))
        ref, T, D = base[s].double(), 0, 0
        for a in range(S):
            on = (row_id[s] == a).double()[:, None]
            A, B, al = down[a].double(), up[a].double(), alphas[a].double()
            t = al * (x[s].double() @ A.t().contiguous()) * on
            ref = ref + t @ B.t().contiguous()
            T = T + t.abs() @ B.abs().t().contiguous()
            D = D + (al.abs() * (x[s].double().abs() @ A.abs().t().contiguous()) * on) @ B.abs().t().contiguous()
        e = 2 * (K + 16) * U * D + (U + 2 * (3 * R + 4) * U) * T + 4 * U * (base[s].double().abs() + ref.abs())
        half = 2.0 ** -8 if bf else U
        ok = (out[s].double() - ref).abs() <= e + half * (ref.abs() + e) + 1e-37
        none = row_id[s] == -2
        assert bool(ok[~none].all()) and torch.equal(out[s][none], before[s][none])


# the most channels: one group in 128 parts, a group a channel, groups of an odd width in 205 parts
@pytest.mark.parametrize("B,rows,C,G,xd", [(1, 33, 65536, 1, BF), (2, 3, 65536, 65536, F32), (1, 700, 65536, 16384, BF), (1, 7, 65535, 5, F32)])
def test_most_channels(B, rows, C, G, xd):
    """Joins over the parts of a group come on top of the rows': 128 or 205 parts of 64 or more
    channels, each lane joins 4 of them at most, within the 256 roundings that the bound counts."""
    c = Norm(33, B, rows, C, G, xd=xd, act=2)
    got = c.call()
    torch.cuda.synchronize()
    c.check(got)


def test_longest_k():
    """K = 2^24: rows with three nonzeros, the first channel, one in the middle and the last, so that t
    is a sum of three exact products: 2 roundings, alpha's, three added products and the output's,
    8 u of the absolute sums in all."""
    M, K, N, R = 3, 1 << 24, 40, 16
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.zeros(M, K, dtype=BF, device=DEV)
    at = torch.tensor([0, (1 << 23) + 5, K - 1], device=DEV)
    x[:, at] = torch.randn(M, 3, generator=g, device=DEV).to(BF)
    down = torch.randn(1, R, K, generator=g, device=DEV, dtype=BF)
    up = torch.randn(1, N, R, generator=g, device=DEV).to(BF)
    alpha, out = torch.tensor([0.3], device=DEV), torch.zeros(M, N, device=DEV)
    starts, ids = torch.tensor([0, M], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    nb = bd.svdq_lora_batch_workspace_bytes(M, K, N, R, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    bd.svdq_lora_batch(M, K, N, R, 1, 1, x, K, down, up, alpha, None, starts, ids, None, 0, 0, DT[F32], out, N, ws, nb)
    torch.cuda.synchronize()
    xs, A, B = x[:, at].double(), down[0][:, at].double(), up[0].double()
    al = alpha.double()
    ref = (al * (xs @ A.t().contiguous())) @ B.t().contiguous()
    size = (al * (xs.abs() @ A.abs().t().contiguous())) @ B.abs().t().contiguous()
    # and the sums over 16 ranks, three terms each, counted twice
    assert bool(((out.double() - ref).abs() <= (8 + 2 * (3 * R + 4)) * U * size).all())


def test_widest_output():
    """N = 2^27: offsets in lora_up pass 2^31 elements.  Rank 1, so an element is base + t B."""
    M, K, N, R = 2, 64, 1 << 27, 16
    g = torch.Generator(device=DEV).manual_seed(9)
    x, down = torch.randn(M, K, generator=g, device=DEV).to(BF), torch.randn(1, R, K, generator=g, device=DEV).to(BF)
    up = torch.empty(1, N, R, dtype=BF, device=DEV)
    for part in up[0].split(1 << 24):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    alpha, ranks = torch.tensor([1.5], device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    base = torch.randn(M, N, generator=g, device=DEV).to(BF)
    out = torch.empty_like(base)
    starts, ids = torch.tensor([0, M], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    nb = bd.svdq_lora_batch_workspace_bytes(M, K, N, R, 1)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    bd.svdq_lora_batch(M, K, N, R, 1, 1, x, K, down, up, alpha, ranks, starts, ids, base, N, 0, DT[BF], out, N, ws, nb)
    torch.cuda.synchronize()
    t = 1.5 * (x.double() * down[0, 0].double()).sum(1)
    D = 1.5 * (x.double() * down[0, 0].double()).abs().sum(1)
    for lo in range(0, N, 1 << 24):
        s = slice(lo, lo + (1 << 24))
        B = up[0, s, 0].double()
        for m in range(M):
            ref = base[m, s].double() + t[m] * B
            e = (2 * (K + 16) * U * D[m] + 8 * U * t[m].abs()) * B.abs() + 4 * U * (base[m, s].double().abs() + ref.abs())
            assert bool(((out[m, s].double() - ref).abs() <= e + 2.0 ** -8 * (ref.abs() + e) + 1e-37).all())
