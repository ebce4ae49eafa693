"""svdq_layer_norm, svdq_rotary and svdq_attention at the limits that their contract names: most rows,
segments, heads and columns."""
import pytest
import torch

import bit_diffusion_amd as bd
from oracle import packed

pytestmark = pytest.mark.gpu
U, DEV, BF = 2.0 ** -24, "cuda:0", torch.bfloat16


def rnd(*shape, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * scale).to(BF)


def test_layer_norm_at_2_30_rows_and_2_16_segments():
    """One column: the norm of a value by itself is 0, so a row gives its segment's shift."""
    M, n = 1 << 30, 1 << 16
    x = torch.zeros(M, dtype=BF, device=DEV)
    out = torch.full((M,), 7.0, dtype=BF, device=DEV)
    shift = rnd(n, 1)
    starts = (torch.arange(n + 1, device=DEV) * (M // n - 1) + 5).to(torch.int32)
    bd.svdq_layer_norm(M, 1, n, 1e-6, 1, x, 1, 1, None, 1, None, None, starts, 1, None, None, shift, 1, None, 1, 1, out, 1)
    torch.cuda.synchronize()
    assert bool((out[:5] == 7.0).all()) and bool((out[int(starts[-1]):] == 7.0).all())
    got = out[5:int(starts[-1])].reshape(n, -1)
    assert torch.equal(got, shift.expand_as(got))


def test_layer_norm_at_16384_columns():
    x = rnd(3, 16384, seed=1)
    out = torch.empty(3, 16384, dtype=torch.float32, device=DEV)
    bd.svdq_layer_norm(3, 16384, 1, 1e-6, 1, x, 16384, 1, None, 0, None, None, None, 0, None, None, None, 0, None, 0, 0, out, 16384)
    torch.cuda.synchronize()
    _, ref, _ = packed.layer_norm(x.double(), None, None, None, torch.zeros(3, dtype=torch.long, device=DEV), None, None, None, 1e-6)
    assert bool(((out.double() - ref).abs() <= 200 * U * (1 + ref.abs())).all())


def test_rotary_at_2_24_rows():
    """One pair a row: (1, 0) turned by the row's angle."""
    M = 1 << 24
    x = torch.zeros(M, 2, device=DEV)
    x[:, 0] = 1.0
    pos = torch.arange(M, dtype=torch.float32, device=DEV)
    f = torch.full((1,), 0.1, dtype=torch.float64, device=DEV)
    bd.svdq_rotary(M, 1, 0, 2, [1], bd.SVDQ_ROTARY_INTERLEAVED, pos, 1, f, 0.0, None, None, 0, x, 2, None, 0, 0, x, 2, None, 0)
    torch.cuda.synchronize()
    angle = pos.double() * 0.1
    assert bool(((x[:, 0].double() - torch.cos(angle)).abs() <= 1e-6).all())
    assert bool(((x[:, 1].double() - torch.sin(angle)).abs() <= 1e-6).all())


@pytest.mark.parametrize("D", [2, 8])
def test_rotary_at_2_16_heads(D):
    H, M = 1 << 16, 3
    x = rnd(M, 2 * H * D, seed=2)
    out = torch.empty(M, 2 * H * D, dtype=torch.float32, device=DEV)
    pos = torch.tensor([[0.0], [1.5], [-3.0]], device=DEV)
    f = torch.linspace(0.3, 1.0, D // 2, dtype=torch.float64, device=DEV)
    bd.svdq_rotary(M, H, H, D, [D // 2], bd.SVDQ_ROTARY_HALVES, pos, 1, f, 0.0, None, None, 1, x, 2 * H * D, x[:, H * D:], 2 * H * D, 0,
                   out, 2 * H * D, out[:, H * D:], 2 * H * D)
    torch.cuda.synchronize()
    ref, size, _ = packed.rotary(x.double(), 2 * H, torch.zeros(D // 2, dtype=torch.long, device=DEV), pos.double(), f, None, 0.0, True)
    assert bool(((out.double() - ref).abs() <= 13 * U * size + 1e-37).all())


def test_attention_at_2_16_segments():
    """A row and a key each, but for empty ones: the row gives its key's value."""
    n, D = 1 << 16, 8
    starts = torch.arange(n + 1, device=DEV, dtype=torch.int32)
    starts[1000:2000] = 1000              # empty ones, then 1001 rows in one
    q, k, v = (rnd(n, D, seed=s) for s in (3, 4, 5))
    out = torch.full((n, D), 9.0, dtype=BF, device=DEV)
    nb = bd.svdq_attention_workspace_bytes(n, n, 1, 1, D, n)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=DEV)
    bd.svdq_attention(n, n, 1, 1, D, n, 1.0, 0.0, 0, starts, starts, None, None, q, D, k, D, v, D, out, D, ws, nb)
    torch.cuda.synchronize()
    alone = torch.ones(n, dtype=torch.bool, device=DEV)
    alone[1000:2000] = False
    assert torch.equal(out[alone], v[alone])
    ref, wabs, _, _, _ = packed.attention(q[1000:2000].double(), k[1000:2000].double(), v[1000:2000].double(), 1.0, 0.0, False, 0, None)
    assert bool(((out[1000:2000].double() - ref).abs() <= 2.0 ** -7 * wabs + 2.0 ** -8 * ref.abs()).all())


@pytest.mark.parametrize("G", [1, 1 << 15])
def test_attention_at_2_16_heads(G):
    H, D, M, Mk = 1 << 16, 8, 3, 70
    q, k, v = rnd(M, H * D, seed=6), rnd(Mk, G * D, seed=7), rnd(Mk, G * D, seed=8)
    out = torch.empty(M, H * D, dtype=BF, device=DEV)
    qs, ks = (torch.tensor([0, m], dtype=torch.int32, device=DEV) for m in (M, Mk))
    nb = bd.svdq_attention_workspace_bytes(M, Mk, H, G, D, 1)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=DEV)
    bd.svdq_attention(M, Mk, H, G, D, 1, 0.5, 0.0, bd.SVDQ_MASK_CAUSAL, qs, ks, None, None, q, H * D, k, G * D, v, G * D, out, H * D, ws, nb)
    torch.cuda.synchronize()
    for h in (0, 1, 127, 128, 40000, H - 1):
        g = h * G // H * D
        ref, wabs, _, _, _ = packed.attention(q[:, h * D:h * D + D].double(), k[:, g:g + D].double(), v[:, g:g + D].double(), 0.5, 0.0, True, 0, None)
        assert bool(((out[:, h * D:h * D + D].double() - ref).abs() <= 2.0 ** -7 * wabs + 2.0 ** -8 * ref.abs()).all()), h


def test_attention_at_most_rows_times_heads():
    """2^24 rows of one head, in segments of 256 whose keys are all alike."""
    n, D = 1 << 16, 8
    M = n * 256
    starts = (torch.arange(n + 1, device=DEV) * 256).to(torch.int32)
    ks = (torch.arange(n + 1, device=DEV) * 3).to(torch.int32)
    q, k = rnd(M, D, seed=9), rnd(3 * n, D, seed=10)
    v = rnd(n, D, seed=11).repeat_interleave(3, dim=0)
    out = torch.empty(M, D, dtype=BF, device=DEV)
    assert bd.svdq_attention_workspace_bytes(M, 3 * n, 1, 1, D, n) == 0
    bd.svdq_attention(M, 3 * n, 1, 1, D, n, 1.0, 0.0, 0, starts, ks, None, None, q, D, k, D, v, D, out, D, None, 0)
    torch.cuda.synchronize()
    want = v[::3].double()
    assert bool(((out.reshape(n, 256, D).double() - want[:, None]).abs() <= 2.0 ** -7 * want.abs()[:, None]).all())
