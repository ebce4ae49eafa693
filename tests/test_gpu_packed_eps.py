"""svdq_layer_norm and svdq_rotary at the smallest eps their contract takes, subnormal ones among them:
rows without variance give exactly their offset, heads of zeros zeros, others their norm."""
import pytest
import torch

import bit_diffusion_amd as bd
from oracle import packed

pytestmark = pytest.mark.gpu
U, DEV = 2.0 ** -24, "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
EPS = [2.0 ** -149, 1e-42, 1e-40, 1.1e-38, 2.0 ** -126, 1e-30]


@pytest.mark.parametrize("C", [1, 63, 122, 1170, 2048, 9000])
@pytest.mark.parametrize("eps", EPS)
def test_layer_norm(eps, C):
    """Rows 0 to 3 hold one value each, rows 4 and 5 values 2^-50 and 1 apart."""
    print("eps", eps, C, flush=True)
    g = torch.Generator().manual_seed(C)
    x = torch.empty(6, C)
    x[0], x[1], x[2], x[3] = 0.0, 1.0, -3e4, 1e-20
    x[4:] = torch.randint(-1, 2, (2, C), generator=g).float()
    x[4] *= 2.0 ** -50
    x = x.to(DEV)
    shift, scale = (torch.randn(1, C, generator=g).to(DEV) for _ in range(2))
    out = torch.full((6, C), 9.0, device=DEV)
    bd.svdq_layer_norm(6, C, 1, eps, 0, x, C, 0, None, 0, None, None, None, 0, None, scale, shift, C, None, 0, 0, out, C)
    torch.cuda.synchronize()
    assert torch.equal(out[:4], shift.expand(4, C))
    _, ref, p = packed.layer_norm(x.double(), None, None, None, torch.zeros(6, dtype=torch.long, device=DEV), None,
                                  scale.double(), shift.double(), eps)
    # the relative errors of test_gpu_layer_norm's bound: 80 additions in a row's sum, 10 roundings
    size = (p["d"].abs() + p["d"].abs().amax(1, keepdim=True)) * p["rstd"] * p["A"].abs() + p["Dabs"]
    assert bool(((out.double() - ref).abs() <= 200 * U * size).all())


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("D,halves", [(64, False), (128, True), (90, False), (6, True)])
@pytest.mark.parametrize("xd", [BF, F32])
def test_rotary(eps, D, halves, xd):
    """Rows 0 and 1 are zeros, row 2 holds numbers near 2^-50, row 3 near 1."""
    print("eps", eps, D, halves, flush=True)
    g = torch.Generator().manual_seed(D)
    H, G = 3, 2
    x = torch.randn(4, (H + G) * D, generator=g)
    x[:2] = 0.0
    x[2] *= 2.0 ** -50
    x = x.to(xd).to(DEV)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(BF).to(DEV) for _ in range(2)]
    pos = torch.tensor([[0.0], [2.0], [-1.5], [7.0]], device=DEV)
    f = torch.linspace(0.1, 1.0, D // 2, dtype=torch.float64, device=DEV)
    out = torch.full((4, (H + G) * D), 9.0, device=DEV)
    wide = (H + G) * D
    bd.svdq_rotary(4, H, G, D, [D // 2], bd.SVDQ_ROTARY_HALVES if halves else bd.SVDQ_ROTARY_INTERLEAVED, pos, 1, f, eps, *w,
                   bd.SVDQ_DT_BF16 if xd == BF else bd.SVDQ_DT_F32, x, wide, x[:, H * D:], wide, bd.SVDQ_DT_F32, out, wide,
                   out[:, H * D:], wide)
    torch.cuda.synchronize()
    assert bool((out[:2] == 0.0).all())
    axis = torch.zeros(D // 2, dtype=torch.long, device=DEV)
    for a, n, wt in ((0, H, w[0]), (H * D, G, w[1])):
        ref, size, _ = packed.rotary(x[:, a:a + n * D].double(), n, axis, pos.double(), f, wt.double(), eps, halves)
        got = out[:, a:a + n * D].double()
        # the sum of squares 40 roundings, half of which pass the root; 13 for the rest
        assert bool(((got - ref).abs() <= 40 * U * size).all())
