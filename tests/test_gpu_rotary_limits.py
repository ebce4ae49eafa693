"""svdq_rotary with its most rows and so many heads that a workgroup would take one row each."""
import pytest
import torch

import bit_diffusion_amd as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("M", [(1 << 23) + 1, 1 << 24])
def test_many_heads(M):
    """In place, pairs (1, 0) turned by the row's angle: (cos, sin), alike in all heads."""
    H = 256
    x = torch.zeros(M, H, 2, dtype=torch.bfloat16, device=DEV)
    x[..., 0] = 1.0
    pos = torch.arange(M, dtype=torch.float32, device=DEV)
    f = torch.full((1,), 0.1, dtype=torch.float64, device=DEV)
    bd.svdq_rotary(M, H, 0, 2, [1], bd.SVDQ_ROTARY_INTERLEAVED, pos, 1, f, 0.0, None, None, bd.SVDQ_DT_BF16, x, 2 * H, None, 0,
                   bd.SVDQ_DT_BF16, x, 2 * H, None, 0)
    torch.cuda.synchronize()
    angle = pos.double() * 0.1
    want = torch.stack([torch.cos(angle), torch.sin(angle)], dim=1)
    # the fp32 result is within 2^-22, its rounding to bf16 within 2^-8 of it
    assert bool(((x[:, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -21).all())
    for a in range(0, M, 1 << 20):
        rows = x[a:a + (1 << 20)]
        assert bool((rows == rows[:, :1]).all())
