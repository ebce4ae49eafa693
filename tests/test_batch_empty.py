"""svdq_lora_batch and svdq_group_norm on empty batches, as tensors bring them: a tensor without
elements has the address NULL."""
import pytest
import torch

import bit_diffusion_amd as bd
from test_batch_host import FAKE, INV, _lora, _norm

PASSED = (bd.SVDQ_OK, bd.SVDQ_ERR_UNSUPPORTED_DEVICE)     # the arguments were taken; a GPU may be missing


@pytest.mark.parametrize("kw", [dict(M=0, x=None, base=None, out=None, ws=None, wb=0), dict(n=0, ids=None, ws=None, wb=0),
                                dict(M=0, n=0, x=None, base=None, out=None, ids=None, ws=None, wb=0)])
def test_lora_batch_takes_null_for_empty_buffers(kw):
    assert _lora(**kw) in PASSED, bd.svdq_last_error()


@pytest.mark.parametrize("kw,word", [(dict(M=0, x=None, starts=None), "seg_start"), (dict(n=0, x=None), "x is NULL"),
                                     (dict(M=0, x=FAKE + 8), "aligned"), (dict(M=0, out=None, ids=None), "seg_adapter")])
def test_lora_batch_still_needs_the_others(kw, word):
    assert _lora(**kw) == INV
    assert word in bd.svdq_last_error()


@pytest.mark.parametrize("kw", [dict(B=0, x=None, out=None, ms=None, mt=None, ws=None, wb=0), dict(rows=0, x=None, out=None, ws=None, wb=0)])
def test_group_norm_takes_null_for_empty_buffers(kw):
    assert _norm(**kw) in PASSED, bd.svdq_last_error()


def test_group_norm_still_needs_the_others():
    assert _norm(B=0, x=FAKE + 1) == INV
    assert _norm(out=None) == INV


@pytest.mark.gpu
def test_empty_tensors():
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda:0")   # noqa: E731
    i32 = torch.int32
    down, up, al = e(3, 16, 64), e(3, 40, 16), e(3, dt=torch.float32)
    for M, n in ((0, 2), (0, 0), (5, 0)):
        x, base, out = e(M, 64), e(M, 40), torch.full((M, 40), 5.0, dtype=torch.bfloat16, device="cuda:0")
        nb = bd.svdq_lora_batch_workspace_bytes(M, 64, 40, 16, n)
        assert nb == 0
        bd.svdq_lora_batch(M, 64, 40, 16, 3, n, x, 64, down, up, al, None, torch.zeros(n + 1, dtype=i32, device="cuda:0"),
                           e(n, dt=i32), base, 40, bd.SVDQ_ACT_GELU_TANH, bd.SVDQ_DT_BF16, out, 40, e(nb, dt=torch.uint8), nb)
        torch.cuda.synchronize()
        assert bool((out == 5.0).all())
    for B, rows in ((0, 9), (2, 0), (0, 0)):
        x, mod = e(B * rows, 64), e(B, 128)
        nb = bd.svdq_group_norm_workspace_bytes(B, rows, 64, 8)
        bd.svdq_group_norm(B, rows, 64, 8, 1e-5, bd.SVDQ_DT_BF16, x, 64, None, None, bd.SVDQ_DT_BF16, mod[:, :64], mod[:, 64:], 128,
                           bd.SVDQ_ACT_SILU, bd.SVDQ_DT_BF16, e(B * rows, 64), 64, e(nb, dt=torch.uint8), nb)
    torch.cuda.synchronize()
