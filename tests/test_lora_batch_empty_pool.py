"""svdq_lora_batch with an empty pool (a server that holds no adapter yet): every segment is
without adapter, whatever its index, out = act(base)."""
import pytest
import torch

import bit_diffusion_amd as bd
from oracle import batch
from test_batch_host import INV, _lora

EMPTY = dict(S=0, down=None, up=None, alphas=None)


@pytest.mark.parametrize("kw", [dict(), dict(ranks=None), dict(M=300, R=128)])
def test_taken(kw):
    assert _lora(**EMPTY, **kw) in (bd.SVDQ_OK, bd.SVDQ_ERR_UNSUPPORTED_DEVICE), bd.svdq_last_error()


@pytest.mark.parametrize("kw", [dict(EMPTY, S=-1), dict(EMPTY, S=1), dict(S=0, up=None, alphas=None), dict(S=0, down=None, alphas=None),
                                dict(S=0, down=None, up=None)])
def test_refused(kw):
    assert _lora(**kw) == INV
    assert any(w in bd.svdq_last_error() for w in ("n_adapters", "lora_down"))


# one launch; two; one row a segment at the highest rank
@pytest.mark.gpu
@pytest.mark.parametrize("M,N,R,starts", [(50, 200, 16, [0, 20, 50]), (5000, 1030, 64, [0, 17, 4000, 4990]), (90, 300, 128, list(range(91)))])
@pytest.mark.parametrize("bf,act,inplace", [(True, 2, False), (False, 0, False), (True, 1, True), (False, 0, True)])
def test_out_is_the_activated_base(M, N, R, starts, bf, act, inplace):
    print("empty pool", M, N, R, bf, act, inplace, flush=True)
    dev, dt = "cuda:0", torch.bfloat16 if bf else torch.float32
    g = torch.Generator().manual_seed(M)
    base, before = torch.randn(M, N, generator=g).to(dt), torch.randn(M, N, generator=g).to(dt)
    x = torch.full((M, 64), float("nan"), dtype=torch.bfloat16, device=dev)
    n = len(starts) - 1
    ids = torch.tensor([(0, -1, 1 << 30)[i % 3] for i in range(n)], dtype=torch.int32, device=dev)
    none = torch.empty(0, R, 64, dtype=torch.bfloat16, device=dev)
    nb = bd.svdq_lora_batch_workspace_bytes(M, 64, N, R, n)
    work = torch.empty(max(nb, 16), dtype=torch.uint8, device=dev)
    db = base.to(dev)
    out = db if inplace else before.to(dev)
    bd.svdq_lora_batch(M, 64, N, R, 0, n, x, 64, none, none, none.float(), None, torch.tensor(starts, dtype=torch.int32, device=dev), ids,
                       db, N, act, bd.SVDQ_DT_BF16 if bf else bd.SVDQ_DT_F32, out, N, work, nb)
    torch.cuda.synchronize()
    got, lo, hi = out.cpu(), starts[0], starts[-1]
    rest = base if inplace else before
    assert torch.equal(got[:lo], rest[:lo]) and torch.equal(got[hi:], rest[hi:])
    want = torch.from_numpy(batch.act(base[lo:hi].double().numpy(), act))
    # the activation's 32 roundings (2^-24 each) and half a step of the output
    tol = want.abs() * ((32 * 2.0 ** -24 if act else 0) + (2.0 ** -8 if bf and act else 0)) + 1e-37
    assert bool(((got[lo:hi].double() - want).abs() <= tol).all())
