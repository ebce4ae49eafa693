"""Argument rules of svdq_lora_batch and svdq_group_norm, checked without a GPU: every bad
argument is refused before any device is touched, and the workspace sizes."""
import ctypes

import pytest
import torch

import bit_diffusion_amd as bd

FAKE = 1 << 20
INV, UNS = bd.SVDQ_ERR_INVALID_ARG, bd.SVDQ_ERR_UNSUPPORTED_CONFIG


def _lora(**kw):
    a = dict(M=5, K=128, N=100, R=16, S=2, n=3, x=FAKE, xs=128, down=FAKE, up=FAKE, alphas=FAKE, ranks=None,
             starts=FAKE, ids=FAKE, base=FAKE, bs=100, act=0, dt=0, out=FAKE, os=100, ws=FAKE, wb=1 << 30)
    a.update(kw)
    return bd.lib().svdq_lora_batch(a["M"], a["K"], a["N"], a["R"], a["S"], a["n"], a["x"], a["xs"], a["down"],
                                    a["up"], a["alphas"], a["ranks"], a["starts"], a["ids"], a["base"], a["bs"],
                                    a["act"], a["dt"], a["out"], a["os"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), INV, "M"), (dict(M=(1 << 26) + 1), UNS, "too large"), (dict(K=100), INV, "K"), (dict(K=0), INV, "K"),
    (dict(N=0), INV, "N"), (dict(R=0), INV, "max_rank"), (dict(R=24), INV, "max_rank"),
    (dict(R=144), UNS, "max_rank"), (dict(S=0), INV, "n_adapters"), (dict(n=-1), INV, "n_segments"),
    (dict(n=(1 << 20) + 1), UNS, "n_segments"), (dict(n=(1 << 16) + 1), UNS, "n_segments"),
    (dict(K=(1 << 24) + 64, xs=1 << 25), UNS, "K"), (dict(M=(1 << 22) + 1), UNS, "too large"),
    (dict(M=1 << 22, N=1 << 13, bs=1 << 13, os=1 << 13), UNS, "too large"),
    (dict(N=(1 << 31) - 1, bs=1 << 31, os=1 << 31), UNS, "too large"), (dict(x=None), INV, "x is NULL"), (dict(x=FAKE + 8), INV, "aligned"),
    (dict(xs=120), INV, "x_stride"), (dict(xs=132), INV, "x_stride"), (dict(down=None), INV, "lora_down"),
    (dict(up=FAKE + 4), INV, "lora_up"), (dict(alphas=None), INV, "alphas"), (dict(ranks=FAKE + 2), INV, "ranks"),
    (dict(starts=None), INV, "seg_start"), (dict(ids=None), INV, "seg_adapter"), (dict(base=FAKE + 2), INV, "base"),
    (dict(bs=99), INV, "base_stride"), (dict(bs=104), INV, "base_stride"), (dict(act=3), INV, "act"),
    (dict(dt=2), INV, "out_dtype"), (dict(out=None), INV, "out"), (dict(os=99), INV, "out_stride"),
    (dict(ws=None), INV, "workspace"), (dict(ws=FAKE + 8), INV, "workspace"), (dict(wb=16), INV, "workspace"),
])
def test_lora_batch_refuses(kw, status, word):
    assert _lora(**kw) == status
    assert word in bd.svdq_last_error()


def _norm(**kw):
    a = dict(B=2, rows=9, C=64, G=8, eps=1e-5, xd=1, x=FAKE, xs=64, w=None, b=None, md=0, ms=FAKE, mt=FAKE, mst=64,
             act=2, od=1, out=2 * FAKE, os=64, ws=FAKE, wb=1 << 30)
    a.update(kw)
    return bd.lib().svdq_group_norm(a["B"], a["rows"], a["C"], a["G"], a["eps"], a["xd"], a["x"], a["xs"], a["w"],
                                    a["b"], a["md"], a["ms"], a["mt"], a["mst"], a["act"], a["od"], a["out"],
                                    a["os"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(B=-1), INV, "B"), (dict(B=65536), UNS, "too large"), (dict(rows=-1), INV, "rows"),
    (dict(rows=(1 << 30) + 1), UNS, "too large"), (dict(C=0), INV, "C"), (dict(G=0), INV, "groups"),
    (dict(G=7), INV, "groups"), (dict(C=65544, xs=65544, os=65544), UNS, "C"), (dict(eps=0.0), INV, "eps"),
    (dict(eps=float("nan")), INV, "eps"), (dict(xd=2), INV, "x_dtype"), (dict(md=5), INV, "mod_dtype"),
    (dict(od=-1), INV, "out_dtype"), (dict(act=3), INV, "act"), (dict(x=None), INV, "x is NULL"),
    (dict(x=FAKE + 1), INV, "aligned"), (dict(xs=63), INV, "x_stride"), (dict(w=FAKE + 1), INV, "weight"),
    (dict(b=FAKE + 1), INV, "bias"), (dict(ms=FAKE + 2), INV, "mod_scale"), (dict(mt=FAKE + 2), INV, "mod_shift"),
    (dict(mst=63), INV, "mod_stride"), (dict(out=None), INV, "out"), (dict(os=0), INV, "out_stride"),
    (dict(out=FAKE, od=0), INV, "x is out"), (dict(out=FAKE, os=72), INV, "x is out"),
    (dict(ws=FAKE + 4), INV, "workspace"), (dict(rows=100000, wb=8), INV, "workspace"),
])
def test_group_norm_refuses(kw, status, word):
    assert _norm(**kw) == status
    assert word in bd.svdq_last_error()


def test_existing_calls_do_not_take_silu():
    cfg = bd.LayerCfg.make(128, 64, 16)
    assert bd.lib().svdq_gemm_w4a4(ctypes.byref(cfg), 4, FAKE, FAKE, 1.0, FAKE, FAKE, 1.0, FAKE, FAKE, None,
                                   bd.SVDQ_ACT_SILU, 0, FAKE, None) == INV


def test_workspace_queries():
    assert bd.svdq_lora_batch_workspace_bytes(0, 128, 64, 16, 4) == 0
    assert bd.svdq_lora_batch_workspace_bytes(100, 128, 64, 16, 0) == 0
    one = bd.svdq_lora_batch_workspace_bytes(16384, 128, 64, 32, 4)
    assert one >= 16384 * 32 * 4
    with pytest.raises(bd.SvdqError):
        bd.svdq_lora_batch_workspace_bytes(-1, 128, 64, 16, 4)
    assert bd.svdq_group_norm_workspace_bytes(0, 10, 64, 8) == 0
    assert bd.svdq_group_norm_workspace_bytes(2, 0, 64, 8) == 0
    assert bd.svdq_group_norm_workspace_bytes(2, 1 << 20, 64, 8) >= 2 * 8 * 8
    with pytest.raises(bd.SvdqError):
        bd.svdq_group_norm_workspace_bytes(1, 10, 64, 7)
    n = ctypes.c_int64(0)
    assert bd.lib().svdq_lora_batch_workspace_bytes(4, 128, 64, 16, 4, None) == INV
    assert bd.lib().svdq_group_norm_workspace_bytes(4, 128, 64, 16, None) == INV
    assert n.value == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros(1024)
    with pytest.raises(bd.SvdqError) as e:
        bd.svdq_group_norm(1, 1, 64, 8, 1e-5, 0, t, 64, None, None, 0, None, None, 64, 0, 0, t, 64, FAKE, 1024, stream=0)
    assert "x is on cpu" in e.value.message
    with pytest.raises(bd.SvdqError) as e:
        bd.svdq_lora_batch(1, 64, 8, 16, 1, 1, FAKE, 64, FAKE, FAKE, t, None, FAKE, FAKE, None, 0, 0, 0, FAKE, 8,
                           FAKE, 1 << 20, stream=0)
    assert "alphas is on cpu" in e.value.message
