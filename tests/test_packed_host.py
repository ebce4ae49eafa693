"""Argument rules of svdq_layer_norm, svdq_rotary and svdq_attention, checked without a GPU: every bad
argument is refused before any device is touched, and the workspace sizes."""
import ctypes

import pytest
import torch

import bit_diffusion_amd as bd

FAKE = 1 << 20
INV, UNS = bd.SVDQ_ERR_INVALID_ARG, bd.SVDQ_ERR_UNSUPPORTED_CONFIG


def _layer(**kw):
    a = dict(M=5, C=64, n=2, eps=1e-6, xd=1, x=FAKE, xs=64, yd=1, y=2 * FAKE, ys=64, w=FAKE, b=FAKE, st=FAKE, md=0, g=FAKE, s=FAKE,
             t=FAKE, ms=64, xo=3 * FAKE, xos=64, od=1, out=4 * FAKE, os=64)
    a.update(kw)
    return bd.lib().svdq_layer_norm(a["M"], a["C"], a["n"], a["eps"], a["xd"], a["x"], a["xs"], a["yd"], a["y"], a["ys"], a["w"],
                                    a["b"], a["st"], a["md"], a["g"], a["s"], a["t"], a["ms"], a["xo"], a["xos"], a["od"], a["out"],
                                    a["os"], None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), INV, "M"), (dict(M=(1 << 30) + 1), UNS, "too large"), (dict(C=0), INV, "C"), (dict(C=-4), INV, "C"),
    (dict(C=16388, xs=16388), UNS, "C"), (dict(n=-1), INV, "n_segments"), (dict(n=(1 << 16) + 1), UNS, "n_segments"),
    (dict(eps=0.0), INV, "eps"), (dict(eps=float("inf")), INV, "eps"), (dict(eps=float("nan")), INV, "eps"), (dict(xd=2), INV, "x_dtype"),
    (dict(yd=-1), INV, "y_dtype"), (dict(md=3), INV, "mod_dtype"), (dict(od=9), INV, "out_dtype"), (dict(x=None), INV, "x is NULL"),
    (dict(x=FAKE + 1), INV, "x is not"), (dict(xs=63), INV, "x_stride"), (dict(y=FAKE + 1), INV, "y is not"), (dict(ys=0), INV, "y_stride"),
    (dict(y=None), INV, "y is NULL"), (dict(y=None, xo=None), INV, "mod_gate"), (dict(y=None, g=None), INV, "x_out"),
    (dict(w=FAKE + 1), INV, "weight"), (dict(b=FAKE + 1), INV, "bias"), (dict(st=None), INV, "seg_start"), (dict(st=FAKE + 2), INV, "seg_start"),
    (dict(g=FAKE + 2), INV, "mod_gate"), (dict(s=FAKE + 2), INV, "mod_scale"), (dict(t=FAKE + 2), INV, "mod_shift"),
    (dict(ms=63), INV, "mod_stride"), (dict(xo=FAKE + 1), INV, "x_out"), (dict(xos=63), INV, "x_out_stride"),
    (dict(xo=FAKE, xos=72), INV, "x_out is x"), (dict(xo=2 * FAKE, yd=0), INV, "x_out is y"), (dict(xo=2 * FAKE, ys=72), INV, "x_out is y"),
    (dict(xo=4 * FAKE), INV, "x_out is out"), (dict(out=None), INV, "out is NULL"), (dict(out=FAKE + 1), INV, "out is not"),
    (dict(os=63), INV, "out_stride"), (dict(out=FAKE, od=0), INV, "out is x"), (dict(out=FAKE, os=72), INV, "out is x"),
    (dict(out=2 * FAKE, od=0), INV, "out is y"), (dict(out=2 * FAKE, os=72), INV, "out is y"),
    (dict(C=8193, xs=8193, ys=8193, ms=8193, xos=8193, os=8193), UNS, "8192"),
    (dict(C=8196, xs=8197, ys=8196, ms=8196, xos=8196, os=8196), UNS, "8192"),
    (dict(C=8196, xs=8196, ys=8196, ms=8196, xos=8196, os=8196, w=FAKE + 2), UNS, "8192"),
])
def test_layer_norm_refuses(kw, status, word):
    assert _layer(**kw) == status
    assert word in bd.svdq_last_error()


def _rotary(**kw):
    a = dict(M=5, H=4, G=2, D=64, axes=[8, 12, 12], n=None, pr=0, pos=FAKE, ps=3, f=FAKE, eps=1e-6, qw=FAKE, kw=FAKE, xd=1, q=FAKE,
             qs=512, k=2 * FAKE, ks=512, od=1, qo=3 * FAKE, qos=256, ko=4 * FAKE, kos=128)
    a.update(kw)
    ax = None if a["axes"] is None else (ctypes.c_int32 * len(a["axes"]))(*a["axes"])
    n = a["n"] if a["n"] is not None else len(a["axes"])
    return bd.lib().svdq_rotary(a["M"], a["H"], a["G"], a["D"], n, ax, a["pr"], a["pos"], a["ps"], a["f"], a["eps"], a["qw"], a["kw"],
                                a["xd"], a["q"], a["qs"], a["k"], a["ks"], a["od"], a["qo"], a["qos"], a["ko"], a["kos"], None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), INV, "M"), (dict(M=(1 << 24) + 1), UNS, "too large"), (dict(H=-1), INV, "n_q_heads"), (dict(G=-2), INV, "n_k_heads"),
    (dict(H=(1 << 16) + 1), UNS, "too large"), (dict(D=0), INV, "head_dim"), (dict(D=63), INV, "head_dim"), (dict(D=258, axes=[129]), UNS, "head_dim"),
    (dict(axes=[32], n=0), INV, "n_axes"), (dict(axes=[8, 8, 8, 4, 4]), UNS, "n_axes"), (dict(axes=None, n=1), INV, "axis_pairs"),
    (dict(axes=[40, -8]), INV, "axis_pairs"), (dict(axes=[8, 12, 11]), INV, "axis_pairs"), (dict(axes=[2 ** 31 - 1, 2 ** 31 - 1]), INV, "axis_pairs"),
    (dict(pr=2), INV, "pairing"), (dict(pos=None), INV, "positions"), (dict(pos=FAKE + 2), INV, "positions"), (dict(ps=2), INV, "pos_stride"),
    (dict(f=None), INV, "freqs"), (dict(f=FAKE + 4), INV, "freqs"), (dict(qw=FAKE + 1), INV, "q_weight"), (dict(kw=FAKE + 1), INV, "k_weight"),
    (dict(eps=0.0), INV, "eps"), (dict(eps=float("nan"), qw=None), INV, "eps"), (dict(xd=5), INV, "x_dtype"), (dict(od=-1), INV, "out_dtype"),
    (dict(q=None), INV, "q is NULL"), (dict(q=FAKE + 1), INV, "q is not"), (dict(qs=255), INV, "q_stride"), (dict(k=None), INV, "k is NULL"),
    (dict(ks=127), INV, "k_stride"), (dict(qo=None), INV, "q_out"), (dict(qos=255), INV, "q_out_stride"), (dict(ko=FAKE + 1), INV, "k_out"),
    (dict(kos=0), INV, "k_out_stride"), (dict(qo=FAKE), INV, "q_out is q"), (dict(ko=2 * FAKE, kos=512, od=0), INV, "k_out is k"),
])
def test_rotary_refuses(kw, status, word):
    assert _rotary(**kw) == status
    assert word in bd.svdq_last_error()


def _attn(**kw):
    a = dict(Mq=5, Mk=7, H=4, G=2, D=64, n=2, scale=0.125, cap=0.0, mask=0, qs=FAKE, ks=FAKE, pf=None, sl=None, q=FAKE, qst=256, k=FAKE,
             kst=128, v=FAKE, vst=128, out=2 * FAKE, ost=256, ws=None, wb=0)
    a.update(kw)
    return bd.lib().svdq_attention(a["Mq"], a["Mk"], a["H"], a["G"], a["D"], a["n"], a["scale"], a["cap"], a["mask"], a["qs"], a["ks"],
                                   a["pf"], a["sl"], a["q"], a["qst"], a["k"], a["kst"], a["v"], a["vst"], a["out"], a["ost"], a["ws"],
                                   a["wb"], None)


LONG = dict(Mk=1 << 16)      # few rows over many keys: these take a workspace


@pytest.mark.parametrize("kw,status,word", [
    (dict(Mq=-1), INV, "Mq"), (dict(Mk=-1), INV, "Mkv"), (dict(H=0), INV, "n_heads"), (dict(G=0), INV, "n_kv_heads"), (dict(G=3), INV, "n_heads"),
    (dict(H=(1 << 16) + 2), UNS, "n_heads"), (dict(D=0), INV, "head_dim"), (dict(D=60), INV, "head_dim"), (dict(D=136), UNS, "head_dim"),
    (dict(n=-1), INV, "n_segments"), (dict(n=(1 << 16) + 1), UNS, "n_segments"), (dict(Mq=(1 << 24) + 1), UNS, "too large"),
    (dict(Mq=1 << 23), UNS, "too large"), (dict(Mk=(1 << 30) + 1), UNS, "too large"), (dict(scale=0.0), INV, "scale"),
    (dict(scale=-1.0), INV, "scale"), (dict(scale=float("nan")), INV, "scale"), (dict(cap=-1.0), INV, "cap"), (dict(cap=float("inf")), INV, "cap"),
    (dict(mask=2), INV, "mask"), (dict(pf=FAKE), INV, "prefix"), (dict(mask=1, pf=FAKE + 2), INV, "prefix"), (dict(qs=None), INV, "q_start"),
    (dict(ks=FAKE + 2), INV, "kv_start"), (dict(sl=FAKE + 1), INV, "slopes"), (dict(q=None), INV, "q is NULL"), (dict(q=FAKE + 8), INV, "q is not"),
    (dict(qst=248), INV, "q_stride"), (dict(qst=260), INV, "q_stride"), (dict(qst=(1 << 24) + 8), UNS, "q_stride"), (dict(k=None), INV, "k is NULL"),
    (dict(kst=120), INV, "k_stride"), (dict(kst=(1 << 24) + 8), UNS, "k_stride"), (dict(v=FAKE + 2), INV, "v is not"), (dict(vst=0), INV, "v_stride"),
    (dict(vst=1 << 40), UNS, "v_stride"), (dict(out=None), INV, "out"), (dict(ost=255), INV, "out_stride"), (dict(ost=258), INV, "out_stride"),
    (dict(ws=FAKE + 8), INV, "workspace"), (dict(LONG), INV, "workspace"), (dict(LONG, ws=FAKE, wb=64), INV, "workspace"),
])
def test_attention_refuses(kw, status, word):
    assert _attn(**kw) == status
    assert word in bd.svdq_last_error()


def test_workspace_queries():
    f = bd.svdq_attention_workspace_bytes
    assert f(0, 0, 4, 2, 64, 0) == 0 and f(4608, 4608, 24, 24, 128, 1) == 0 and f(1, 100, 24, 24, 128, 1) == 0
    for n in (1, 8, 40):
        one = f(n, 20000, 8, 2, 72, n)
        assert one > 0 and one % (n * 8 * (72 + 2) * 4) == 0
    for Mq, Mk, H, G, D, n in ((1 << 24, 1 << 30, 1, 1, 8, 1 << 16), (1, 1 << 30, 1 << 16, 1, 128, 1), (1 << 9, 1 << 30, 1 << 16, 1 << 16 >> 1, 128, 1)):
        try:
            assert 0 <= f(Mq, Mk, H, G, D, n) < 1 << 32
        except bd.SvdqError as e:
            assert e.status == UNS
    with pytest.raises(bd.SvdqError):
        f(-1, 0, 4, 2, 64, 1)
    assert bd.lib().svdq_attention_workspace_bytes(1, 1, 1, 1, 8, 1, None) == INV


def test_binding_refuses_host_tensors():
    t = torch.zeros(1024)
    with pytest.raises(bd.SvdqError) as e:
        bd.svdq_layer_norm(1, 8, 1, 1e-6, 0, FAKE, 8, 0, None, 0, None, None, None, 0, None, t, None, 8, None, 0, 0, FAKE, 8, stream=0)
    assert "mod_scale is on cpu" in e.value.message
    with pytest.raises(bd.SvdqError) as e:
        bd.svdq_rotary(1, 1, 1, 8, [4], 0, FAKE, 1, t, 0.0, None, None, 0, FAKE, 8, FAKE, 8, 0, FAKE, 8, FAKE, 8, stream=0)
    assert "freqs is on cpu" in e.value.message
    with pytest.raises(bd.SvdqError) as e:
        bd.svdq_attention(1, 1, 1, 1, 8, 1, 1.0, 0.0, 0, FAKE, t, None, None, FAKE, 8, FAKE, 8, FAKE, 8, FAKE, 8, None, 0, stream=0)
    assert "kv_start is on cpu" in e.value.message
