"""The batched operators as they are used together, on one stream: the modulation layer of a batch
of requests (AWQ GEMV) with each request's adapter on its row, its scale and shift rows into the
group norm of the requests' images, the norm's output through the 4-bit linear (packed activation
kernel and GEMM), and each request's adapter on that linear's output.  Every step is compared with
its own fp64 form on the step's actual inputs, and the whole run captured and replayed."""
import numpy as np
import pytest
import torch

import bit_diffusion_amd as bd
import oracle
import synth
from oracle import batch

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")
DEV, BF, F32 = "cuda:0", bd.SVDQ_DT_BF16, bd.SVDQ_DT_F32


def bf(bits):
    return gu.dev(bits).view(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


class Block:
    """Three requests: B images of 8 x 9 positions, C channels, N outputs, adapters of ranks 16 and
    5 in a pool of four; the third request has none."""

    def __init__(self):
        rng = np.random.default_rng(77)
        self.B, self.rows, self.C, self.G, self.N, self.r, self.R, self.S, self.T = 3, 72, 320, 32, 448, 32, 16, 4, 256
        B, C, N, T, M = self.B, self.C, self.N, self.T, self.B * self.rows
        self.M = M
        self.cond = bf(synth.random_bf16(rng, (B, T), 1.0))
        self.q = synth.random_packed_nibbles(rng, 2 * C, T)
        self.qs, self.qz = synth.random_bf16(rng, (2 * C, T // 64), 0.02), np.full((2 * C, T // 64), 0x4100, np.uint16)
        self.alphas = torch.tensor([0.5, 1.0, -0.75, 2.0], device=DEV)
        self.ranks = torch.tensor([16, 5, 16, 1], dtype=torch.int32, device=DEV)
        self.ids = torch.tensor([2, 1, -1], dtype=torch.int32, device=DEV)
        self.one = torch.arange(B + 1, dtype=torch.int32, device=DEV)
        self.many = self.one * self.rows
        self.md, self.mu = bf(synth.random_bf16(rng, (4, 16, T), 0.05)), bf(synth.random_bf16(rng, (4, 2 * C, 16), 0.05))
        self.xd, self.xu = bf(synth.random_bf16(rng, (4, 16, C), 0.05)), bf(synth.random_bf16(rng, (4, N, 16), 0.2))
        self.x = bf(synth.random_bf16(rng, (M, C), 2.0))
        self.w, self.b = bf(synth.random_bf16(rng, (C,), 1.0)), bf(synth.random_bf16(rng, (C,), 0.2))
        self.si = rng.uniform(0.5, 2.0, C).astype(np.float32)
        self.l1, self.l2 = synth.random_bf16(rng, (self.r, C), 0.05), synth.random_bf16(rng, (N, self.r), 0.1)
        self.wc = synth.random_packed_nibbles(rng, N, C)
        self.ws = rng.uniform(0.001, 0.05, (N, C // 64)).astype(np.float32)
        self.bias = synth.random_bf16(rng, (N,), 0.3)
        self.dq, self.dqs, self.dqz, self.dsi = gu.dev(self.q), gu.dev(self.qs), gu.dev(self.qz), gu.dev(self.si)
        self.l1p, self.wpk = gu.prepack_l1(self.l1, C), gu.prepack(self.wc, self.ws, C, N)
        self.dl2, self.dbias = gu.dev(self.l2), gu.dev(self.bias)
        self.cfg = bd.LayerCfg.make(C, N, self.r)
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=DEV)   # noqa: E731
        self.mod0, self.mod = e((B, 2 * C), torch.float32), e((B, 2 * C), torch.float32)
        self.h = e((M, C), torch.bfloat16)
        self.apk = e(bd.svdq_act_packed_bytes(self.cfg, M), torch.uint8)
        self.sc, self.lora = e((M, C // 64), torch.float32), e((M, self.r), torch.int16)
        self.y0, self.y = e((M, N), torch.bfloat16), e((M, N), torch.bfloat16)
        sizes = (bd.svdq_lora_batch_workspace_bytes(B, T, 2 * C, 16, B), bd.svdq_group_norm_workspace_bytes(B, self.rows, C, self.G),
                 bd.svdq_lora_batch_workspace_bytes(M, C, N, 16, B))
        self.nb = max(sizes)
        self.work = e(self.nb, torch.uint8)      # steps of one stream share it

    def run(self, stream=None):
        B, C, N, T, M = self.B, self.C, self.N, self.T, self.M
        bd.awq_gemm_w4a16(B, T, 2 * C, 64, self.cond, self.dq, self.dqs, self.dqz, None, F32, self.mod0, stream)
        bd.svdq_lora_batch(B, T, 2 * C, 16, self.S, B, self.cond, T, self.md, self.mu, self.alphas, self.ranks, self.one,
                           self.ids, self.mod0, 2 * C, bd.SVDQ_ACT_NONE, F32, self.mod, 2 * C, self.work, self.nb, stream)
        bd.svdq_group_norm(B, self.rows, C, self.G, 1e-5, BF, self.x, C, self.w, self.b, F32, self.mod, self.mod[:, C:],
                           2 * C, bd.SVDQ_ACT_SILU, BF, self.h, C, self.work, self.nb, stream)
        bd.svdq_quantize_act_packed(self.cfg, M, self.h, self.dsi, self.l1p, self.apk, self.sc, self.lora, stream)
        bd.svdq_gemm_w4a4_packed(self.cfg, M, self.apk, self.wpk, self.lora, self.dl2, self.dbias, bd.SVDQ_ACT_NONE, BF,
                                 self.y0, stream)
        bd.svdq_lora_batch(M, C, N, 16, self.S, B, self.h, C, self.xd, self.xu, self.alphas, self.ranks, self.many,
                           self.ids, self.y0, N, bd.SVDQ_ACT_GELU_TANH, BF, self.y, N, self.work, self.nb, stream)


def test_a_block_of_batched_requests():
    k = Block()
    k.run()
    torch.cuda.synchronize()
    ids, ranks, one, many = k.ids.tolist(), k.ranks.tolist(), k.one.tolist(), k.many.tolist()
    # the modulation rows: the AWQ oracle on the same inputs, then the adapters
    ref0 = gu.host(k.mod0).astype(np.float64)
    want = batch.lora_batch(f64(k.cond), f64(k.md), f64(k.mu), f64(k.alphas), ranks, one, ids, ref0, 0, np.zeros_like(ref0))[0]
    assert gu.rel_fro(f64(k.mod), want) <= 1e-6
    # the norm on the modulation as computed: half a bf16 step, and as much again for its arithmetic
    mod = f64(k.mod)
    hn, _ = batch.group_norm(f64(k.x).reshape(k.B, k.rows, k.C), k.G, 1e-5, f64(k.w), f64(k.b), mod[:, :k.C],
                             mod[:, k.C:], 2)
    h = f64(k.h).reshape(hn.shape)
    assert (np.abs(h - hn) <= 2.0 ** -7 * np.abs(hn) + 1e-4).all()
    # the 4-bit linear's codes and scales, bit for bit, and its output
    hb = k.h.view(torch.int16).cpu().numpy().view(np.uint16)
    oc, os_, ol = oracle.quant_act_int4(hb, k.si, k.l1)
    assert np.array_equal(gu.host(k.sc), os_)
    ref = oracle.gemm_w4a4_int4(oc, os_, k.wc, k.ws, ol, k.l2, k.bias)
    assert gu.rel_fro(f64(k.y0), ref) <= 2.0 ** -8
    # the adapters on top
    want = batch.lora_batch(f64(k.h), f64(k.xd), f64(k.xu), f64(k.alphas), ranks, many, ids, f64(k.y0), 1,
                            np.zeros((k.M, k.N)))[0]
    assert gu.rel_fro(f64(k.y), want) <= 2.0 ** -8


def test_the_block_captured_and_replayed():
    k = Block()
    k.run()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            k.run(side)
    torch.cuda.synchronize()
    for i in range(3):
        k.x.copy_(torch.randn(k.M, k.C, device=DEV).to(torch.bfloat16))
        k.ids.copy_(torch.tensor([[0, 1, 2], [-1, 3, 3], [2, -1, 0]][i], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = k.y.clone()
        k.y.zero_()
        k.work.fill_(0xFF)
        k.run()
        torch.cuda.synchronize()
        assert torch.equal(k.y, got), i
