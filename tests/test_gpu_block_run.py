"""A transformer block's attention half as a packed batch of requests runs it, on one stream: the
modulation layer (AWQ GEMV), the modulated layer norm, the q, k, v linear in 4 bits, rotary positions
with the q and k norm, attention within each request, the output linear in 4 bits, and its result
through the gate onto the residual stream with the next norm.  Every step is compared with its own
fp64 form on the step's actual inputs, and the whole run captured and replayed with other cuts."""
import numpy as np
import pytest
import torch

import bit_diffusion_amd as bd
import oracle
import synth
from oracle import packed

pytestmark = pytest.mark.gpu
gu = pytest.importorskip("gpu_util")
DEV, BF, F32 = "cuda:0", bd.SVDQ_DT_BF16, bd.SVDQ_DT_F32


def bf(bits):
    return gu.dev(bits).view(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu()


class Linear:
    def __init__(self, rng, K, N, r=16):
        self.K, self.N, self.cfg = K, N, bd.LayerCfg.make(K, N, r)
        self.si = rng.uniform(0.5, 2.0, K).astype(np.float32)
        self.l1, self.l2 = synth.random_bf16(rng, (r, K), 0.05), synth.random_bf16(rng, (N, r), 0.05)
        self.wc, self.ws = synth.random_packed_nibbles(rng, N, K), rng.uniform(0.001, 0.02, (N, K // 64)).astype(np.float32)
        self.bias = synth.random_bf16(rng, (N,), 0.1)
        self.dsi, self.l1p, self.wpk = gu.dev(self.si), gu.prepack_l1(self.l1, K), gu.prepack(self.wc, self.ws, K, N)
        self.dl2, self.dbias = gu.dev(self.l2), gu.dev(self.bias)

    def buffers(self, M):
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=DEV)   # noqa: E731
        self.M, self.apk = M, e(bd.svdq_act_packed_bytes(self.cfg, M), torch.uint8)
        self.sc, self.lora = e((M, self.K // 64), torch.float32), e((M, self.cfg.rank), torch.int16)
        self.out = e((M, self.N), torch.bfloat16)
        return self

    def run(self, x, stream):
        bd.svdq_quantize_act_packed(self.cfg, self.M, x, self.dsi, self.l1p, self.apk, self.sc, self.lora, stream)
        bd.svdq_gemm_w4a4_packed(self.cfg, self.M, self.apk, self.wpk, self.lora, self.dl2, self.dbias, bd.SVDQ_ACT_NONE, BF, self.out,
                                 stream)

    def check(self, x):
        xb = x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
        oc, os_, ol = oracle.quant_act_int4(xb, self.si, self.l1)
        assert np.array_equal(gu.host(self.sc), os_)
        ref = oracle.gemm_w4a4_int4(oc, os_, self.wc, self.ws, ol, self.l2, self.bias)
        assert gu.rel_fro(f64(self.out).numpy(), ref) <= 2.0 ** -8


class Block:
    """Three requests of 8 x 9, 5 x 7 and 1 x 1 positions behind 6, 3 and 0 text rows, 4 heads of 64 over
    2 of k and v, 256 channels; rows behind the last request."""

    def __init__(self):
        rng = np.random.default_rng(91)
        self.n, self.H, self.G, self.D, self.T = 3, 4, 2, 64, 128
        self.C = C = self.H * self.D
        self.M, M, n, T = 130, 130, self.n, self.T
        self.cuts = [0, 78, 116, 117]
        self.start = torch.tensor(self.cuts, dtype=torch.int32, device=DEV)
        self.cond = bf(synth.random_bf16(rng, (n, T), 1.0))
        self.q = synth.random_packed_nibbles(rng, 5 * C, T)
        self.dq = gu.dev(self.q)
        self.dqs, self.dqz = gu.dev(synth.random_bf16(rng, (5 * C, T // 64), 0.02)), gu.dev(np.full((5 * C, T // 64), 0x4100, np.uint16))
        self.qkv = Linear(rng, C, (self.H + 2 * self.G) * self.D).buffers(M)
        self.proj = Linear(rng, C, C).buffers(M)
        self.x = bf(synth.random_bf16(rng, (M, C), 2.0))
        self.qw, self.kw = bf(synth.random_bf16(rng, (self.D,), 1.0)), bf(synth.random_bf16(rng, (self.D,), 1.0))
        self.pairs = [8, 12, 12]
        self.freqs = torch.cat([10000.0 ** (-torch.arange(p, dtype=torch.float64) / p) for p in self.pairs]).to(DEV)
        self.pos = torch.randint(0, 40, (M, 3), generator=torch.Generator().manual_seed(3)).float().to(DEV)
        e = lambda shape, dt=torch.bfloat16: torch.full(shape, 7.0, dtype=dt, device=DEV)   # noqa: E731
        self.mod = e((n, 5 * C), torch.float32)      # scale | shift | gate | scale | shift
        self.h, self.qr, self.kr, self.att = e((M, C)), e((M, C)), e((M, self.G * self.D)), e((M, C))
        self.x2, self.h2 = e((M, C)), e((M, C))
        self.nb = bd.svdq_attention_workspace_bytes(M, M, self.H, self.G, self.D, n)
        self.ws = torch.empty(max(self.nb, 16), dtype=torch.uint8, device=DEV)

    def run(self, stream=None):
        M, C, n, H, G, D = self.M, self.C, self.n, self.H, self.G, self.D
        w = (H + 2 * G) * D
        bd.awq_gemm_w4a16(n, self.T, 5 * C, 64, self.cond, self.dq, self.dqs, self.dqz, None, F32, self.mod, stream)
        m = [self.mod[:, i * C:] for i in range(5)]
        bd.svdq_layer_norm(M, C, n, 1e-6, BF, self.x, C, BF, None, C, None, None, self.start, F32, None, m[0], m[1], 5 * C, None, C, BF,
                           self.h, C, stream)
        self.qkv.run(self.h, stream)
        o = self.qkv.out
        bd.svdq_rotary(M, H, G, D, self.pairs, bd.SVDQ_ROTARY_INTERLEAVED, self.pos, 3, self.freqs, 1e-6, self.qw, self.kw, BF, o, w,
                       o[:, H * D:], w, BF, self.qr, C, self.kr, G * D, stream)
        bd.svdq_attention(M, M, H, G, D, n, D ** -0.5, 0.0, bd.SVDQ_MASK_NONE, self.start, self.start, None, None, self.qr, C, self.kr,
                          G * D, o[:, (H + G) * D:], w, self.att, C, self.ws, self.nb, stream)
        self.proj.run(self.att, stream)
        bd.svdq_layer_norm(M, C, n, 1e-6, BF, self.x, C, BF, self.proj.out, C, None, None, self.start, F32, m[2], m[3], m[4], 5 * C,
                           self.x2, C, BF, self.h2, C, stream)

    def check(self):
        C, H, G, D, rows = self.C, self.H, self.G, self.D, self.cuts[-1]
        seg = packed.segment_of(self.cuts, self.M)
        mod = [f64(self.mod[:, i * C:(i + 1) * C]) for i in range(5)]
        # half a bf16 step, and as much again for the arithmetic
        close = lambda got, want, size: bool(((f64(got) - want).abs() <= 2.0 ** -7 * want.abs() + size)[:rows].all())   # noqa: E731
        _, out, _ = packed.layer_norm(f64(self.x), None, None, None, seg, None, mod[0], mod[1], 1e-6)
        assert close(self.h, out, 1e-4)
        self.qkv.check(self.h)
        axis = torch.tensor([0] * 8 + [1] * 12 + [2] * 12)
        qkv = f64(self.qkv.out)
        for got, cols, heads, w in ((self.qr, qkv[:, :C], H, self.qw), (self.kr, qkv[:, C:C + G * D], G, self.kw)):
            want, size, _ = packed.rotary(cols, heads, axis, f64(self.pos), f64(self.freqs), f64(w), 1e-6, False)
            assert bool(((f64(got) - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5 * (1 + size)).all())
        q, k, v = f64(self.qr), f64(self.kr), qkv[:, (H + G) * D:]
        for a, b in zip(self.cuts[:-1], self.cuts[1:]):
            for h in range(H):
                kv = slice(h // 2 * D, h // 2 * D + D)
                want, wabs, _, _, _ = packed.attention(q[a:b, h * D:h * D + D], k[a:b, kv], v[a:b, kv], D ** -0.5, 0.0, False, 0, None)
                # the weights' rounding and the result's
                assert bool(((f64(self.att[a:b, h * D:h * D + D]) - want).abs() <= 2.0 ** -7 * wabs + 2.0 ** -8 * want.abs()).all())
        self.proj.check(self.att)
        h2, out2, _ = packed.layer_norm(f64(self.x), f64(self.proj.out), None, None, seg, mod[2], mod[3], mod[4], 1e-6)
        assert close(self.x2, h2, 1e-4) and close(self.h2, out2, 1e-4)


def test_the_attention_half_of_a_block():
    k = Block()
    k.run()
    torch.cuda.synchronize()
    k.check()
    rows = k.cuts[-1]
    for t in (k.h, k.att, k.x2, k.h2):
        assert bool((t[rows:] == 7.0).all()), "rows behind the last request were written"


def test_captured_and_replayed_with_other_cuts():
    k = Block()
    k.run()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            k.run(side)
    torch.cuda.synchronize()
    for i, cuts in enumerate(([0, 40, 40, 130], [0, 1, 2, 129], [0, 78, 116, 117])):
        k.cuts = cuts
        k.start.copy_(torch.tensor(cuts, dtype=torch.int32))
        k.x.copy_(torch.randn(k.M, k.C, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        k.check()
        got = k.h2.clone(), k.x2.clone()
        k.h2.fill_(7.0)
        k.x2.fill_(7.0)
        k.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a[:cuts[-1]], b[:cuts[-1]]) for a, b in zip(got, (k.h2, k.x2))), i
