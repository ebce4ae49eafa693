"""Cases of the batched-adapter and group-norm operators: inputs, plain forms and the library's calls.

Two operators stand beside the 4-bit linears:

  lora  rows of one batch belong to different requests, each with its own low-rank adapter (or
        none):  out = act(base + alpha_s (x A_s^T) B_s^T)  on the rows of every segment.
  norm  group normalisation of channels-last images, affine, optionally modulated by per-image
        scale and shift rows, then an activation; its output is the activation kernel's input.

``own`` says whether ``run`` makes the library's calls or computes the plain forms.
"""
import math
import random

import torch

own = False

NONE, GELU, SILU = "none", "gelu", "silu"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def _lora(name, M, K, N, R, adapters, segments, dtype, act=NONE, tail=0, mixed=False):
    c = {"op": "lora", "M": M, "K": K, "N": N, "R": R, "adapters": adapters, "segments": segments,
         "dtype": dtype, "act": act, "tail": tail, "mixed": mixed}
    return {"name": name, **c} if name else c


def _norm(name, B, rows, C, groups, x, out, act=NONE, affine=True, mod=None):
    c = {"op": "norm", "B": B, "rows": rows, "C": C, "groups": groups, "x": x, "out": out,
         "act": act, "affine": affine, "mod": mod or ""}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the modulation layer of a batch of two requests: one conditioning row and one adapter each
        _lora("lora_modulation", 2, 3072, 18432, 16, 8, 2, "bf16"),
        # one row per request (pooled embeddings, single tokens): many short segments, odd width
        _lora("lora_single_rows", 37, 1536, 1530, 32, 24, 37, "f32"),
        # the attention projection of one 64 x 64 patch grid's worth of rows, four small images
        _lora("lora_attention", 4096, 3072, 3072, 16, 6, 4, "bf16"),
        # a ragged batch: adapters of mixed ranks, empty requests, rows behind the last one, fp32
        _lora("lora_ragged", 1237, 1088, 1000, 64, 12, 11, "f32", tail=29, mixed=True),
        # the MLP's first linear: image and text rows, GELU after the adapter
        _lora("lora_mlp", 4608, 3072, 12288, 32, 4, 3, "bf16", act=GELU),
        # a large batch at the highest rank
        _lora("lora_rank128", 16384, 4096, 4096, 128, 16, 16, "bf16"),
        # the deepest level of a small image: latency counts
        _norm("norm_8x8", 2, 64, 1280, 32, "bf16", "bf16", act=SILU),
        # a middle level with the conditioning's scale and shift
        _norm("norm_32x32_modulated", 2, 1024, 640, 32, "bf16", "bf16", act=SILU, mod="f32"),
        # in front of a projection of the 64 x 64 patch grid
        _norm("norm_64x64", 1, 4096, 320, 32, "bf16", "bf16"),
        # odd: an uneven image, 11 channels a group, fp32 in and out
        _norm("norm_odd", 3, 1023, 330, 30, "f32", "f32", act=GELU, mod="bf16"),
        # the decoder's levels: large images
        _norm("norm_256x256", 1, 65536, 512, 32, "bf16", "bf16", act=SILU),
        _norm("norm_512x512", 1, 262144, 256, 32, "f32", "bf16", act=SILU),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            M = _logint(rng, 1, 16384)
            K = 64 * _logint(rng, 4, 64)
            N = _logint(rng, 200, 18432)
            if rng.random() < 0.5:
                N = (N + 63) // 64 * 64
            R = rng.choice([16, 16, 32, 32, 48, 64, 128])
            dtype = rng.choice(["bf16", "bf16", "f32"])
            adapters = rng.randint(1, 24)
            # what a pass moves and computes, and the plain form's product over all adapters
            size = M * (2 * K + 2 * N * (2 if dtype == "bf16" else 4))
            if size <= 2.5e8 and M * adapters * R * (K + N) <= 2.0e11:
                break
        segments = min(M, _logint(rng, 1, 64))
        return _lora(None, M, K, N, R, adapters, segments, dtype, act=rng.choice([NONE, NONE, GELU, SILU]),
                     tail=rng.randint(0, min(M // 8, 64)), mixed=rng.random() < 0.5)
    groups = rng.choice([1, 8, 16, 30, 32, 32, 32, 64])
    C = groups * _logint(rng, 4, 64)
    while True:
        B = rng.randint(1, 8)
        rows = _logint(rng, 1, 131072)
        if B * rows * C <= 4.0e7:
            break
    return _norm(None, B, rows, C, groups, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]),
                 act=rng.choice([NONE, SILU, SILU, GELU]), affine=rng.random() < 0.8,
                 mod=rng.choice([None, None, "bf16", "f32"]))


# ------------------------------------------------------------------------------------ inputs
def _plan(case, seed):
    """Rows of every segment, the adapter of each (-1: none) and the adapters' ranks."""
    r = random.Random(seed * 1009 + 17)
    M, S, n = case["M"] - case["tail"], case["adapters"], case["segments"]
    if n == M:                                   # one row a request
        cuts = list(range(M + 1))
    else:
        # requests of like size, unevenly cut; two cuts may meet (an empty request)
        inner = sorted(min(M, max(0, int(round(M * (i + r.uniform(-0.45, 0.45)) / n)))) for i in range(1, n))
        cuts = [0] + inner + [M]
    ids = [(i + r.randint(0, 1)) % S if r.random() < 0.9 or n < 3 else -1 for i in range(n)]
    ranks = [r.choice([4, 8, case["R"] // 2, case["R"]]) if case["mixed"] else case["R"] for _ in range(S)]
    return cuts, ids, ranks


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0, dtype=torch.float32):
        t = torch.randn(*shape, generator=g, device="cuda") * scale
        return t.to(dtype)

    if case["op"] == "lora":
        M, K, N, R, S = (case[k] for k in ("M", "K", "N", "R", "adapters"))
        cuts, ids, ranks = _plan(case, seed)
        x = normal(M, K)
        x[:, torch.randint(0, K, (max(1, K // 100),), generator=g, device="cuda")] *= 30.0   # outlier channels
        dt = _DT[case["dtype"]]
        return {"case": case, "x": x.to(torch.bfloat16),
                "down": normal(S, R, K, scale=K ** -0.5, dtype=torch.bfloat16),
                "up": normal(S, N, R, scale=0.05, dtype=torch.bfloat16),
                "alpha": torch.rand(S, generator=g, device="cuda") + 0.5,
                "ranks": torch.tensor(ranks, dtype=torch.int32, device="cuda"),
                "starts": torch.tensor(cuts, dtype=torch.int32, device="cuda"),
                "ids": torch.tensor(ids, dtype=torch.int32, device="cuda"),
                "rows": cuts[-1],
                "base": normal(M, N, dtype=dt), "out": normal(M, N, dtype=dt)}
    B, rows, C = (case[k] for k in ("B", "rows", "C"))
    x = normal(B * rows, C)
    x = x * (torch.rand(C, generator=g, device="cuda") * 2 + 0.2) + normal(C, scale=1.5)     # uneven channels
    s = {"case": case, "x": x.to(_DT[case["x"]]), "out": torch.empty(B * rows, C, dtype=_DT[case["out"]], device="cuda"),
         "weight": None, "bias": None, "scale": None, "shift": None}
    if case["affine"]:
        s["weight"] = (1 + normal(C, scale=0.3)).to(torch.bfloat16)
        s["bias"] = normal(C, scale=0.3, dtype=torch.bfloat16)
    if case["mod"]:
        s["mod"] = normal(B, 2 * C, scale=0.3, dtype=_DT[case["mod"]])                        # [scale | shift] rows
        s["scale"], s["shift"] = s["mod"][:, :C], s["mod"][:, C:]
    return s


# ---------------------------------------------------------------------------------- one pass
def _act(y, act):
    if act == GELU:
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == SILU:
        return y / (1 + torch.exp(-y))
    return y


def _plain_lora(s):
    case = s["case"]
    S, R, M = case["adapters"], case["R"], s["rows"]
    lens = (s["starts"][1:] - s["starts"][:-1]).long()
    ids = torch.repeat_interleave(s["ids"].long(), lens, output_size=M)
    live = torch.arange(R, device="cuda")[None, :] < s["ranks"][:, None]                      # [S, R]
    gain = torch.where(live, s["alpha"][:, None], torch.zeros_like(s["alpha"])[:, None]).reshape(1, S * R)
    mine = (torch.arange(S, device="cuda").repeat_interleave(R, output_size=S * R)[None, :] == ids[:, None])
    t = s["x"][:M].float() @ s["down"].float().reshape(S * R, -1).t()                         # every adapter's down
    t = t * (mine * gain)
    y = s["base"][:M].float() + t @ s["up"].float().permute(0, 2, 1).reshape(S * R, -1)
    out = s["out"].clone()
    out[:M] = _act(y, case["act"]).to(out.dtype)
    return out


def _plain_norm(s):
    case = s["case"]
    B, rows, C, G = (case[k] for k in ("B", "rows", "C", "groups"))
    x = s["x"].float().reshape(B, rows, G, C // G)
    d = x - x.mean(dim=(1, 3), keepdim=True)
    y = (d * torch.rsqrt((d * d).mean(dim=(1, 3), keepdim=True) + 1e-5)).reshape(B, rows, C)
    if s["weight"] is not None:
        y = y * s["weight"].float() + s["bias"].float()
    if s["scale"] is not None:
        y = y * (1 + s["scale"].float())[:, None, :] + s["shift"].float()[:, None, :]
    return _act(y, case["act"]).to(s["out"].dtype).reshape(B * rows, C)


def run(state):
    s, case = state, state["case"]
    if own:
        import bit_diffusion_amd as bd
        act = {NONE: bd.SVDQ_ACT_NONE, GELU: bd.SVDQ_ACT_GELU_TANH, SILU: bd.SVDQ_ACT_SILU}[case["act"]]
        dts = {"bf16": bd.SVDQ_DT_BF16, "f32": bd.SVDQ_DT_F32}
        if case["op"] == "lora":
            M, K, N, R, S, n = (case[k] for k in ("M", "K", "N", "R", "adapters", "segments"))
            if "ws" not in s:                    # the workspace a program allocates once for its shapes
                s["ws_bytes"] = bd.svdq_lora_batch_workspace_bytes(M, K, N, R, n)
                s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
            bd.svdq_lora_batch(M, K, N, R, S, n, s["x"], K, s["down"], s["up"], s["alpha"], s["ranks"],
                               s["starts"], s["ids"], s["base"], N, act, dts[case["dtype"]], s["out"], N,
                               s["ws"], s["ws_bytes"])
            return s["out"]
        B, rows, C, G = (case[k] for k in ("B", "rows", "C", "groups"))
        if "ws" not in s:
            s["ws_bytes"] = bd.svdq_group_norm_workspace_bytes(B, rows, C, G)
            s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
        bd.svdq_group_norm(B, rows, C, G, 1e-5, dts[case["x"]], s["x"], C, s["weight"], s["bias"],
                           dts[case["mod"] or "f32"], s["scale"], s["shift"], 2 * C, act, dts[case["out"]],
                           s["out"], C, s["ws"], s["ws_bytes"])
        return s["out"]
    return _plain_lora(s) if case["op"] == "lora" else _plain_norm(s)


# --------------------------------------------------------------------------- work and values
def work(case):
    if case["op"] == "lora":
        M, K, N, R = (case[k] for k in ("M", "K", "N", "R"))
        m, esz = M - case["tail"], 2 if case["dtype"] == "bf16" else 4
        used = min(case["adapters"], case["segments"])
        return {"bytes": m * (2 * K + 2 * N * esz) + used * R * (K + N) * 2, "flops": 2 * m * R * (K + N)}
    n = case["B"] * case["rows"] * case["C"]
    return {"bytes": n * ((2 if case["x"] == "bf16" else 4) + (2 if case["out"] == "bf16" else 4)), "flops": 10 * n}


def exact(case, seed):
    s = prepare(case, seed)

    def act(y):
        if case["act"] == GELU:
            return y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
        return y * torch.sigmoid(y) if case["act"] == SILU else y

    if case["op"] == "lora":
        cuts, ids, ranks = _plan(case, seed)
        out = s["out"].double()
        for i, a in enumerate(ids):
            lo, hi = cuts[i], cuts[i + 1]
            y = s["base"][lo:hi].double()
            if a >= 0 and hi > lo:
                r = ranks[a]
                t = s["x"][lo:hi].double() @ s["down"][a, :r].double().t().contiguous()
                y = y + s["alpha"][a].double() * (t @ s["up"][a, :, :r].double().t().contiguous())
            out[lo:hi] = act(y)
        return out
    B, rows, C, G = (case[k] for k in ("B", "rows", "C", "groups"))
    out = torch.empty(B * rows, C, dtype=torch.float64, device="cuda")
    cg = C // G
    for b in range(B):
        xb = s["x"][b * rows:(b + 1) * rows].double()
        mean = xb.sum(0).reshape(G, cg).sum(1) / (rows * cg)
        mean = mean.repeat_interleave(cg)
        var = ((xb - mean) ** 2).sum(0).reshape(G, cg).sum(1) / (rows * cg)
        y = (xb - mean) / torch.sqrt(var + 1e-5).repeat_interleave(cg)
        if s["weight"] is not None:
            y = y * s["weight"].double() + s["bias"].double()
        if s["scale"] is not None:
            y = y * (1 + s["scale"][b].double()) + s["shift"][b].double()
        out[b * rows:(b + 1) * rows] = act(y)
    return out
