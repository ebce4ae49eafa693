"""Cases of the operators around the attention of a packed batch: inputs, plain forms and the
library's calls.

The rows of all requests of a batch stand one after the other, request i's from seg_start[i] to
seg_start[i + 1] - 1.  Between the 4-bit linears of a transformer block run three operators:

  layer   h = x + gate_i y (the branch before, onto the residual stream), then
          out = ((h - mean) / sqrt(var + eps) w + b) (1 + scale_i) + shift_i, which the next linear takes
  rotary  q and k heads as the q, k, v linear leaves them: an optional RMS norm over each head, then
          every channel pair turned by the angle  positions[row, axis of the pair] freqs[pair]
  attn    softmax attention within each request, grouped heads; optionally scores capped by a tanh, a
          bias by distance, a causal mask with a prefix that every row sees

``own`` says whether ``run`` makes the library's calls or computes the plain forms.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def _attn(name, q, kv, heads, kv_heads, D, cap=0.0, causal=False, prefix=False, bias=False, tail=0):
    """q, kv: rows of every request, as text ("7 30 1"); kv "" means the same rows as q."""
    c = {"op": "attn", "q": q, "kv": kv, "heads": heads, "kv_heads": kv_heads, "D": D, "cap": cap,
         "causal": causal, "prefix": prefix, "bias": bias, "tail": tail}
    return {"name": name, **c} if name else c


def _rotary(name, M, heads, kv_heads, D, pairs, pairing, x, norm=True, far=1):
    c = {"op": "rotary", "M": M, "heads": heads, "kv_heads": kv_heads, "D": D, "pairs": pairs,
         "pairing": pairing, "x": x, "norm": norm, "far": far}
    return {"name": name, **c} if name else c


def _layer(name, rows, C, x, out, mod, residual=True, gate=True, affine=False, tail=0):
    c = {"op": "layer", "rows": rows, "C": C, "x": x, "out": out, "mod": mod, "residual": residual,
         "gate": gate, "affine": affine, "tail": tail}
    return {"name": name, **c} if name else c


def _text(lens):
    return " ".join(str(n) for n in lens)


def listed():
    return [
        # the joint attention of one image: 64 x 64 patches and 512 text rows
        _attn("attn_joint", "4608", "", 24, 24, 128),
        # a larger image, 96 x 96 patches and 512 text rows
        _attn("attn_large", "9728", "", 24, 24, 128),
        # a served batch of images of uneven sizes, narrow heads, rows behind the last request
        _attn("attn_packed", "1101 337 2500 64 1 913", "", 16, 16, 72, tail=29),
        # image rows over their request's text rows, capped scores; one request has no text
        _attn("attn_cross", "1024 1024 1024 1024", "77 300 0 128", 16, 16, 64, cap=30.0),
        # text to image in one sequence: the prompt sees itself, image rows it and what came before
        _attn("attn_prefix", "1500 2047 700", "", 32, 8, 128, causal=True, prefix=True, bias=True),
        # one row of each request over all that it has so far
        _attn("attn_single", "1 1 1 1 1 1 1 1", "8000 311 4096 1 2777 0 6000 5003", 32, 8, 128, bias=True),
        # q and k of the joint attention's linear: text rows stand at the origin
        _rotary("rotary_joint", 4608, 24, 24, 128, "8 28 28", "interleaved", "bf16"),
        # video: fp32 rows of a linear, few k heads, frames far from the first
        _rotary("rotary_video", 6001, 16, 4, 96, "16 16 16", "halves", "f32", far=100000),
        # one row a request: latency counts
        _rotary("rotary_rows", 3, 24, 24, 128, "64", "interleaved", "bf16", norm=False),
        # attention's output through its gate onto the residual stream, then the next linear's input
        _layer("layer_joint", "4608", 3072, "bf16", "bf16", "f32"),
        # a ragged batch on an fp32 residual stream, odd width, empty requests, rows behind the last
        _layer("layer_ragged", "300 0 1 517 64 0 355", 1170, "f32", "bf16", "bf16", affine=True, tail=21),
        # the first norm of a few pooled rows
        _layer("layer_rows", "1 1", 1152, "bf16", "f32", "f32", residual=False, gate=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cut(rng, total, n):
    """n lengths of the sum total, some of them zero or one."""
    at = sorted(rng.randint(0, total) for _ in range(n - 1))
    lens = [b - a for a, b in zip([0] + at, at + [total])]
    if n > 2 and rng.random() < 0.3:
        i = rng.randrange(n)
        j = (i + 1) % n
        lens[i], lens[j] = 1, lens[j] + max(0, lens[i] - 1)
    return lens


def draw(rng):
    kind = rng.random()
    if kind < 0.5:
        while True:
            D = rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128, 128])
            kv_heads = rng.choice([1, 2, 4, 8, 16, 24])
            heads = kv_heads * rng.choice([1, 1, 2, 4])
            n = _logint(rng, 1, 24)
            causal = rng.random() < 0.3
            q = _cut(rng, _logint(rng, n, 9728), n)
            shape = rng.random()
            if causal or shape < 0.5:
                kv = q
            elif shape < 0.75:
                kv = [rng.choice([0, 1]) if rng.random() < 0.1 else _logint(rng, 1, 512) for _ in q]
            else:
                q, kv = [1] * n, [0 if rng.random() < 0.05 else _logint(rng, 1, 8192) for _ in q]
            if heads * sum(a * b for a, b in zip(q, kv)) <= 2.0e9 and sum(kv) * kv_heads * D <= 6.0e7:
                break
        return _attn(None, _text(q), "" if kv is q else _text(kv), heads, kv_heads, D,
                     cap=rng.choice([0.0, 0.0, 0.0, 15.0, 50.0]), causal=causal,
                     prefix=causal and rng.random() < 0.6, bias=rng.random() < 0.25, tail=rng.randint(0, 40))
    if kind < 0.75:
        while True:
            pairs = [rng.randint(1, 24) for _ in range(rng.randint(1, 4))]
            if rng.random() < 0.6:
                pairs[-1] += -sum(pairs) % 8
            D = 2 * sum(pairs)
            kv_heads = rng.choice([1, 2, 4, 8, 16, 24])
            heads = kv_heads * rng.choice([1, 1, 2, 4])
            M = _logint(rng, 1, 16384)
            if D <= 128 and M * (heads + kv_heads) * D <= 2.8e7:
                break
        return _rotary(None, M, heads, kv_heads, D, _text(pairs), rng.choice(["interleaved", "halves"]),
                       rng.choice(["bf16", "bf16", "f32"]), norm=rng.random() < 0.7, far=rng.choice([1, 1, 1000, 100000]))
    while True:
        C = _logint(rng, 64, 8192)
        if rng.random() < 0.7:
            C = (C + 7) // 8 * 8
        n = _logint(rng, 1, 32)
        total = _logint(rng, n, 16384)
        if total * C <= 1.4e7:
            break
    residual = rng.random() < 0.7
    return _layer(None, _text(_cut(rng, total, n)), C, rng.choice(["bf16", "bf16", "f32"]),
                  rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32"]), residual=residual,
                  gate=residual and rng.random() < 0.7, affine=rng.random() < 0.4, tail=rng.randint(0, 30))


def _lens(text):
    return [int(t) for t in text.split()]


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"case": case}
    if case["op"] == "attn":
        r = random.Random(seed * 1009 + 17)
        q, H, G, D = _lens(case["q"]), case["heads"], case["kv_heads"], case["D"]
        kv = _lens(case["kv"]) if case["kv"] else q
        s["qs"], s["ks"] = _starts(q), _starts(kv)
        Mq, Mk = s["qs"][-1] + case["tail"], s["ks"][-1]
        # heads of different sharpness: some look at everything, some at a few keys
        sharp = torch.linspace(0.5, 3.0, H, device="cuda").repeat_interleave(D)
        if case["kv"]:
            s["q"] = (normal(Mq, H * D) * sharp).to(torch.bfloat16)
            s["kvm"] = normal(max(Mk, 1), 2 * G * D, dtype=torch.bfloat16)       # the k, v linear's output
            s["k"], s["v"], s["kv_stride"] = s["kvm"][:, :G * D], s["kvm"][:, G * D:], 2 * G * D
        else:
            s["q"] = (normal(Mq, H * D) * sharp).to(torch.bfloat16)
            s["k"] = normal(Mq, G * D, dtype=torch.bfloat16)                     # as the rotary call leaves them
            s["qkv"] = normal(Mq, (H + 2 * G) * D, dtype=torch.bfloat16)
            s["v"], s["kv_stride"] = s["qkv"][:, (H + G) * D:], G * D
            Mk = Mq
        s["v_stride"] = s["v"].stride(0)
        s["Mq"], s["Mk"] = Mq, Mk
        s["q_start"] = i32(s["qs"])
        s["kv_start"] = i32(s["ks"]) if case["kv"] else s["q_start"]
        s["prefix"] = i32([r.randint(0, n // 2) for n in kv]) if case["prefix"] else None
        # slopes fall geometrically over the heads
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H) if case["bias"] else None
        s["scale"] = D ** -0.5
        s["out"] = normal(Mq, H * D, dtype=torch.bfloat16)
        return s
    if case["op"] == "rotary":
        M, H, G, D = case["M"], case["heads"], case["kv_heads"], case["D"]
        pairs = _lens(case["pairs"])
        s["pairs"] = pairs
        s["qkv"] = (normal(M, (H + 2 * G) * D) * (torch.rand((H + 2 * G) * D, generator=g, device="cuda") * 2 + 0.2)
                    ).to(_DT[case["x"]])
        s["freqs"] = torch.cat([10000.0 ** (-torch.arange(p, dtype=torch.float64, device="cuda") / p) for p in pairs])
        row = torch.arange(M, device="cuda")
        side = max(1, int(M ** 0.5))
        pos = torch.stack([(row // (side * side) * case["far"]).float(), (row // side % side).float() - 0.5 * side,
                           (row % side).float() * 0.75, row.float()], dim=1)[:, :len(pairs)]
        pos = pos + torch.randint(0, 8, (1, len(pairs)), generator=g, device="cuda") * float(case["far"])
        pos[:M // 9] = 0.0                                                        # text rows
        s["pos"] = pos.contiguous()
        s["qw"] = (1 + normal(D, scale=0.2)).to(torch.bfloat16) if case["norm"] else None
        s["kw"] = (1 + normal(D, scale=0.2)).to(torch.bfloat16) if case["norm"] else None
        s["qo"] = torch.empty(M, H * D, dtype=torch.bfloat16, device="cuda")
        s["ko"] = torch.empty(M, G * D, dtype=torch.bfloat16, device="cuda")
        return s
    lens, C = _lens(case["rows"]), case["C"]
    s["ss"] = _starts(lens)
    M, n = s["ss"][-1] + case["tail"], len(lens)
    s["M"], s["n"] = M, n
    s["start"] = i32(s["ss"])
    s["x"] = (normal(M, C) * (torch.rand(C, generator=g, device="cuda") * 2 + 0.2) + normal(C, scale=1.5)).to(_DT[case["x"]])
    s["y"] = normal(M, C, dtype=torch.bfloat16) if case["residual"] else None
    s["w"] = (1 + normal(C, scale=0.3)).to(torch.bfloat16) if case["affine"] else None
    s["b"] = normal(C, scale=0.3, dtype=torch.bfloat16) if case["affine"] else None
    # the modulation layer's rows: gate | scale | shift
    s["mod"] = normal(n, 3 * C, scale=0.4, dtype=_DT[case["mod"]])
    s["gate"] = s["mod"][:, :C] if case["gate"] else None
    s["scale"], s["shift"] = s["mod"][:, C:2 * C], s["mod"][:, 2 * C:]
    s["out"] = normal(M, C, dtype=_DT[case["out"]])
    s["xo"] = normal(M, C, dtype=_DT[case["x"]]) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------------- one pass
def _plain_attn(s):
    case = s["case"]
    H, G, D = case["heads"], case["kv_heads"], case["D"]
    out = s["out"].clone()
    for i in range(len(s["qs"]) - 1):
        q0, q1, k0, k1 = s["qs"][i], s["qs"][i + 1], s["ks"][i], s["ks"][i + 1]
        if q1 == q0:
            continue
        if k1 == k0:
            out[q0:q1] = 0
            continue
        q = s["q"][q0:q1].float().reshape(q1 - q0, H, D).transpose(0, 1)
        k = s["k"][k0:k1].float().reshape(k1 - k0, G, D).transpose(0, 1).repeat_interleave(H // G, 0)
        v = s["v"][k0:k1].float().reshape(k1 - k0, G, D).transpose(0, 1).repeat_interleave(H // G, 0)
        far = torch.arange(k1 - k0, device="cuda")[None, :] - (torch.arange(q1 - q0, device="cuda")[:, None]
                                                               + (k1 - k0) - (q1 - q0))
        step = max(1, int(5e8 // far.numel()))                   # heads whose scores are held at a time
        for h in range(0, H, step):
            p = torch.matmul(q[h:h + step], k[h:h + step].transpose(1, 2)) * s["scale"]
            if case["cap"]:
                p = case["cap"] * torch.tanh(p / case["cap"])
            if s["slopes"] is not None:
                p = p - s["slopes"][h:h + step, None, None] * far.abs()
            if case["causal"]:
                seen = far <= 0
                if s["prefix"] is not None:
                    seen = seen | (torch.arange(k1 - k0, device="cuda")[None, :] < s["prefix"][i])
                p = torch.where(seen, p, float("-inf"))
            p = torch.exp(p - p.amax(dim=2, keepdim=True))
            o = torch.matmul(p, v[h:h + step]) / p.sum(dim=2, keepdim=True)
            out[q0:q1, h * D:h * D + o.shape[0] * D] = o.transpose(0, 1).reshape(q1 - q0, -1).to(out.dtype)
    return out


def _plain_rotary(s):
    case = s["case"]
    M, H, G, D = case["M"], case["heads"], case["kv_heads"], case["D"]
    axis = torch.repeat_interleave(torch.arange(len(s["pairs"]), device="cuda"),
                                   torch.tensor(s["pairs"], device="cuda"), output_size=D // 2)
    angle = s["pos"].double()[:, axis] * s["freqs"]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]

    def turn(x, w, heads):
        x = x.float().reshape(M, heads, D)
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + 1e-6) * w.float()
        if case["pairing"] == "halves":
            a, b = x[..., :D // 2], x[..., D // 2:]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=2)
        else:
            a, b = x[..., 0::2], x[..., 1::2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=3)
        return y.reshape(M, heads * D).to(torch.bfloat16)

    return turn(s["qkv"][:, :H * D], s["qw"], H), turn(s["qkv"][:, H * D:(H + G) * D], s["kw"], G)


def _plain_layer(s):
    m = s["ss"][-1]
    lens = (s["start"][1:] - s["start"][:-1]).long()
    seg = torch.repeat_interleave(torch.arange(s["n"], device="cuda"), lens, output_size=m)
    h = s["x"][:m].float()
    if s["y"] is not None:
        y = s["y"][:m].float()
        h = h + (y if s["gate"] is None else s["gate"].float()[seg] * y)
    d = h - h.mean(dim=1, keepdim=True)
    z = d * torch.rsqrt((d * d).mean(dim=1, keepdim=True) + 1e-6)
    if s["w"] is not None:
        z = z * s["w"].float() + s["b"].float()
    z = z * (1 + s["scale"].float()[seg]) + s["shift"].float()[seg]
    out = s["out"].clone()
    out[:m] = z.to(out.dtype)
    if s["y"] is None:
        return out
    xo = s["xo"].clone()
    xo[:m] = h.to(xo.dtype)
    return out, xo


def run(state):
    s, case = state, state["case"]
    if own:
        import bit_diffusion_amd as bd
        dts = {"bf16": bd.SVDQ_DT_BF16, "f32": bd.SVDQ_DT_F32}
        if case["op"] == "attn":
            H, G, D, n = case["heads"], case["kv_heads"], case["D"], len(s["qs"]) - 1
            if "ws" not in s:                    # the workspace a program allocates once for its shapes
                s["ws_bytes"] = bd.svdq_attention_workspace_bytes(s["Mq"], s["Mk"], H, G, D, n)
                s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
            bd.svdq_attention(s["Mq"], s["Mk"], H, G, D, n, s["scale"], case["cap"],
                              bd.SVDQ_MASK_CAUSAL if case["causal"] else bd.SVDQ_MASK_NONE, s["q_start"],
                              s["kv_start"], s["prefix"], s["slopes"], s["q"], H * D, s["k"], s["kv_stride"],
                              s["v"], s["v_stride"], s["out"], H * D, s["ws"], s["ws_bytes"])
            return s["out"]
        if case["op"] == "rotary":
            M, H, G, D = case["M"], case["heads"], case["kv_heads"], case["D"]
            w = (H + 2 * G) * D
            bd.svdq_rotary(M, H, G, D, s["pairs"],
                           bd.SVDQ_ROTARY_HALVES if case["pairing"] == "halves" else bd.SVDQ_ROTARY_INTERLEAVED,
                           s["pos"], len(s["pairs"]), s["freqs"], 1e-6, s["qw"], s["kw"], dts[case["x"]], s["qkv"],
                           w, s["qkv"][:, H * D:], w, bd.SVDQ_DT_BF16, s["qo"], H * D, s["ko"], G * D)
            return s["qo"], s["ko"]
        C = case["C"]
        bd.svdq_layer_norm(s["M"], C, s["n"], 1e-6, dts[case["x"]], s["x"], C, bd.SVDQ_DT_BF16, s["y"], C, s["w"],
                           s["b"], s["start"], dts[case["mod"]], s["gate"], s["scale"], s["shift"], 3 * C,
                           s["xo"], C, dts[case["out"]], s["out"], C)
        return s["out"] if s["xo"] is None else (s["out"], s["xo"])
    return {"attn": _plain_attn, "rotary": _plain_rotary, "layer": _plain_layer}[case["op"]](s)


# --------------------------------------------------------------------------- work and values
def work(case):
    if case["op"] == "attn":
        H, G, D, q = case["heads"], case["kv_heads"], case["D"], _lens(case["q"])
        kv = _lens(case["kv"]) if case["kv"] else q
        seen = 0                                 # pairs of a row and a key that it sees (no prefix counted)
        for a, b in zip(q, kv):
            seen += a * (a + 1) // 2 if case["causal"] else a * b
        rows = sum(a for a, b in zip(q, kv))
        keys = sum(b for a, b in zip(q, kv) if a)
        return {"bytes": 2 * D * (2 * rows * H + 2 * keys * G), "flops": 4 * D * H * seen}
    if case["op"] == "rotary":
        n = case["M"] * (case["heads"] + case["kv_heads"]) * case["D"]
        return {"bytes": n * (2 + (2 if case["x"] == "bf16" else 4)) + case["M"] * 4 * len(_lens(case["pairs"])),
                "flops": n * (7 if case["norm"] else 3)}
    lens = _lens(case["rows"])
    n, segs = sum(lens) * case["C"], sum(1 for v in lens if v) * case["C"]
    xsz, osz, msz = (2 if case[k] == "bf16" else 4 for k in ("x", "out", "mod"))
    per = xsz + osz + (2 + xsz if case["residual"] else 0)
    return {"bytes": n * per + segs * msz * (3 if case["gate"] else 2), "flops": n * (10 if case["residual"] else 8)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        H, G, D = case["heads"], case["kv_heads"], case["D"]
        out = s["out"].double()
        for i, (q0, q1) in enumerate(zip(s["qs"][:-1], s["qs"][1:])):
            k0, k1 = s["ks"][i], s["ks"][i + 1]
            first = 0 if s["prefix"] is None else int(s["prefix"][i])
            keys = torch.arange(k1 - k0, device="cuda")
            for h in range(H):
                kh = s["k"][k0:k1, h // (H // G) * D:(h // (H // G) + 1) * D].double().t().contiguous()
                vh = s["v"][k0:k1, h // (H // G) * D:(h // (H // G) + 1) * D].double().contiguous()
                for a in range(q0, q1, 8192):
                    b = min(q1, a + 8192)
                    at = torch.arange(a - q0, b - q0, device="cuda") + (k1 - k0) - (q1 - q0)
                    t = s["q"][a:b, h * D:(h + 1) * D].double() @ kh * s["scale"]
                    if case["cap"]:
                        t = t / case["cap"]
                        t = case["cap"] * (1 - 2 / (torch.exp(2 * t) + 1))
                    if s["slopes"] is not None:
                        t = t - s["slopes"][h].double() * (at[:, None] - keys[None, :]).abs().double()
                    if case["causal"]:
                        t.masked_fill_((keys[None, :] > at[:, None]) & (keys[None, :] >= first), float("-inf"))
                    if k1 == k0:
                        out[a:b, h * D:(h + 1) * D] = 0
                    else:
                        out[a:b, h * D:(h + 1) * D] = torch.softmax(t, dim=1) @ vh
        return out
    if case["op"] == "rotary":
        M, H, G, D, P = case["M"], case["heads"], case["kv_heads"], case["D"], case["D"] // 2
        axes = [a for a, p in enumerate(s["pairs"]) for _ in range(p)]
        turn = torch.stack([s["pos"][:, a].double() * s["freqs"][j] for j, a in enumerate(axes)], dim=1)
        unit = torch.polar(torch.ones_like(turn), turn)[:, None, :]

        def one(x, w, n):
            x = x.double().reshape(M, n, D)
            if w is not None:
                x = x / torch.sqrt((x ** 2).sum(2, keepdim=True) / D + 1e-6) * w.double()
            halves = case["pairing"] == "halves"
            z = torch.complex(x[..., :P], x[..., P:]) if halves else torch.view_as_complex(x.reshape(M, n, P, 2))
            z = z * unit
            y = torch.cat([z.real, z.imag], 2) if halves else torch.view_as_real(z)
            return y.reshape(M, n * D)

        return one(s["qkv"][:, :H * D], s["qw"], H), one(s["qkv"][:, H * D:(H + G) * D], s["kw"], G)
    out = s["out"].double()
    xo = None if s["xo"] is None else s["xo"].double()
    for i, (a, b) in enumerate(zip(s["ss"][:-1], s["ss"][1:])):
        if b == a:
            continue
        h = s["x"][a:b].double()
        if s["y"] is not None:
            h = h + s["y"][a:b].double() * (1.0 if s["gate"] is None else s["gate"][i].double())
            xo[a:b] = h
        z = (h - h.mean(1, keepdim=True)) / torch.sqrt(h.var(1, unbiased=False, keepdim=True) + 1e-6)
        if s["w"] is not None:
            z = z * s["w"].double() + s["b"].double()
        out[a:b] = z * (1 + s["scale"][i].double()) + s["shift"][i].double()
    return out if xo is None else (out, xo)
