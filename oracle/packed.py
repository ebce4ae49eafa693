"""Plain fp64 forms of the packed rows' operators (svdq_layer_norm, svdq_rotary, svdq_attention),
straight from their formulas, with the sums that the tests' error bounds are made of.  torch
tensors on any device; every input comes as float64 values."""
import torch


def segment_of(starts, M):
    """The segment of each of M rows, -1 outside."""
    seg = torch.full((M,), -1, dtype=torch.long)
    for i, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        seg[a:b] = i
    return seg


def layer_norm(x, y, weight, bias, seg, gate, scale, shift, eps):
    """Rows of a segment (seg >= 0) only matter.  -> (h, out, parts): parts holds d = h - mean, rstd,
    and A, D of out = d rstd A + D, and D's summands' sizes."""
    i = seg.clamp(min=0)
    one = torch.ones(x.shape[1], dtype=x.dtype, device=x.device)
    g = torch.ones_like(x) if gate is None else gate[i]
    h = x if y is None else x + g * y
    d = h - h.mean(dim=1, keepdim=True)
    rstd = 1 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + eps)
    s = torch.ones_like(x) if scale is None else 1 + scale[i]
    t = torch.zeros_like(x) if shift is None else shift[i]
    w = one if weight is None else weight
    b = 0 * one if bias is None else bias
    A, D = w * s, b * s + t
    return h, d * rstd * A + D, {"d": d, "rstd": rstd, "A": A, "D": D, "Dabs": (b * s).abs() + t.abs(),
                                 "hin": x.abs() + (0 if y is None else (g * y).abs())}


def rotary(x, heads, axis, pos, freqs, weight, eps, halves):
    """x [M, heads D], axis [D / 2]: the axis of each pair -> (result, |a| + |b| of each element's pair
    as normed, |angle| of each element's pair)."""
    M = x.shape[0]
    x = x.reshape(M, heads, -1)
    D = x.shape[2]
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(dim=2, keepdim=True) + eps) * weight
    angle = (pos[:, axis] * freqs)[:, None, :]
    a, b = (x[..., :D // 2], x[..., D // 2:]) if halves else (x[..., 0::2], x[..., 1::2])
    c, s = torch.cos(angle), torch.sin(angle)
    pair = [a * c - b * s, a * s + b * c]
    size = a.abs() + b.abs()
    ang = angle.abs().expand_as(a)
    join = (lambda u, v: torch.cat([u, v], dim=2)) if halves else (lambda u, v: torch.stack([u, v], dim=3))
    return tuple(t.reshape(M, heads * D) for t in (join(*pair), join(size, size), join(ang, ang)))


def limits(rows, keys, causal, prefix):
    """How many keys each row of a segment sees: those below."""
    i = torch.arange(rows)
    if not causal:
        return torch.full((rows,), keys)
    return torch.clamp(torch.clamp(i + keys - rows + 1, min=min(max(prefix, 0), keys)), 0, keys)


def attention(q, k, v, scale, cap, causal, prefix, slope):
    """One segment and head: q [Lq, D], k, v [Lk, D] -> (out, |out| of |v|, the root of sum (w v)^2,
    and max over a row's keys of the score's size before the mask: sum |q k| scale, and its bias)."""
    Lq, Lk = q.shape[0], k.shape[0]
    dev = q.device
    if Lk == 0:
        z = torch.zeros_like(q)
        return z, z, z, z[:, :1], z[:, :1]
    t = scale * (q @ k.t().contiguous())
    if cap:
        t = cap * torch.tanh(t / cap)
    far = (torch.arange(Lq, device=dev)[:, None] + Lk - Lq - torch.arange(Lk, device=dev)[None, :]).abs()
    bias = torch.zeros_like(t) if slope is None else slope * far
    t = t - bias
    seen = torch.arange(Lk, device=dev)[None, :] < limits(Lq, Lk, causal, prefix).to(dev)[:, None]
    t = torch.where(seen, t, torch.full_like(t, float("-inf")))
    top = t.amax(dim=1, keepdim=True)
    w = torch.exp(t - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    size = scale * (q.abs() @ k.abs().t().contiguous())
    return (w @ v, w @ v.abs(), torch.sqrt((w * w) @ (v * v)), torch.where(seen, size, 0 * size).amax(dim=1, keepdim=True),
            torch.where(seen, bias.abs(), 0 * size).amax(dim=1, keepdim=True))
