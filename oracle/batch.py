"""Plain fp64 forms of the batched adapters (svdq_lora_batch) and of the group norm
(svdq_group_norm), straight from their formulas, with the sums of absolute values that the
tests' fp32 error bounds are made of.  bf16 tensors come as float64 values."""
import numpy as np


def act(y, kind):
    """kind: 0 none, 1 GELU (tanh form), 2 SiLU."""
    with np.errstate(over="ignore"):
        if kind == 1:
            u = np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)
            return y / (1 + np.exp(-2 * u))
        if kind == 2:
            return y / (1 + np.exp(-y))
    return y


def lora_batch(x, down, up, alphas, ranks, starts, ids, base, kind, out):
    """The call's result and, per element before the activation, the value y, the sums
    T = sum_j |alpha t_j B_nj| and D = sum_j |alpha B_nj| sum_k |x_k A_jk|.  Rows of no segment
    keep `out` (T = D = 0 there)."""
    M, N = out.shape
    res, y, T, D = out.copy(), np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    for i, s in enumerate(ids):
        lo, hi = starts[i], starts[i + 1]
        if hi <= lo:
            continue
        v = base[lo:hi].copy() if base is not None else np.zeros((hi - lo, N))
        r = 0 if s < 0 or s >= len(alphas) else int(ranks[s])
        if r > 0:
            A, B = down[s, :r], up[s, :, :r]
            t = alphas[s] * (x[lo:hi] @ A.T)
            v += t @ B.T
            T[lo:hi] = np.abs(t) @ np.abs(B).T
            D[lo:hi] = abs(alphas[s]) * (np.abs(x[lo:hi]) @ np.abs(A).T) @ np.abs(B).T
        y[lo:hi] = v
        res[lo:hi] = act(v, kind)
    return res, y, T, D


def group_norm(x, groups, eps, weight, bias, scale, shift, kind):
    """x [B, rows, C] -> (result, parts): parts holds xhat = (x - mean) / sqrt(var + eps), the
    factor A and offset D of (x - mean) A + D per element, and max |x| of each image's group."""
    B, rows, C = x.shape
    g = x.reshape(B, rows, groups, C // groups)
    mean = g.mean(axis=(1, 3), keepdims=True)
    var = ((g - mean) ** 2).mean(axis=(1, 3), keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    xhat = ((g - mean) * rstd).reshape(B, rows, C)
    w = np.ones(C) if weight is None else weight
    b = np.zeros(C) if bias is None else bias
    ms = np.ones((B, 1, C)) if scale is None else 1 + scale[:, None, :]
    mt = np.zeros((B, 1, C)) if shift is None else shift[:, None, :]
    F = w * ms
    D = b * ms + mt
    big = np.broadcast_to(np.abs(g).max(axis=(1, 3), keepdims=True), g.shape).reshape(B, rows, C)
    rs = np.broadcast_to(rstd, g.shape).reshape(B, rows, C)
    y = xhat * F + D
    return act(y, kind), {"xhat": xhat, "F": F, "D": D, "big": big, "rstd": rs, "y": y}
