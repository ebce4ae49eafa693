"""Pins of the fp64 forms in oracle/batch.py: the adapters against one dense product per row,
the group norm against torch's own in binary64."""
import numpy as np
import torch

from oracle import batch


def test_lora_batch_equals_a_dense_product_per_row():
    rng = np.random.default_rng(5)
    M, K, N, R, S = 13, 64, 7, 16, 3
    x, down, up = rng.standard_normal((M, K)), rng.standard_normal((S, R, K)), rng.standard_normal((S, N, R))
    alphas, ranks = np.array([0.5, -2.0, 1.0]), np.array([16, 3, 0])
    starts, ids = [1, 4, 4, 9, 11, 12], [1, 0, 0, -1, 2]
    base, out = rng.standard_normal((M, N)), rng.standard_normal((M, N))
    res, _, _, _ = batch.lora_batch(x, down, up, alphas, ranks, starts, ids, base, 0, out)
    who = {1: 1, 2: 1, 3: 1, 4: 0, 5: 0, 6: 0, 7: 0, 8: 0, 9: None, 10: None, 11: 2}
    for m in range(M):
        if m not in who:
            want = out[m]
        else:
            W = np.zeros((N, K))
            if who[m] is not None:
                s = who[m]
                W = alphas[s] * up[s, :, :ranks[s]] @ down[s, :ranks[s]]
            want = base[m] + W @ x[m]
        assert np.allclose(res[m], want, rtol=1e-12, atol=1e-12), m


def test_group_norm_equals_torch():
    rng = np.random.default_rng(6)
    for B, rows, C, G in ((2, 9, 12, 3), (1, 1, 8, 2), (3, 5, 6, 1)):
        x = rng.standard_normal((B, rows, C)) + 3
        w, b = rng.standard_normal(C), rng.standard_normal(C)
        ms, mt = rng.standard_normal((B, C)), rng.standard_normal((B, C))
        ref = torch.nn.functional.group_norm(torch.from_numpy(x).permute(0, 2, 1), G, torch.from_numpy(w),
                                             torch.from_numpy(b), 1e-5).permute(0, 2, 1).numpy()
        ref = ref * (1 + ms[:, None]) + mt[:, None]
        for kind, f in ((0, lambda t: t), (1, lambda t: torch.nn.functional.gelu(t, approximate="tanh")),
                        (2, torch.nn.functional.silu)):
            got, _ = batch.group_norm(x, G, 1e-5, w, b, ms, mt, kind)
            assert np.allclose(got, f(torch.from_numpy(ref)).numpy(), rtol=1e-10, atol=1e-10)
