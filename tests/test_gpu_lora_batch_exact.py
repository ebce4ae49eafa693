"""svdq_lora_batch between its two products: the down-projection's result t enters the second one
with all its 24 bits, for a bf16 output too, and non-finite values of lora_up give what fp32
arithmetic gives.  The sizes reach every form of the up-projection: one launch, 16 and 32 rows a
workgroup, narrow and wide columns, every number of rank blocks."""
import numpy as np
import pytest
import torch

from test_gpu_lora_batch import Case, cuts, f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

# M, N, R, bf16 out
SIZES = [(40, 300, 16, True), (40, 300, 32, True), (40, 300, 64, True), (40, 300, 16, False), (40, 301, 64, False),
         (300, 4400, 16, True), (300, 4400, 32, True), (300, 4400, 64, True), (300, 4400, 128, True),
         (300, 4400, 16, False), (300, 4400, 128, False), (8200, 2060, 16, True), (8200, 2060, 32, True),
         (8200, 1100, 64, True), (8200, 1100, 128, True), (8200, 1028, 32, False)]


@pytest.mark.parametrize("M,N,R,bf", SIZES)
def test_t_keeps_its_bits_where_base_cancels_the_delta(M, N, R, bf):
    """Adapters of rank 1 and rows with one nonzero: t = alpha (x A) is one product, exact in fp32,
    and one rounding by alpha (u).  The delta is t B in three exact partial products, added to base
    with three roundings and stored with one.  Counted twice each: 8 u of |t B|; base is -t B
    rounded to the output's type, so most results are far smaller than what they are made of."""
    print("cancel", M, N, R, bf, flush=True)
    c = Case(M + N + R, M, 64, N, R, cuts(M // 3, M - M // 3), [0, 2], ranks=[1, 1, 1], bf=bf)
    rng = np.random.default_rng(M + R)
    x = torch.zeros(M, 64)
    x[torch.arange(M), torch.from_numpy(rng.integers(0, 64, M))] = torch.from_numpy(rng.uniform(1, 2, M).astype(np.float32))
    c.x = x.to(torch.bfloat16)
    ids = np.repeat([0, 2], [M // 3, M - M // 3])
    down, up, alpha = f64(c.down)[:, 0], f64(c.up)[:, :, 0], f64(c.alphas)
    t = alpha[ids] * np.einsum("mk,mk->m", f64(c.x), down[ids])
    delta = t[:, None] * up[ids]
    c.base = torch.from_numpy((-delta).astype(np.float32)).to(c.dt)
    c.put()
    got = c.call()
    torch.cuda.synchronize()
    res = f64(c.base) + delta
    half = 2.0 ** -8 if bf else U
    e = 8 * U * np.abs(delta)
    tol = e + half * (np.abs(res) + e) + 1e-37
    bad = np.abs(f64(got.cpu()) - res) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(f64(got.cpu()) - res) / tol).max()))


@pytest.mark.parametrize("M,N,R,bf", SIZES)
def test_infinities_of_lora_up(M, N, R, bf):
    """An infinite or NaN value of a used rank spoils its own columns alone, and there as t B does:
    t's sign decides, whatever its bits (powers of two, tiny values), and 0 and opposite infinities
    give NaN."""
    print("infinite", M, N, R, bf, flush=True)
    c = Case(M + N + R + 1, M, 64, N, R, cuts(M // 3, M - M // 3), [0, 2], ranks=[3, 3, 3], bf=bf)
    # rows' t of rank 0: x[m, 0] alone, of rank 1: x[m, 1], of rank 2: x[m, 2]
    c.down[:] = 0
    for j in range(3):
        c.down[:, j, j] = 1.0
    c.alphas[:] = 1.0
    values = torch.tensor([1.0, -1.0, 0.75, -2.0 ** -30, 2.0 ** -100, -3.0, 0.0, 2.0 ** 40, -1.0 - 2.0 ** -7])
    c.x[:, 0] = values[torch.arange(M) % len(values)].to(torch.bfloat16)
    c.x[:, 1] = 1.0
    c.x[0:M:5, 1] = -0.5
    want0 = Case.ref(c)[0]
    c.put()
    plain = c.call().clone()
    inf = float("inf")
    cols = {1: {0: inf}, 7: {0: -inf}, 64: {0: inf, 1: inf}, 100: {0: inf, 1: -inf}, 255: {2: float("nan")}, N - 1: {0: inf}}
    for n, js in cols.items():
        for j, v in js.items():
            c.up[0, n, j] = c.up[2, n, j] = v
    c.put()
    got = c.call()
    torch.cuda.synchronize()
    rest = [n for n in range(N) if n not in cols]
    assert torch.equal(got[:, rest], plain[:, rest])
    assert np.isfinite(want0).all()
    with np.errstate(invalid="ignore"):
        for n in cols:
            t = f64(c.x)[:, :3]
            terms = t * f64(c.up)[0, n, :3]
            want = terms.sum(1)
            g = f64(got[:, n].cpu())
            assert not np.isfinite(want).any()
            np.testing.assert_array_equal(np.where(np.isnan(want), 0, want), np.where(np.isnan(g), 0, g), str(n))
            np.testing.assert_array_equal(np.isnan(want), np.isnan(g), str(n))


def test_full_mantissas_and_extremes_of_t():
    """t of every size: its largest finite value, subnormals, terms with zeros in the middle; times
    a power of two."""
    M, N = 64, 72
    c = Case(5, M, 64, N, 16, [0, M], [0], ranks=[1], bf=False, S=1, base=False)
    c.x[:] = 0
    c.x[:, 0] = 1.0
    c.down[:] = 0
    c.down[0, 0, 0] = 1.0
    for t in (3.4028234e38, 1.0000001, 1.0078126, 1.00390625, -1.9999999, 2.0 ** -126, 3 * 2.0 ** -130, 1.5 + 2.0 ** -23, -0.0):
        c.alphas[:] = t
        c.up[:] = 0.25 if abs(t) > 1e30 else 1.0
        c.put()
        got = c.call(base=None)
        torch.cuda.synchronize()
        want = np.float64(np.float32(t)) * float(c.up[0, 0, 0])
        # three products that are exact, added with two roundings; bits of t below 2^-133
        assert np.abs(f64(got.cpu()) - want).max() <= abs(want) * 2 * U + 2.0 ** -133, t
