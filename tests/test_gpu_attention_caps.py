"""svdq_attention's capped scores over the whole range of caps against their fp64 form: scores far below
the cap keep their relative precision, scores far above it give the cap.

Bound of one element: as test_gpu_attention's, but that a capped score t is off by 12 u of its own size
(u = 2^-24; and the products' 2 D u of sum |q k| scale, as there), whatever the cap.  With z = 2 y log2 e,
y = score / cap: z takes 4 roundings.  Up to |z| = 1.5 t is the score (3 roundings) times tanh(y) / y, which
goes by at most a sixth of z's relative error and takes 0.4 u of its polynomial and 2 u of roundings, and one for
the product: 7 u.  Above, y > 0.51: tanh goes by at most 0.84 of z's relative error, 3.4 u; 1 / (2^z + 1) is off by
the exponential's 2 u (times 0.74), the sum's 1 u and the reciprocal's 2 u, 4.5 u, its double at most 1.1
times tanh: 4.9 u; the difference's rounding 1 u, the cap's in other units 1.5 u, the product 1 u: 12 u."""
import numpy as np
import pytest
import torch

import test_gpu_attention as attn

pytestmark = pytest.mark.gpu
U, DEV = attn.U, attn.DEV
CAPS = [1e-45, 1e-40, 1e-30, 1e-3, 0.5, 7.0, 50.0, 1e4, 1e5, 1e6, 1e8, 1e30, 3e38]
# two waves to a row, whole row tiles, keys in parts
SHAPES = {"few": dict(qs=attn.cut(100, 30), ks=attn.cut(200, 70), H=2, G=1, D=64),
          "many": dict(qs=attn.cut(130, 20), ks=attn.cut(200, 70), H=80, G=80, D=128),
          "parts": dict(qs=[0, 1, 2], ks=attn.cut(3000, 100), H=4, G=2, D=72)}


def check(c):
    for a, b, h, (ref, wabs, wroot, size, bias), n in c.parts():
        got = c.out[a:b, h * c.D:h * c.D + c.D].double()
        e = (2 * c.D + 12) * U * size + 4 * U * bias + 4 * U * 200
        tol = wabs * (2 * e + 4 * U + (n + 16) * U + 2 * U * (n // 64 + 1)) + torch.minimum(2.0 ** -8 * wabs, 7 * 2.0 ** -8 * wroot)
        tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 1e-37
        bad = ~((got - ref).abs() <= tol)
        assert not bad.any(), (a, b, h, int(bad.sum()), float(((got - ref).abs() / tol).max()))


@pytest.mark.parametrize("sharp", [1.0, 30.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("cap", CAPS)
def test_any_cap(cap, shape, bias, sharp):
    print("cap", cap, shape, bias, sharp, flush=True)
    c = attn.Case(3, cap=float(np.float32(cap)), bias=bias, sharp=sharp, **SHAPES[shape])
    assert (c.nb > 0) == (shape == "parts")
    c.q[:, :8] *= 0.01
    c.q[1::4] = 0.0                 # scores of 0 among the others
    c.call()
    torch.cuda.synchronize()
    check(c)


@pytest.mark.parametrize("G", [1, 80])
@pytest.mark.parametrize("cap", [1e-40, 1.0, 1e6, 3e38])
def test_rows_do_not_depend_on_the_rows_beside_them(cap, G):
    """Nor on whether the scores of those are far below the cap or past it, infinite or none."""
    c = attn.Case(12, attn.cut(150, 90), 2 * G, G, 64, cap=cap)
    c.call()
    torch.cuda.synchronize()
    ref = c.out.clone()
    odd = torch.arange(240, device=DEV) % 3 == 1
    for v in (1e-6, 3e4, 3e38, float("inf"), float("nan")):
        c.q[odd] = v
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(c.out[~odd], ref[~odd]), v


def test_infinite_scores_give_the_cap():
    """A row over keys whose scores are plus infinity, minus infinity and numbers near 0."""
    c = attn.Case(9, attn.cut(40), 1, 1, 64, cap=3.0)
    c.q.fill_(1.0)
    c.k.zero_()
    c.k[7], c.k[9] = float("inf"), -float("inf")
    c.call()
    torch.cuda.synchronize()
    w = torch.ones(40, dtype=torch.float64, device=DEV)
    w[7], w[9] = float(np.exp(3.0)), float(np.exp(-3.0))
    v = c.v.double()
    want, wabs = (w @ v) / w.sum(), (w @ v.abs()) / w.sum()
    tol = wabs * (2.0 ** -8 + 60 * U) * (1 + 2.0 ** -7) + 2.0 ** -8 * want.abs()
    assert bool(((c.out.double() - want).abs() <= tol).all())
