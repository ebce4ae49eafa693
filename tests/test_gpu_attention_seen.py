"""svdq_attention: what a row sees reaches it.  Values that are not numbers under weights of 0, scores of
minus infinity, scores past fp32's range; in calls whose keys are cut in parts and in others."""
import pytest
import torch

import test_gpu_attention as attn

pytestmark = pytest.mark.gpu
U, DEV, INF = attn.U, attn.DEV, float("inf")
# two waves to a row, whole row tiles, keys in parts (joined by four waves a row, and by one)
SHAPES = {"few": dict(qs=attn.cut(40), ks=attn.cut(700), H=2, G=1, D=64),
          "many": dict(qs=attn.cut(130, 3), ks=attn.cut(700, 64), H=80, G=80, D=64),
          "parts": dict(qs=[0, 1, 2, 3], ks=attn.cut(3000, 100, 900), H=4, G=2, D=128),
          "parts of many rows": dict(qs=attn.cut(590), ks=attn.cut(9000), H=8, G=8, D=64)}


def case(shape, **kw):
    c = attn.Case(4, **SHAPES[shape], **kw)
    assert (c.nb > 0) == shape.startswith("parts")
    return c


@pytest.mark.parametrize("far", [2, 70, 550, -1])
@pytest.mark.parametrize("bad", [float("nan"), INF, -INF])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_values_under_weights_of_0(shape, bad, far):
    """The first key takes all of the weight, exp(-2000) of it is left for key `far` (-1: the
    last), whose value is none."""
    print(shape, bad, far, flush=True)
    c = case(shape)
    far = far % c.ks[1]
    c.q.zero_()
    c.k.zero_()
    c.q[:, ::c.D] = 200.0
    c.k[0, ::c.D] = 10.0 * c.D ** 0.5
    c.v[far, 3::c.D] = bad
    c.call()
    torch.cuda.synchronize()
    rows = slice(0, c.qs[1])        # of the first segment
    out = c.out[rows].reshape(c.qs[1], c.H, c.D)
    assert not bool(torch.isfinite(out[..., 3]).any())
    want = c.v[0].reshape(1, c.G, c.D).repeat_interleave(c.H // c.G, 1).expand_as(out)
    keep = torch.arange(c.D, device=DEV) != 3
    assert torch.equal(out[..., keep], want[..., keep])


@pytest.mark.parametrize("shape", list(SHAPES))
def test_values_under_scores_of_minus_infinity(shape):
    """The last 200 keys of the first segment have the score minus infinity: they change nothing, but for the
    column of a value that is not a number."""
    c, n = case(shape), SHAPES[shape]["ks"][1]
    c.q[:, ::c.D] = 1.0
    c.k[n - 200:n, ::c.D] = -INF
    c.v[n - 200:n] = 1e4
    c.call()
    torch.cuda.synchronize()
    c.ks, full = [0, n - 200] + c.ks[2:], c.ks
    c.n, qs = 1, c.qs
    for a, b, h, (ref, wabs, wroot, size, _), keys in c.parts():
        got = c.out[a:b, h * c.D:h * c.D + c.D].double()
        tol = wabs * (2 * (2 * c.D + 4) * U * size + (keys + 1000) * U) + torch.minimum(2.0 ** -8 * wabs, 7 * 2.0 ** -8 * wroot)
        assert bool(((got - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all()), h
    ref, c.n, c.ks = c.out.clone(), len(qs) - 1, full
    c.v[n - 1, 3::c.D] = float("nan")
    c.call()
    torch.cuda.synchronize()
    out, ref = (t[:c.qs[1]].reshape(-1, c.H, c.D) for t in (c.out, ref))
    keep = torch.arange(c.D, device=DEV) != 3
    assert bool(torch.isnan(out[..., 3]).all()) and torch.equal(out[..., keep], ref[..., keep])


@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True)])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_keys_of_minus_infinity_weigh_nothing(shape, cap, bias):
    """As above for single keys among others, with values that would show."""
    c = case(shape, cap=cap, bias=bias)
    n = SHAPES[shape]["ks"][1]
    bad = torch.zeros(c.k.shape[0], dtype=torch.bool, device=DEV)
    bad[3:n:61] = True
    c.q[:, ::c.D] = 1.0
    c.k[bad, ::c.D] = -INF
    c.v[bad] = 1e4
    c.call()
    torch.cuda.synchronize()
    got = c.out.clone()
    c.v[bad] = 0.0
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(got, c.out) and bool((got[:c.qs[1], :c.H * c.D].abs() < 1e3).all())


@pytest.mark.parametrize("shape", list(SHAPES))
def test_all_scores_minus_infinity(shape):
    """Weighs nothing: zeros, as of a row that sees no key."""
    c = case(shape)
    c.q[:, ::c.D] = 1.0
    c.k[:, ::c.D] = -INF
    c.call()
    torch.cuda.synchronize()
    assert bool((c.out[:c.qs[-1]] == 0.0).all())


@pytest.mark.parametrize("shape", list(SHAPES))
def test_scores_at_the_end_of_the_range(shape):
    """The largest score takes all of the weight up to 2^127; a row with scores past that is no number.  The
    largest scale, and scores of 2^7."""
    c = case(shape)
    c.q.zero_()
    c.k.zero_()
    c.q[:, ::c.D] = 2.0 ** 63
    for i in range(c.n):
        c.k[c.ks[i], ::c.D] = 2.0 ** 63
    c.scale = 1.0
    c.call()
    torch.cuda.synchronize()
    for i in range(c.n):
        out = c.out[c.qs[i]:c.qs[i + 1]].reshape(-1, c.H, c.D)
        want = c.v[c.ks[i]].reshape(1, c.G, c.D).repeat_interleave(c.H // c.G, 1).expand_as(out)
        assert torch.equal(out, want)
    whole = c.out.clone()
    c.scale = 3.0
    c.call()
    torch.cuda.synchronize()
    assert bool(torch.isnan(c.out[:c.qs[-1]]).all())
    c.q[:, ::c.D] = 2.0 ** -60
    for i in range(c.n):
        c.k[c.ks[i], ::c.D] = 2.0 ** -60
    c.scale = 2.0 ** 127
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out, whole)


@pytest.mark.parametrize("D", [32, 64, 96, 128])
def test_infinite_values_in_every_head(D):
    """As test_gpu_attention's test_infinite_values_where_seen, for every one of 160 heads."""
    c, ref = (attn.Case(8, attn.cut(100), 160, 80, D, causal=True) for _ in range(2))
    ref.call()
    c.v[50, 3::D], c.v[60, 4::D], c.v[70, 5::D] = INF, -INF, float("nan")
    c.v[52, 7::D], c.v[80, 7::D] = INF, -INF
    c.call()
    torch.cuda.synchronize()
    o, r = (t.float().reshape(100, 160, D) for t in (c.out, ref.out))
    assert bool((o[50:, :, 3] == INF).all()) and bool((o[60:, :, 4] == -INF).all()) and bool(torch.isnan(o[70:, :, 5]).all())
    assert bool((o[52:80, :, 7] == INF).all()) and bool(torch.isnan(o[80:, :, 7]).all())
    for col, first in ((3, 50), (4, 60), (5, 70), (7, 52)):
        o[first:, :, col] = r[first:, :, col]
    assert torch.equal(o, r)


@pytest.mark.parametrize("bad", [INF, -INF])
@pytest.mark.parametrize("G", [2, 80])
def test_rows_that_see_infinite_values_say_so(bad, G):
    """Keys are numbers: rows that see an infinite value have it or its sum with the other sign, the others
    are as without it."""
    c, ref = (attn.Case(6, attn.cut(70, 90, 133), 2 * G, G, 72, causal=True, prefix=[0, 3, 0], tail=40) for _ in range(2))
    ref.call()
    hit = torch.zeros(c.Mq, dtype=torch.bool, device=DEV)
    for r, end in {20: 70, 100: 160, 165: 293, 292: 293}.items():
        c.v[r] = bad
        hit[r:end] = True
    c.v[300:] = bad
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out[~hit], ref.out[~hit])
    assert bool((c.out[hit] == bad).all())
