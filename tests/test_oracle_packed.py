"""The fp64 forms of the packed rows' operators against what fixes them: torch's own layer norm and
softmax, rotations that keep lengths and differences of positions, closed forms."""
import torch

from oracle import packed

F64 = torch.float64


def rnd(*shape, seed=0):
    return torch.randn(*shape, dtype=F64, generator=torch.Generator().manual_seed(seed))


def test_layer_norm_is_torchs():
    x, y, w, b, mod = rnd(7, 20), rnd(7, 20, seed=1), rnd(20, seed=2), rnd(20, seed=3), rnd(3, 60, seed=4)
    seg = packed.segment_of([0, 3, 3, 7], 7)
    assert seg.tolist() == [0, 0, 0, 2, 2, 2, 2]
    g, s, t = mod[:, :20], mod[:, 20:40], mod[:, 40:]
    h, out, p = packed.layer_norm(x, y, w, b, seg, g, s, t, 1e-6)
    assert torch.allclose(h, x + g[seg] * y)
    want = torch.nn.functional.layer_norm(h, (20,), w, b, 1e-6) * (1 + s[seg]) + t[seg]
    assert torch.allclose(out, want, atol=1e-12)
    assert torch.allclose(out, p["d"] * p["rstd"] * p["A"] + p["D"])
    _, plain, _ = packed.layer_norm(x, None, None, None, seg, None, None, None, 1e-6)
    assert torch.allclose(plain, torch.nn.functional.layer_norm(x, (20,), eps=1e-6), atol=1e-12)


def test_segments_of_rows():
    assert packed.segment_of([1, 1, 4], 6).tolist() == [-1, 1, 1, 1, -1, -1]


def test_rotary_turns():
    x, pos, f = rnd(5, 2 * 8), rnd(5, 2, seed=1) * 10, rnd(4, seed=2).abs()
    axis = torch.tensor([0, 0, 1, 1])
    for halves in (False, True):
        y, size, ang = packed.rotary(x, 2, axis, pos, f, None, 0.0, halves)
        assert torch.allclose(y.reshape(5, 2, 8).norm(dim=2), x.reshape(5, 2, 8).norm(dim=2))   # lengths stay
        back, _, _ = packed.rotary(y, 2, axis, -pos, f, None, 0.0, halves)
        assert torch.allclose(back, x)
        same, _, _ = packed.rotary(x, 2, axis, pos, 0 * f, None, 0.0, halves)
        assert torch.equal(same, x)
        # products depend on the differences of positions only
        a, b = (packed.rotary(x, 2, axis, pos + c, f, None, 0.0, halves)[0].reshape(5, 2, 8)[:, 0] for c in (0.0, 3.5))
        assert torch.allclose(a @ a.t(), b @ b.t())
    one, _, _ = packed.rotary(torch.tensor([[1.0, 0.0]], dtype=F64), 1, torch.tensor([0]), torch.tensor([[1.0]], dtype=F64),
                              torch.tensor([torch.pi / 2], dtype=F64), None, 0.0, False)
    assert torch.allclose(one, torch.tensor([[0.0, 1.0]], dtype=F64), atol=1e-15)
    n, _, _ = packed.rotary(x * 3, 2, axis, pos, f, torch.ones(8, dtype=F64), 0.0, True)
    assert torch.allclose(n.reshape(5, 2, 8).pow(2).mean(dim=2), torch.ones(5, 2, dtype=F64))


def test_limits():
    assert packed.limits(3, 5, False, 0).tolist() == [5, 5, 5]
    assert packed.limits(3, 5, True, 0).tolist() == [3, 4, 5]
    assert packed.limits(4, 2, True, 0).tolist() == [0, 0, 1, 2]
    assert packed.limits(4, 4, True, 3).tolist() == [3, 3, 3, 4]
    assert packed.limits(2, 3, True, 9).tolist() == [3, 3] and packed.limits(3, 1, True, -4).tolist() == [0, 0, 1]


def test_attention_is_torchs():
    q, k, v = rnd(6, 8), rnd(9, 8, seed=1), rnd(9, 8, seed=2)
    out = packed.attention(q, k, v, 0.3, 0.0, False, 0, None)[0]
    assert torch.allclose(out, torch.softmax(0.3 * q @ k.t(), dim=1) @ v)
    out = packed.attention(q, k, v, 0.3, 2.0, True, 2, 0.25)[0]
    far = (torch.arange(6)[:, None] + 3 - torch.arange(9)).abs()
    t = 2 * torch.tanh(0.15 * q @ k.t()) - 0.25 * far
    for i in range(6):
        seen = [j for j in range(9) if j < 2 or j <= i + 3]
        assert torch.allclose(out[i], torch.softmax(t[i, seen], 0) @ v[seen])


def test_attention_without_keys_is_zero():
    q, k = rnd(4, 8), rnd(2, 8, seed=1)
    out = packed.attention(q, k, k, 1.0, 0.0, True, 0, None)[0]
    assert torch.equal(out[:2], torch.zeros(2, 8, dtype=F64)) and bool((out[2:] != 0).all())
    assert torch.equal(packed.attention(q, k[:0], k[:0], 1.0, 0.0, False, 0, None)[0], 0 * q)
