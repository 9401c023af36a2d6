"""Pins of the token operators' oracle (CPU): closed forms, torch's float64
autograd and softmax, finite differences and hand-worked cases."""
import numpy as np
import pytest
import torch

from oracle import tokens as ref


def _rope(rng, sections):
    half = sum(sections)
    return (10000.0 ** (-np.arange(half) / max(half, 1))).astype(np.float32)


@pytest.mark.parametrize("adjacent", [False, True])
def test_turn_by_hand(adjacent):
    x = np.arange(1.0, 17.0).reshape(1, 1, 16)
    pos = np.array([[1], [2]], np.int32)
    f = np.array([np.pi / 2] * 4 + [np.pi / 4] * 4)     # quarter turns on axis 0 and (2x) 1
    y = ref.turn(x, pos, f, (4, 4), adjacent)
    if adjacent:
        want = np.stack([-x[0, 0, 1::2], x[0, 0, 0::2]], -1).reshape(-1)
    else:
        want = np.concatenate([-x[0, 0, 8:], x[0, 0, :8]])
    assert np.allclose(y[0, 0], want, atol=1e-14)


def test_turn_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    sections, dim = (8, 4, 4), 48
    f = _rope(rng, sections)
    x, y = rng.standard_normal((2, 5, 3, dim))
    p, d = rng.integers(-50, 50, (3, 5)), np.array([[7], [-2], [30]])
    for adjacent in (False, True):
        a, b = ref.turn(x, p, f, sections, adjacent), ref.turn(y, p, f, sections, adjacent)
        assert np.allclose((a * a).sum(-1), (x * x).sum(-1))
        a2, b2 = (ref.turn(v, p + d, f, sections, adjacent) for v in (x, y))
        assert np.allclose((a * b).sum(-1), (a2 * b2).sum(-1))      # position differences only
        assert np.array_equal(a[..., 32:], x[..., 32:])
        assert np.allclose(ref.turn(a, p, f, sections, adjacent, -1.0), x)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_backward_is_the_gradient(adjacent, normed):
    rng = np.random.default_rng(1)
    sections, dim, eps = (4, 4), 32, 1e-2
    f, pos = _rope(rng, sections), rng.integers(0, 40, (2, 4))
    x, dy = rng.standard_normal((2, 4, 3, dim))
    w = 1 + 0.3 * rng.standard_normal(dim) if normed else None
    dx, dw = ref.norm_turn_backward(dy, x, w, eps, pos, f, sections, adjacent)

    def loss(x, w):
        return (ref.norm_turn(x, w, eps, pos, f, sections, adjacent) * dy).sum()

    h = 1e-5
    for _ in range(30):
        at = tuple(rng.integers(0, n) for n in x.shape)
        up, dn = x.copy(), x.copy()
        up[at] += h
        dn[at] -= h
        assert abs((loss(up, w) - loss(dn, w)) / (2 * h) - dx[at]) < 1e-7
    if not normed:
        assert dw is None
        return
    for i in range(0, dim, 5):
        up, dn = w.copy(), w.copy()
        up[i] += h
        dn[i] -= h
        assert abs((loss(x, up) - loss(x, dn)) / (2 * h) - dw[i]) < 1e-7


def test_norm_is_rms():
    x = np.full((1, 1, 16), -3.0)
    assert np.allclose(ref.norm(x, np.full(16, 2.0), 0.0), -2.0)
    assert np.array_equal(ref.norm(x, None, 0.0), x)


def test_append_by_hand():
    k = np.arange(5.0)[:, None, None] * np.ones((5, 1, 16)) + 1
    cache = np.zeros((3, 1, 16, 16))
    table = np.array([[2, 0], [1, 7]])
    # sequence 0: tokens 0-2 at places 15, 16, 17; sequence 1: tokens 3, 4 at 31 and 32
    kc, vc, hit = ref.append(k, -k, cache, cache, [0, 3, 5], [18, 33], table)
    assert kc[2, 0, 15, 0] == 1 and kc[0, 0, 0, 0] == 2 and kc[0, 0, 1, 0] == 3
    assert hit.sum() == 3                       # page 7 is no page, place 32 has no entry
    assert (vc[hit.nonzero()[0], 0, hit.nonzero()[1]] < 0).all()


@pytest.mark.parametrize("causal", [False, True])
def test_attention_matches_torch_softmax(causal):
    rng = np.random.default_rng(2)
    page, hk, dim, hq = 16, 2, 16, 6
    kc, vc = rng.standard_normal((2, 5, hk, page, dim))
    q = rng.standard_normal((7, hq, dim))
    table = np.array([[3, 0, 4]])
    out, mag, _, seen = ref.attention(q, kc, vc, [0, 7], [40], table, 0.3, causal, 0)
    k = torch.tensor(kc[table[0]]).transpose(1, 2).reshape(48, hk, dim)[:40]
    v = torch.tensor(vc[table[0]]).transpose(1, 2).reshape(48, hk, dim)[:40]
    x = torch.einsum("thd,jhd->htj", torch.tensor(q), k.repeat_interleave(3, 1)) * 0.3
    if causal:
        x = x.masked_fill(torch.arange(40)[None, None] > torch.arange(33, 40)[None, :, None],
                          -np.inf)
    want = torch.einsum("htj,jhd->thd", torch.softmax(x, -1), v.repeat_interleave(3, 1))
    assert np.allclose(out, want.numpy())
    assert (mag >= np.abs(out) - 1e-12).all()
    assert (seen[:, 0] == (np.arange(34, 41) if causal else 40)).all()


def test_attention_masks():
    rng = np.random.default_rng(3)
    kc, vc = rng.standard_normal((2, 4, 1, 16, 16))
    q = rng.standard_normal((4, 1, 16))
    table = np.array([[0, -1, 2], [1, 1, 1]])
    # a window of one place: the weight is 1 on the token's own value
    out, *_ = ref.attention(q, kc, vc, [0, 2, 2], [48, 0], table, 1.0, True, 1)
    assert np.allclose(out[0], vc[2, 0, 14]) and np.allclose(out[1], vc[2, 0, 15])
    assert np.isnan(out[2:]).all()                     # outside every sequence
    # places on no page are not there; more new tokens than cached ones: the first see none
    out, _, _, seen = ref.attention(q, kc, vc, [0, 4, 4], [2, 0], table, 1.0, True, 0)
    assert (out[:2] == 0).all() and (seen[:, 0] == [0, 0, 1, 2]).all()
    _, _, _, seen = ref.attention(q, kc, vc, [0, 1, 1], [48, 0], table, 1.0, True, 0)
    assert seen[0, 0] == 32
    # a uniform softmax averages
    out, *_ = ref.attention(0 * q, kc, vc, [0, 1, 1], [16, 0], table, 1.0, True, 0)
    assert np.allclose(out[0, 0], vc[0, 0].mean(0))
