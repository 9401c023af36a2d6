"""Query/key norm with rotary positions, and its gradient, against the
float64 oracle (bounds derived in token_util)."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from oracle import tokens as ref
from token_util import (DT, E32, TINY, U, dev, host, make_rope, packed, turned_bound, values,
                        within)

pytestmark = pytest.mark.gpu
EPS = 1e-6

# tokens, query heads, key heads, dim, sections, adjacent
SHAPES = [
    (1, 1, 0, 16, (8,), False),
    (1, 8, 2, 64, (8, 12, 12), False),
    (7, 3, 1, 16, (4, 4), True),
    (5, 2, 2, 32, (16,), True),
    (3, 5, 5, 80, (12, 12), True),
    (67, 4, 4, 80, (8, 16, 16), False),
    (33, 6, 2, 96, (24, 24), False),
    (130, 16, 4, 128, (16, 24, 24), False),
    (9, 7, 1, 144, (8, 8, 8, 8), True),
    (65, 2, 1, 256, (32, 48, 48), True),
    (21, 3, 2, 256, (16, 0, 16), False),
    (12, 4, 2, 128, (), False),
    (1030, 3, 1, 48, (8, 8), False),
]


def _inputs(shape, dtype, norm, seed, wdtype=None, pack=True):
    n, hq, hk, dim, sections, adjacent = shape
    rng = np.random.default_rng(seed)
    pos_t, pos, f_t, f = make_rope(rng, sections, n)
    rope = dws.Rope(f_t, sections, dws.ROPE_ADJACENT if adjacent else dws.ROPE_HALVES)
    heads = [hq, hk, 1] if hk else [hq, 1]
    qkv = packed(rng, n, heads, dim, dtype) if pack else \
        [values(rng, (n, h, dim), dtype) for h in heads]
    q, k = qkv[0], qkv[1] if hk else (None, None)
    ws = [None, None]
    if norm:
        ws = [values(rng, (dim,), wdtype or dtype, 0.3) for _ in range(2)]
        ws = [((t + 1).to(t.dtype), None) for t, _ in ws]
        ws = [(t, host(t)) for t, _ in ws]
    return rng, rope, pos_t, pos, f, q, k, [w or (None, None) for w in ws]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("norm", [True, False])
def test_forward(shape, dtype, norm):
    n, hq, hk, dim, sections, adjacent = shape
    _, rope, pos_t, pos, f, q, k, ws = _inputs(shape, dtype, norm, 1)
    got = dws.bevpool_qk_norm_rope(q[0], k[0], pos_t, rope, ws[0][0], ws[1][0], EPS)
    torch.cuda.synchronize()
    for y, x, w in zip(got, (q, k), ws):
        if x[0] is None:
            assert y is None
            continue
        n64 = ref.norm(x[1], w[1], EPS)
        want = ref.turn(n64, pos, f, sections, adjacent)
        within(host(y), want, turned_bound(n64, sum(sections), adjacent, dim, dtype, want))


def _grad_bounds(dy, x, w, g, dx, dim, dtype, half, adjacent):
    # |g| and its pair enter with the angle's error; everything else is a few
    # roundings of terms no larger than those summed here
    part = turned_bound(np.abs(dy), half, adjacent, dim, "f32", 0 * dy) / ((dim / 2 + 16) * E32)
    if w is None:
        return part * 16 * E32 + U[dtype] * np.abs(dx) + TINY[dtype], None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    xh = np.abs(x * r)
    big = r * (np.abs(w) * part + xh * (xh * np.abs(w) * part).mean(-1, keepdims=True))
    bx = big * (2 * dim + 64) * E32 * (1 + U[dtype]) + U[dtype] * np.abs(dx) + TINY[dtype]
    terms = dy.shape[0] * dy.shape[1]
    return bx, (part * xh).sum((0, 1)) * (terms + dim + 64) * E32


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("norm", [True, False])
def test_backward(shape, dtype, norm):
    n, hq, hk, dim, sections, adjacent = shape
    rng, rope, pos_t, pos, f, q, k, ws = _inputs(shape, dtype, norm, 2)
    dys = [values(rng, (n, h, dim), dtype) if h else (None, None) for h in (hq, hk)]
    got = dws.bevpool_qk_norm_rope_backward(dys[0][0], dys[1][0], q[0], k[0], pos_t, rope,
                                            ws[0][0], ws[1][0] if hk else None, EPS)
    torch.cuda.synchronize()
    for i, (dy, x, w) in enumerate(zip(dys, (q, k), ws)):
        if dy[0] is None:
            assert got[i] is None and got[2 + i] is None
            continue
        dx, dw = ref.norm_turn_backward(dy[1], x[1], w[1], EPS, pos, f, sections, adjacent)
        bx, bw = _grad_bounds(dy[1], x[1], w[1], None, dx, dim, dtype, sum(sections), adjacent)
        within(host(got[i]), dx, bx, "dx")
        if norm:
            assert got[2 + i].dtype == torch.float32
            within(host(got[2 + i]), dw, bw + U["f32"] * np.abs(dw), "dw")
        else:
            assert got[2 + i] is None


@pytest.mark.parametrize("side", ["q", "k"])
def test_backward_against_differences(side):
    """The kernel's own gradient against differences of its own forward, in
    fp32: a step of 2^-6 leaves an error of h^2 f''' / 6 (below 2e-4 here, the
    third derivative of the loss along one coordinate being under 5) and
    rounding of 1e-6 * |loss terms| / h."""
    n, heads, dim, sections = 2, 2, 32, (8, 8)
    rng = np.random.default_rng(3)
    pos_t, _, f_t, _ = make_rope(rng, sections, n, 20)
    rope = dws.Rope(f_t, sections)
    x, _ = values(rng, (n, heads, dim), "f32", 2.0)
    dy, _ = values(rng, (n, heads, dim), "f32")
    w = values(rng, (dim,), "f32", 0.2)[0] + 1
    one = torch.ones_like(x[:, :1])

    def forward(x, w):
        if side == "q":
            return dws.bevpool_qk_norm_rope(x, None, pos_t, rope, w, None, EPS)[0]
        return dws.bevpool_qk_norm_rope(one, x, pos_t, rope, None, w, EPS)[1]

    if side == "q":
        dx, _, dw, _ = dws.bevpool_qk_norm_rope_backward(dy, None, x, None, pos_t, rope, w, None,
                                                         EPS)
    else:
        _, dx, _, dw = dws.bevpool_qk_norm_rope_backward(one, dy, None, x, pos_t, rope, None, w,
                                                         EPS)
    h = 2.0 ** -6
    for i in range(0, x.numel(), 5):
        up, dn = x.clone(), x.clone()
        up.view(-1)[i] += h
        dn.view(-1)[i] -= h
        d = float(((forward(up, w) - forward(dn, w)).double() * dy).sum() / (2 * h))
        assert abs(d - float(dx.view(-1)[i])) < 3e-4, i
    for i in range(0, dim, 3):
        up, dn = w.clone(), w.clone()
        up[i] += h
        dn[i] -= h
        d = float(((forward(x, up) - forward(x, dn)).double() * dy).sum() / (2 * h))
        assert abs(d - float(dw[i])) < 3e-4, i


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_weights_in_fp32_and_one_side_only(dtype):
    shape = (40, 4, 2, 64, (8, 12, 12), False)
    n, hq, hk, dim, sections, adjacent = shape
    _, rope, pos_t, pos, f, q, k, ws = _inputs(shape, dtype, True, 4, "f32")
    for use in ((1, 1), (1, 0), (0, 1)):
        w = [x if u else (None, None) for x, u in zip(ws, use)]
        got = dws.bevpool_qk_norm_rope(q[0], k[0], pos_t, rope, w[0][0], w[1][0], EPS)
        grad = dws.bevpool_qk_norm_rope_backward(q[0], k[0], q[0], k[0], pos_t, rope, w[0][0],
                                                 w[1][0], EPS)
        for i, (x, wi) in enumerate(zip((q, k), w)):
            n64 = ref.norm(x[1], wi[1], EPS)
            want = ref.turn(n64, pos, f, sections, adjacent)
            within(host(got[i]), want, turned_bound(n64, 32, adjacent, dim, dtype, want))
            dx, dw = ref.norm_turn_backward(x[1], x[1], wi[1], EPS, pos, f, sections, adjacent)
            bx, bw = _grad_bounds(x[1], x[1], wi[1], None, dx, dim, dtype, 32, adjacent)
            within(host(grad[i]), dx, bx)
            if wi[0] is not None:
                within(host(grad[2 + i]), dw, bw + U["f32"] * np.abs(dw))


def test_far_positions_keep_their_angle():
    """At positions near 2^31 an fp32 angle is off by whole turns; the bound
    is that of near ones plus the fp64 product's 2^-53 of 2^31 radians."""
    n, dim, sections = 64, 32, (8, 8)
    rng = np.random.default_rng(5)
    _, _, f_t, f = make_rope(rng, sections, n)
    pos = rng.integers(2 ** 31 - 5000, 2 ** 31, (2, n)).astype(np.int32)
    pos[1] = -pos[1]
    x, xh = values(rng, (n, 2, dim), "f32")
    y, _ = dws.bevpool_qk_norm_rope(x, None, torch.from_numpy(pos).to(dev()),
                                    dws.Rope(f_t, sections))
    # the reference angle itself: exact products (24 + 31 bits) need long double
    th = pos[[0] * 8 + [1] * 8].astype(np.longdouble) * f[:, None].astype(np.longdouble)
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    th = (th - np.rint(th / two_pi) * two_pi).astype(np.float64)
    c, s = np.cos(th).T[:, None], np.sin(th).T[:, None]
    want = np.concatenate([xh[..., :16] * c - xh[..., 16:] * s, xh[..., 16:] * c + xh[..., :16] * s],
                          -1)
    slack = (np.abs(xh[..., :16]) + np.abs(xh[..., 16:])) * 2.0 ** -20
    within(host(y), want, turned_bound(xh, 16, False, dim, "f32", want) +
           np.concatenate([slack, slack], -1))


@pytest.mark.parametrize("shape,dtype", [((20011, 3, 2, 128, (16, 24, 24), False), "bf16"),
                                         ((50021, 2, 1, 48, (8, 8), True), "f32")])
def test_backward_many_tokens(shape, dtype):
    """More token groups than waves: each walks over several, and the weight
    gradient is a sum over all of them."""
    n, hq, hk, dim, sections, adjacent = shape
    rng, rope, pos_t, pos, f, q, k, ws = _inputs(shape, dtype, True, 10)
    dys = [values(rng, (n, h, dim), dtype) for h in (hq, hk)]
    got = dws.bevpool_qk_norm_rope_backward(dys[0][0], dys[1][0], q[0], k[0], pos_t, rope,
                                            ws[0][0], ws[1][0], EPS)
    torch.cuda.synchronize()
    for i, (dy, x, w) in enumerate(zip(dys, (q, k), ws)):
        dx, dw = ref.norm_turn_backward(dy[1], x[1], w[1], EPS, pos, f, sections, adjacent)
        bx, bw = _grad_bounds(dy[1], x[1], w[1], None, dx, dim, dtype, sum(sections), adjacent)
        within(host(got[i]), dx, bx, "dx")
        # the terms' own errors, and a sum of which a lane adds at most 2^7 terms in a
        # row and the strips under 2^9 more: within 2^10 e of the sum of the sizes
        bw = bw * (2.0 ** 10 + dim + 64) / (n * x[1].shape[1] + dim + 64)
        within(host(got[2 + i]), dw, bw + U["f32"] * np.abs(dw), "dw")


def test_in_place_and_given_outputs():
    shape = (50, 4, 2, 80, (8, 16, 16), False)
    _, rope, pos_t, pos, f, q, k, ws = _inputs(shape, "bf16", True, 6)
    w = [x[0] for x in ws]
    y = dws.bevpool_qk_norm_rope(q[0], k[0], pos_t, rope, *w)
    g = dws.bevpool_qk_norm_rope_backward(*y, q[0], k[0], pos_t, rope, *w)
    out = [torch.full((50, h + 1, 80), 7.0, dtype=torch.bfloat16, device=dev())[:, :h]
           for h in (4, 2)]
    z = dws.bevpool_qk_norm_rope(q[0], k[0], pos_t, rope, *w, q_out=out[0], k_out=out[1])
    assert z[0] is out[0] and all(torch.equal(a, b) for a, b in zip(z, y))
    # the gradient into its own input, and the forward into its own input
    dy = [v.clone() for v in y]
    gi = dws.bevpool_qk_norm_rope_backward(*dy, q[0], k[0], pos_t, rope, *w, dq=dy[0], dk=dy[1])
    assert gi[0] is dy[0] and all(torch.equal(a, b) for a, b in zip(gi, g))
    dws.bevpool_qk_norm_rope(q[0], k[0], pos_t, rope, *w, q_out=q[0], k_out=k[0])
    assert torch.equal(q[0], y[0]) and torch.equal(k[0], y[1])
    assert (out[0]._base[:, 4] == 7).all()


def test_same_bits_every_time():
    shape = (4099, 6, 2, 128, (16, 24, 24), False)
    _, rope, pos_t, _, _, q, k, ws = _inputs(shape, "bf16", True, 7)
    w = [x[0] for x in ws]
    first = None
    for _ in range(4):
        g = dws.bevpool_qk_norm_rope_backward(q[0], k[0], q[0], k[0], pos_t, rope, *w)
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, g))
        first = g


def test_non_finite_rows_stay_where_they_are():
    shape = (20, 3, 1, 64, (32,), False)
    _, rope, pos_t, _, _, q, k, ws = _inputs(shape, "f32", True, 8, pack=False)
    q[0][3, 1, 5] = float("nan")
    q[0][7, 2, 0] = float("inf")
    y, _ = dws.bevpool_qk_norm_rope(q[0], None, pos_t, rope, ws[0][0], None, EPS)
    bad = ~torch.isfinite(y).all(-1)
    assert bad[3, 1] and bad[7, 2] and int(bad.sum()) == 2
    # infinity over its own infinite root is NaN, finite over it is 0
    assert torch.isnan(y[7, 2]).any()


@pytest.mark.parametrize("adjacent", [0, 1])
def test_infinities_past_the_rotation_stay(adjacent):
    """A coordinate that is passed through has no influence on its neighbours,
    forward or backward."""
    rng = np.random.default_rng(10)
    pos_t, pos, f_t, f = make_rope(rng, (8,), 4)
    rope = dws.Rope(f_t, (8,), adjacent)
    x, xh = values(rng, (4, 1, 48), "f32")
    for at, bad in ((16, np.inf), (31, -np.inf), (32, np.nan), (47, np.inf)):
        x[:, :, at] = bad
    for y in (dws.bevpool_qk_norm_rope(x, None, pos_t, rope)[0],
              dws.bevpool_qk_norm_rope_backward(x, None, None, None, pos_t, rope)[0]):
        assert torch.equal(y[..., 16:].isfinite(), x[..., 16:].isfinite())
        assert torch.equal(y[..., 16:].nan_to_num(), x[..., 16:].nan_to_num())
        assert torch.isfinite(y[..., :16]).all()


def test_no_tokens():
    rope = dws.Rope(torch.ones(8, device=dev()), (8,))
    e = torch.empty((0, 2, 32), dtype=torch.bfloat16, device=dev())
    pos = torch.empty((1, 0), dtype=torch.int32, device=dev())
    w = torch.ones(32, dtype=torch.bfloat16, device=dev())
    y = dws.bevpool_qk_norm_rope(e, e, pos, rope, w, w)
    assert y[0].shape == e.shape
    g = dws.bevpool_qk_norm_rope_backward(e, e, e, e, pos, rope, w, w)
    assert torch.equal(g[2], torch.zeros(32, device=dev())) and torch.equal(g[3], g[2])


def test_other_stream_and_graph():
    """On a given stream, and captured: three replays with new inputs and the
    program's own work between them."""
    shape = (300, 8, 2, 128, (16, 24, 24), False)
    _, rope, pos_t, _, _, q, k, ws = _inputs(shape, "bf16", True, 9)
    w = [x[0] for x in ws]

    def step():
        y = dws.bevpool_qk_norm_rope(q[0], k[0], pos_t, rope, *w)
        return y + dws.bevpool_qk_norm_rope_backward(*y, q[0], k[0], pos_t, rope, *w)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = dws.bevpool_qk_norm_rope(q[0], k[0], pos_t, rope, *w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y[0], want[0])
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        q[0].copy_(torch.randn_like(q[0]))
        k[0].mul_(0.5)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
