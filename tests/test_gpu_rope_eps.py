"""The norm without an epsilon, against the float64 oracle: forward, gradient
and append, at token counts that leave lanes of the last wave without a token
(bounds derived in token_util and below)."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from oracle import tokens as ref
from token_util import E32, TINY, U, Batch, host, make_rope, packed, turned_bound, values, within

pytestmark = pytest.mark.gpu

# dim, sections, adjacent
WIDTHS = [(16, (8,), False), (80, (8, 16, 16), True), (128, (16, 24, 24), False), (256, (), False)]


def _weights(rng, dim, dtype):
    t = values(rng, (dim,), dtype, 0.3)[0] + 1
    return t, host(t)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [1, 7, 67, 520])
@pytest.mark.parametrize("dim,sections,adjacent", WIDTHS)
def test_norm_without_eps(n, dim, sections, adjacent, dtype):
    rng = np.random.default_rng(51)
    pos_t, pos, f_t, f = make_rope(rng, sections, n)
    rope = dws.Rope(f_t, sections, int(adjacent))
    half = sum(sections)
    q, k = packed(rng, n, [3, 2], dim, dtype)
    dys = [values(rng, x[1].shape, dtype) for x in (q, k)]
    ws = [_weights(rng, dim, dtype) for _ in range(2)]
    y = dws.bevpool_qk_norm_rope(q[0], k[0], pos_t, rope, ws[0][0], ws[1][0], 0.0)
    g = dws.bevpool_qk_norm_rope_backward(dys[0][0], dys[1][0], q[0], k[0], pos_t, rope, ws[0][0],
                                          ws[1][0], 0.0)
    torch.cuda.synchronize()
    for i, (x, dy, w) in enumerate(zip((q, k), dys, ws)):
        n64 = ref.norm(x[1], w[1], 0.0)
        want = ref.turn(n64, pos, f, sections, adjacent)
        within(host(y[i]), want, turned_bound(n64, half, adjacent, dim, dtype, want), "y")
        dx, dw = ref.norm_turn_backward(dy[1], x[1], w[1], 0.0, pos, f, sections, adjacent)
        # |g| and its pair, and the sizes of the terms of dx and dw; each term is
        # a product of a few factors that are within (dim / 2 + 16) e, and the sums
        # have dim terms (dx) or one for each row (dw)
        size = np.abs(dy[1])
        part = turned_bound(size, half, adjacent, dim, "f32", 0 * size) / ((dim / 2 + 16) * E32)
        r = 1 / np.sqrt((x[1] * x[1]).mean(-1, keepdims=True))
        xh = np.abs(x[1] * r)
        aw = np.abs(w[1])
        big = r * (aw * part + xh * (xh * aw * part).mean(-1, keepdims=True))
        within(host(g[i]), dx, big * (2 * dim + 64) * E32 * (1 + U[dtype]) + U[dtype] * np.abs(dx) +
               TINY[dtype], "dx")
        terms = n * x[1].shape[1]
        within(host(g[2 + i]), dw, (part * xh).sum((0, 1)) * (terms + dim + 64) * E32 +
               U["f32"] * np.abs(dw), "dw")


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "e4m3")])
@pytest.mark.parametrize("new,dim", [([1], 128), ([3, 0, 4], 16), ([60, 7], 80)])
def test_append_without_eps(new, dim, dtype, cache):
    """Keys of the cache and queries; the lanes without a token store nothing."""
    rng = np.random.default_rng(52)
    b = Batch(rng, new, [5] * len(new), 2, dim, 16, dtype, cache, lead=1, tail=2)
    q, k, v = packed(rng, b.n, [3, 2, 2], dim, dtype)
    wq, wk = (_weights(rng, dim, dtype) for _ in range(2))
    got = dws.bevpool_kv_append(k[0], v[0], b.pool, b.batch, None, None, q=q[0], q_weight=wq[0],
                                k_weight=wk[0], eps=0.0)
    torch.cuda.synchronize()
    inside = slice(1, b.n - 2)
    nq, nk = ref.norm(q[1], wq[1], 0.0), ref.norm(k[1], wk[1], 0.0)
    within(host(got)[inside], nq[inside], turned_bound(nq, 0, False, dim, dtype, nq)[inside], "q")
    kc, vc, hit = ref.append(nk, v[1], b.k0, b.v0, b.offsets, b.kv, b.table)
    on = np.broadcast_to(hit[:, None, :, None], kc.shape)
    assert hit.sum() == sum(new)
    for t, want, scale, slack in ((b.kt, kc, b.k_scale, dim / 2 + 18), (b.vt, vc, b.v_scale, 2)):
        z = want[on] / scale
        if cache == "e4m3":
            z = np.clip(z, -448, 448)
        err = np.abs(z) * slack * E32
        within(host(t)[on], z, err * (1 + U[cache]) + U[cache] * np.abs(z) + TINY[cache])
