"""From camera features to attention over earlier frames, in one program: each
frame is pooled into a BEV grid (bf16 cells), a cell's channels are its query,
key and value heads, and its token joins the cache and reads it.  Eager and as
a captured graph, against the float64 oracles (bounds: the pooling's bar and
one rounding, then those derived in token_util from the pooled values)."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
import oracle
from gpu_util import TOL, gpu_map, map_to_numpy, oracle_reference, to_gpu
from oracle import tokens as ref
from token_util import DT, E32, TINY, U, dev, host, make_rope, turned_bound, values, within

pytestmark = pytest.mark.gpu

IMG, D, H, W, ROWS, COLS = 2, 5, 4, 11, 9, 8
CELLS, FRAMES, PAGE = ROWS * COLS, 4, 16
HQ, HK, DIM, SECTIONS = 4, 2, 32, (4, 6, 6)
C = (HQ + 2 * HK) * DIM


def _frame(rng):
    depth = rng.random((IMG, D, H, W)).astype(np.float16)
    return depth, rng.standard_normal((IMG, H, W, C)).astype(np.float16)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_pool_then_tokens(cache):
    oracle.build(force=False)
    rng = np.random.default_rng(131)
    # some cells stay empty, some points fall outside
    point_cell = rng.integers(-8, CELLS - 5, IMG * D * H * W)
    m = gpu_map(np.maximum(point_cell, -1), IMG, D, H, W, CELLS)
    ref_map = map_to_numpy(m)
    k_scale, v_scale = (0.03, 0.02) if cache == "e4m3" else (1.0, 1.0)
    width = -(-FRAMES * CELLS // PAGE)
    kt, vt = (torch.full((width + 2, HK, PAGE, DIM), float("nan"), device=dev()).to(DT[cache])
              for _ in range(2))
    pool = dws.PagedCache(kt, vt, k_scale, v_scale)
    table = rng.permutation(width + 2)[:width].astype(np.int32)[None]
    lens, pos = to_gpu(np.zeros(1, np.int32)), to_gpu(np.zeros((3, CELLS), np.int32))
    batch = dws.PagedBatch(to_gpu(np.array([0, CELLS], np.int32)), lens, to_gpu(table))
    _, _, f_t, f = make_rope(rng, SECTIONS, 1)
    rope = dws.Rope(f_t, SECTIONS)
    wq, wk = (values(rng, (DIM,), "bf16", 0.3) for _ in range(2))
    depth_t, feat_t = (to_gpu(x) for x in _frame(rng))

    def step():
        cells = dws.bevpool_forward_ex(depth_t, feat_t, m, CELLS, torch.bfloat16)
        heads = cells.view(CELLS, HQ + 2 * HK, DIM)
        q, k, v = heads[:, :HQ], heads[:, HQ:HQ + HK], heads[:, HQ + HK:]
        qt = dws.bevpool_kv_append(k, v, pool, batch, pos, rope, q=q, q_weight=wq[0], k_weight=wk[0])
        return cells, qt, dws.bevpool_paged_attention(qt, pool, batch, causal=False)

    def load(frame):
        depth, feat = _frame(rng)
        depth_t.copy_(to_gpu(depth))
        feat_t.copy_(to_gpu(feat))
        i = np.arange(CELLS)
        point = np.stack([np.full(CELLS, frame), i // COLS, i % COLS]).astype(np.int32)
        pos.copy_(to_gpu(point))
        lens.fill_((frame + 1) * CELLS)
        return depth, feat, point

    def check(got, inputs, frame):
        depth, feat, point = inputs
        want, size = oracle_reference(depth, feat, "f16", 1.0, C, ref_map, CELLS)
        tol = TOL["f16"] * size
        within(host(got[0]), want, tol + U["bf16"] * (np.abs(want) + tol) + TINY["bf16"], "cells")
        heads = host(got[0]).reshape(CELLS, -1, DIM)
        q, k, v = heads[:, :HQ], heads[:, HQ:HQ + HK], heads[:, HQ + HK:]
        nq, nk = ref.norm(q, wq[1], 1e-6), ref.norm(k, wk[1], 1e-6)
        tq, tk = (ref.turn(x, point, f, SECTIONS, False) for x in (nq, nk))
        within(host(got[1]), tq, turned_bound(nq, 16, False, DIM, "bf16", tq), "q")
        # the frame's places of the cache
        j = np.arange(frame * CELLS, (frame + 1) * CELLS)
        k64, v64 = host(kt) * k_scale, host(vt) * v_scale
        at = table[0, j // PAGE], slice(None), j % PAGE
        for stored, x, n, scale in ((k64, tk, nk, k_scale), (v64, v, None, v_scale)):
            err = 2 * E32 * np.abs(x) + U[cache] * np.abs(x) + TINY[cache] * scale
            if n is not None:
                err = err + turned_bound(n, 16, False, DIM, "f32", tk) * (1 + U[cache])
            x = np.clip(x, -448 * scale, 448 * scale) if cache == "e4m3" else x
            within(stored[at], x, err, "cache")
        want, mag, spread, seen = ref.attention(host(got[1]), k64, v64, [0, CELLS],
                                                [(frame + 1) * CELLS], table, DIM ** -0.5, False, 0)
        u = U["f16" if cache == "e4m3" else "bf16"]
        rel = (u + 4 * (DIM + 8) * E32 * spread + 2.0 ** -20 + 2 * seen * E32 + 2.0 ** -20)[..., None]
        within(host(got[2]), want, mag * rel * (1 + U["bf16"]) + U["bf16"] * np.abs(want) +
               TINY["bf16"] + (seen * 2.0 ** -25)[..., None] * np.nanmax(np.abs(v64)), "out")

    inputs = load(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    check(got, inputs, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for frame in range(FRAMES):                     # the first frame again, then the next ones
        inputs = load(frame)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in captured]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager)), frame
        check(eager, inputs, frame)
