"""Infinities and NaN among the values of the cache: a coordinate of a token's
output is finite exactly if the coordinate of every value it sees is, however
small the weight (bounds of the finite ones derived in token_util)."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from oracle import tokens as ref
from token_util import E32, TINY, U, Batch, host, values, within

pytestmark = pytest.mark.gpu

# new, ctx, hq, hk, dim, table entries past the sequences
CASES = [([1], [70], 4, 2, 64, 0), ([1, 1], [900, 33], 8, 1, 64, 400), ([130], [200], 4, 2, 80, 0),
         ([50, 3], [2000, 40], 4, 1, 128, 0), ([300], [500], 2, 2, 64, 0), ([40], [300], 2, 1, 256, 0)]


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "f16"), ("f16", "e4m3")])
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (False, 90)])
@pytest.mark.parametrize("size", [1.5, 40.0])
def test_what_sees_a_value_that_is_not_finite(case, dtype, cache, causal, window, size):
    new, ctx, hq, hk, dim, wide = case
    rng = np.random.default_rng(81)
    b = Batch(rng, new, ctx, hk, dim, 16, dtype, cache, wide=wide)
    b.table[0, 1] = -1                              # a page that is not there
    b.gpu()
    bad = torch.zeros(b.vt.shape, dtype=torch.bool)
    v = b.vt.float().cpu()
    for s, kv in enumerate(b.kv):
        kinds = [np.nan] if cache == "e4m3" else [np.inf, -np.inf, np.nan]
        for j in np.concatenate([[0, kv - 1], rng.integers(0, kv, 6)]):
            page = b.table[s, j // 16]
            if page < 0:
                continue
            for g in range(hk):
                d = rng.integers(0, dim)
                v[page, g, j % 16, d] = rng.choice(kinds)
                bad[page, g, j % 16, d] = True
    b.vt.copy_(v)
    q = values(rng, (b.n, hq, dim), dtype, size)
    got = dws.bevpool_paged_attention(q[0], b.pool, b.batch, causal=causal, window=window)
    torch.cuda.synchronize()
    got = host(got)
    v64 = np.where(np.isnan(b.v0), np.nan, host(b.vt) * b.v_scale)
    v64 = np.where(b.live & ~bad.numpy(), v64, 0.0)
    want, mag, spread, seen = ref.attention(q[1], b.k0, v64, b.offsets, b.kv, b.table, dim ** -0.5,
                                            causal, window)
    # which outputs see one: a softmax of equal weights over the marks
    mark, _, _, _ = ref.attention(0 * q[1], 0 * np.nan_to_num(b.k0), bad.numpy().astype(np.float64),
                                  b.offsets, b.kv, b.table, 1.0, causal, window)
    sees = mark > 0
    assert (sees.any(-1) | (seen == 0)).any() and not sees.all()
    assert np.array_equal(~np.isfinite(got), sees)
    u = U["f16" if cache == "e4m3" else dtype]
    d = 2 * (dim + 8) * E32 * spread + 2.0 ** -21
    rel = (u + 2 * d + 2 * seen * E32 + 2.0 ** -20)[..., None]
    err = mag * rel * (1 + U[dtype]) + U[dtype] * np.abs(want) + TINY[dtype]
    if u == U["f16"]:
        err = err + (seen * 2.0 ** -25)[..., None] * np.abs(v64).max()
    within(got[~sees], want[~sees], err[~sees])
