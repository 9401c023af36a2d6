"""Sequences that pass their table and offsets that pass the tokens, append
and attention against the float64 oracle (bounds derived in token_util)."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from oracle import tokens as ref
from token_util import E32, TINY, U, Batch, dev, host, packed, values, within

pytestmark = pytest.mark.gpu

# new tokens, lengths and offsets past the ends: places 0 to 79 of five pages of 16
CASES = [
    ([1], [81], None),                          # one token, one place past the table
    ([1, 1, 1], [80, 81, 82], None),
    ([5, 20, 1], [82, 85, 2 ** 31 - 1], None),
    ([70, 40], [100, 79], None),
    ([6, 5], [40, 30], [-3, 6, 14]),            # three before the first token, three past the last
    ([6, 5], [90, 81], [-(2 ** 31), 6, 2 ** 31 - 1]),
    ([300], [130], [-5, 309]),
]


def _batch(rng, new, lengths, offsets, hk, dim, dtype, cache):
    b = Batch(rng, new, [max(80 - n, 0) for n in new], hk, dim, 16, dtype, cache)
    b.table = b.table[:, :5].copy()             # the first has more where it has more new tokens
    b.kv = np.array(lengths)
    if offsets is not None:
        b.offsets = np.array(offsets)
    b.offsets = b.offsets.astype(np.int32)
    b.gpu()
    return b


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "e4m3")])
@pytest.mark.parametrize("new,lengths,offsets", CASES)
def test_append_places(new, lengths, offsets, dtype, cache):
    rng = np.random.default_rng(61)
    b = _batch(rng, new, lengths, offsets, 2, 64, dtype, cache)
    k, v = packed(rng, b.n, [2, 2], 64, dtype)
    before = b.kt.clone(), b.vt.clone()
    dws.bevpool_kv_append(k[0], v[0], b.pool, b.batch, None, None)
    torch.cuda.synchronize()
    kc, vc, hit = ref.append(k[1], v[1], b.k0, b.v0, b.offsets, b.kv, b.table)
    on = np.broadcast_to(hit[:, None, :, None], kc.shape)
    for t, old, want, scale in ((b.kt, before[0], kc, b.k_scale), (b.vt, before[1], vc, b.v_scale)):
        same = (t.view(torch.uint8) == old.view(torch.uint8)).cpu().numpy()
        assert same.reshape(*kc.shape, -1)[~on].all()
        z = want[on] / scale
        within(host(t)[on], z, np.abs(z) * (U[cache] + 2 * E32) + TINY[cache])


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f16", "e4m3")])
@pytest.mark.parametrize("new,lengths,offsets", CASES)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (False, 0), (False, 20),
                                           (True, 2 ** 31 - 1)])
def test_attention_places(new, lengths, offsets, dtype, cache, causal, window):
    rng = np.random.default_rng(62)
    b = _batch(rng, new, lengths, offsets, 2, 64, dtype, cache)
    # every slot of the table holds a key
    for name in ("kt", "vt"):
        t = getattr(b, name)
        setattr(b, name, torch.where(torch.isnan(t.float()), 1.0, t.float()).to(t.dtype))
    b.gpu()
    k64, v64 = host(b.kt) * b.k_scale, host(b.vt) * b.v_scale
    q = values(rng, (b.n, 4, 64), dtype, 1.5)
    out = torch.full_like(q[0], 7.0)
    got = dws.bevpool_paged_attention(q[0], b.pool, b.batch, causal=causal, window=window, out=out)
    torch.cuda.synchronize()
    want, mag, spread, seen = ref.attention(q[1], k64, v64, b.offsets, b.kv, b.table, 0.125, causal,
                                            window)
    u = U["f16" if cache == "e4m3" else dtype]
    d = 2 * (64 + 8) * E32 * spread + 2.0 ** -21
    rel = (u + 2 * d + 2 * seen * E32 + 2.0 ** -20)[..., None]
    err = mag * rel * (1 + U[dtype]) + U[dtype] * np.abs(want) + TINY[dtype]
    if u == U["f16"]:
        err = err + (seen * 2.0 ** -25)[..., None] * np.abs(v64).max()
    assert not np.isnan(want).any()             # every token has a sequence
    within(host(got), want, err)
