"""Batches of thousands of sequences, most of them short or without a new
token: the search for a token's or a tile's owner takes several steps."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from oracle import tokens as ref
from token_util import E32, TINY, U, Batch, host, packed, values, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs", [65, 4095, 4097, 5000])
@pytest.mark.parametrize("most", [1, 3])
def test_many_sequences(seqs, most):
    rng = np.random.default_rng(141)
    new = rng.integers(0, most + 1, seqs)
    b = Batch(rng, new, rng.integers(0, 20, seqs), 1, 16, 16, "bf16", "bf16", lead=3, tail=2)
    k, v = packed(rng, b.n, [1, 1], 16, "bf16")
    dws.bevpool_kv_append(k[0], v[0], b.pool, b.batch, None, None)
    torch.cuda.synchronize()
    kc, vc, hit = ref.append(k[1], v[1], b.k0, b.v0, b.offsets, b.kv, b.table)
    assert hit.sum() == new.sum()
    on = np.broadcast_to(hit[:, None, :, None], kc.shape)
    for t, want in ((b.kt, kc), (b.vt, vc)):
        assert np.array_equal(host(t)[on], want[on])           # bf16 to bf16
        assert np.array_equal(host(t)[~on], want[~on], equal_nan=True)
    q = values(rng, (b.n, 2, 16), "bf16", 1.5)
    out = torch.full_like(q[0], 7.0)
    got = dws.bevpool_paged_attention(q[0], b.pool, b.batch, out=out)
    want, mag, spread, seen = ref.attention(q[1], host(b.kt), host(b.vt), b.offsets, b.kv, b.table,
                                            0.25, True, 0)
    inside = slice(3, b.n - 2)
    assert (got[:3] == 7).all() and (got[inside.stop:] == 7).all()
    rel = (U["bf16"] + 4 * (16 + 8) * E32 * spread + 2.0 ** -19 + 2 * seen * E32)[..., None]
    err = mag * rel * (1 + U["bf16"]) + U["bf16"] * np.abs(want) + TINY["bf16"]
    within(host(got)[inside], want[inside], err[inside])
