"""Tensors that the token calls write in place: autograd is told."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from token_util import Batch, dev, make_rope, packed

pytestmark = pytest.mark.gpu


def _parts():
    rng = np.random.default_rng(121)
    b = Batch(rng, [3, 40], [9, 30], 2, 64, 16, "bf16", "bf16")
    pos, _, f, _ = make_rope(rng, (32,), b.n)
    q, k, v = (x[0].clone() for x in packed(rng, b.n, [4, 2, 2], 64, "bf16"))
    return b, pos, dws.Rope(f, (32,)), q, k, v


def _versions(call, *tensors):
    before = [t._version for t in tensors]
    call()
    return [t._version - v for t, v in zip(tensors, before)]


def test_versions():
    b, pos, rope, q, k, v = _parts()
    w = torch.ones(64, dtype=q.dtype, device=dev())
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    turn, back = dws.bevpool_qk_norm_rope, dws.bevpool_qk_norm_rope_backward
    assert _versions(lambda: turn(q, k, pos, rope, w, w), q, k, pos, w) == [0] * 4
    assert _versions(lambda: turn(q, k, pos, rope, q_out=qo), q, k, qo) == [0, 0, 1]
    assert _versions(lambda: turn(q, k, pos, rope, q_out=qo, k_out=k), q, k, qo) == [0, 1, 1]
    assert _versions(lambda: back(q, k, q, k, pos, rope, w, w), q, k, w) == [0] * 3
    assert _versions(lambda: back(q, k, q, k, pos, rope, dq=q, dk=ko), q, k, ko) == [1, 0, 1]
    cache = b.pool.k, b.pool.v
    append, attend = dws.bevpool_kv_append, dws.bevpool_paged_attention
    assert _versions(lambda: append(k, v, b.pool, b.batch, pos, rope), k, v, *cache) == [0, 0, 1, 1]
    assert _versions(lambda: append(k, v, b.pool, b.batch, pos, rope, q=q, q_out=qo), q, qo,
                     *cache) == [0, 1, 1, 1]
    assert _versions(lambda: attend(q, b.pool, b.batch), q, *cache) == [0] * 3
    assert _versions(lambda: attend(q, b.pool, b.batch, out=qo), q, qo, *cache) == [0, 1, 0, 0]
    # a slice counts for the tensor it is part of
    both = torch.cat([q, q], 1)
    assert _versions(lambda: turn(both[:, :4], None, pos, rope, q_out=both[:, :4]), both) == [1]
    with torch.inference_mode():
        attend(q, b.pool, b.batch, out=torch.empty_like(q))


def test_a_kept_tensor_that_is_overwritten():
    """torch keeps q for a product's gradient; the call then turns q in place."""
    _, pos, rope, q, _, _ = _parts()
    leaf = torch.ones_like(q, requires_grad=True)
    y = leaf * q
    dws.bevpool_qk_norm_rope(q, None, pos, rope, q_out=q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
