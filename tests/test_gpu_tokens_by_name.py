"""Every token call with all of its arguments by name gives what it gives
with positional ones, on the current stream and on another."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from token_util import Batch, make_rope, packed, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("other", [False, True])
def test_arguments_by_name(other):
    rng = np.random.default_rng(91)
    b = Batch(rng, [3, 40], [9, 30], 2, 64, 16, "bf16", "bf16")
    pos, _, f, _ = make_rope(rng, (32,), b.n)
    rope = dws.Rope(inv_freq=f, sections=(32,), layout=dws.ROPE_HALVES)
    (q, _), (k, _), (v, _) = packed(rng, b.n, [4, 2, 2], 64, "bf16")
    wq, wk = (values(rng, (64,), "bf16")[0] for _ in range(2))
    on = {}
    if other:
        on["stream"] = torch.cuda.Stream()
        on["stream"].wait_stream(torch.cuda.current_stream())
    turned = dws.bevpool_qk_norm_rope(q, k, pos, rope, wq, wk, 1e-5)
    named = dws.bevpool_qk_norm_rope(eps=1e-5, k_weight=wk, q_weight=wq, rope=rope, positions=pos,
                                     k=k, q=q, **on)
    grads = dws.bevpool_qk_norm_rope_backward(q, k, q, k, pos, rope, wq, wk, 1e-5)
    named_grads = dws.bevpool_qk_norm_rope_backward(dq_out=q, dk_out=k, q=q, k=k, positions=pos,
                                                    rope=rope, q_weight=wq, k_weight=wk, eps=1e-5,
                                                    **on)
    qt = dws.bevpool_kv_append(k, v, b.pool, b.batch, pos, rope, q=q, q_weight=wq, k_weight=wk)
    torch.cuda.synchronize()
    kept = b.kt.clone(), b.vt.clone()
    named_qt = dws.bevpool_kv_append(v=v, k=k, batch=b.batch, cache=b.pool, rope=rope, positions=pos,
                                     q=q, q_weight=wq, k_weight=wk, eps=1e-6, **on)
    torch.cuda.synchronize()
    out = dws.bevpool_paged_attention(qt, b.pool, b.batch, 0.125, True, 20)
    named_out = dws.bevpool_paged_attention(cache=b.pool, batch=b.batch, q=qt, window=20, causal=True,
                                            scale=0.125, **on)
    torch.cuda.synchronize()
    for got, want in ((named, turned), (named_grads, grads), ([named_qt], [qt]), ([named_out], [out])):
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    for t, old in zip((b.kt, b.vt), kept):
        assert torch.equal(t.view(torch.int16), old.view(torch.int16))
