"""Keys of no heads: nothing is turned, and the gradient of their weight is a sum of
nothing."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from token_util import make_rope, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [0, 1, 70])
def test_keys_of_no_heads(n):
    rng = np.random.default_rng(151)
    pos, _, f, _ = make_rope(rng, (16,), n)
    rope = dws.Rope(f, (16,))
    q, _ = values(rng, (n, 3, 32), "bf16")
    w = [values(rng, (32,), "bf16")[0] for _ in range(2)]
    k = q[:, :0]
    y = dws.bevpool_qk_norm_rope(q, k, pos, rope, *w)
    assert torch.equal(y[0], dws.bevpool_qk_norm_rope(q, None, pos, rope, w[0])[0])
    assert y[1].shape == (n, 0, 32)
    want = dws.bevpool_qk_norm_rope_backward(q, None, q, None, pos, rope, w[0])
    for _ in range(3):
        junk = torch.full((32,), 7.0, device=q.device)          # what a new tensor may hold
        del junk
        g = dws.bevpool_qk_norm_rope_backward(q, k, q, k, pos, rope, *w)
        assert torch.equal(g[0], want[0]) and torch.equal(g[2], want[2])
        assert g[1].shape == (n, 0, 32) and torch.equal(g[3], torch.zeros_like(g[3]))
    leaf, kw = q.clone().requires_grad_(), w[1].clone().requires_grad_()
    a, b = dws.bevpool_qk_norm_rope(leaf, leaf[:, :0], pos, rope, w[0], kw)
    (a.float().sum() + b.float().sum()).backward()
    assert (kw.grad == 0).all() and leaf.grad.shape == q.shape
