"""Norm and rotation inside torch's graph of gradients, and the refusals of
the calls that have no gradient."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from oracle import tokens as ref
from token_util import E32, TINY, U, Batch, dev, host, make_rope, turned_bound, values, within

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _case(seed, n=37, hq=4, hk=2, dim=64, sections=(8, 12, 12), dtype="bf16", wdtype=None):
    rng = np.random.default_rng(seed)
    pos_t, pos, f_t, f = make_rope(rng, sections, n)
    rope = dws.Rope(f_t, sections)
    qkv = values(rng, (n, hq + 2 * hk, dim), dtype)[0]
    w = [(values(rng, (dim,), wdtype or dtype, 0.3)[0] + 1) for _ in range(2)]
    dy = [values(rng, (n, h, dim), dtype)[0] for h in (hq, hk)]
    return rope, pos_t, pos, f, qkv, w, dy


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_backward_through_a_packed_projection(dtype, wdtype):
    """Queries and keys are slices of one leaf, as after a projection: its
    gradient against the formula's in float64, bits against the plain call."""
    rope, pos_t, pos, f, qkv, w, dy = _case(101, dtype=dtype, wdtype=wdtype)
    leaf = qkv.clone().requires_grad_()
    ws = [x.clone().requires_grad_() for x in w]
    y = dws.bevpool_qk_norm_rope(leaf[:, :4], leaf[:, 4:6], pos_t, rope, *ws, EPS)
    plain = dws.bevpool_qk_norm_rope(qkv[:, :4], qkv[:, 4:6], pos_t, rope, *w, EPS)
    assert all(torch.equal(a, b) and a.requires_grad and not b.requires_grad
               for a, b in zip(y, plain))
    torch.autograd.backward(y, dy)
    g = dws.bevpool_qk_norm_rope_backward(*dy, qkv[:, :4], qkv[:, 4:6], pos_t, rope, *w, EPS)
    assert torch.equal(leaf.grad[:, :4], g[0]) and torch.equal(leaf.grad[:, 4:6], g[1])
    assert (leaf.grad[:, 6:] == 0).all()
    for got, want, x in zip((ws[0].grad, ws[1].grad), g[2:], w):
        assert got.dtype == x.dtype and torch.equal(got, want.to(x.dtype))
    for lo, hi, i in ((0, 4, 0), (4, 6, 1)):
        x, d, w64 = host(qkv[:, lo:hi]), host(dy[i]), host(w[i])
        dx, dw = ref.norm_turn_backward(d, x, w64, EPS, pos, f, (8, 12, 12), False)
        size = np.abs(d)
        part = turned_bound(size, 32, False, 64, "f32", 0 * size) / ((64 / 2 + 16) * E32)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        xh, aw = np.abs(x * r), np.abs(w64)
        big = r * (aw * part + xh * (xh * aw * part).mean(-1, keepdims=True))
        within(host(leaf.grad[:, lo:hi]), dx, big * (2 * 64 + 64) * E32 * (1 + U[dtype]) +
               U[dtype] * np.abs(dx) + TINY[dtype], "dx")
        err = (part * xh).sum((0, 1)) * (d.shape[0] * d.shape[1] + 128) * E32
        within(host(ws[i].grad), dw, err * (1 + U[wdtype]) + U[wdtype] * np.abs(dw) + TINY[wdtype])


@pytest.mark.parametrize("which", range(4))
def test_each_leaf_alone(which):
    """One of q, k and the weights wants a gradient: it gets the same bits, the
    others none."""
    rope, pos_t, _, _, qkv, w, dy = _case(102)
    given = [qkv[:, :4].clone(), qkv[:, 4:6].clone(), w[0], w[1]]
    want = dws.bevpool_qk_norm_rope_backward(*dy, given[0], given[1], pos_t, rope, *w, EPS)
    leaves = [t.clone().requires_grad_(i == which) for i, t in enumerate(given)]
    y = dws.bevpool_qk_norm_rope(leaves[0], leaves[1], pos_t, rope, leaves[2], leaves[3], EPS)
    torch.autograd.backward(y, dy)
    assert torch.equal(leaves[which].grad, want[which].to(leaves[which].dtype))
    assert all(t.grad is None for i, t in enumerate(leaves) if i != which)


@pytest.mark.parametrize("used", ["q", "k"])
def test_one_output_used(used):
    """A loss of one output alone; and the gradient of a sum, which is one
    number expanded over the output."""
    rope, pos_t, _, _, qkv, w, _ = _case(103)
    q, k = (qkv[:, a:b].clone().requires_grad_() for a, b in ((0, 4), (4, 6)))
    ws = [x.clone().requires_grad_() for x in w]
    y = dws.bevpool_qk_norm_rope(q, k, pos_t, rope, *ws, EPS)
    one = [torch.ones_like(t) if name == used else torch.zeros_like(t) for name, t in zip("qk", y)]
    y["qk".index(used)].sum().backward()
    want = dws.bevpool_qk_norm_rope_backward(*one, q.detach(), k.detach(), pos_t, rope, *w, EPS)
    for name, t, weight, g, gw in (("q", q, ws[0], want[0], want[2]), ("k", k, ws[1], want[1], want[3])):
        if name == used:
            assert torch.equal(t.grad, g) and torch.equal(weight.grad, gw.to(weight.dtype))
        else:
            assert t.grad is None or (t.grad == 0).all()
            assert weight.grad is None or (weight.grad == 0).all()


def test_shared_leaves_and_odd_gradients():
    """The same leaf as queries and keys, one weight for both, and gradients
    that are transposed and sliced tensors."""
    rope, pos_t, _, _, qkv, w, _ = _case(104, dtype="f32")
    n = qkv.shape[0]
    x, weight = qkv[:, :4].clone().requires_grad_(), w[0].clone().requires_grad_()
    dq = torch.randn(4, n, 64, device=dev()).transpose(0, 1)
    dk = torch.randn(n, 4, 65, device=dev())[..., 1:]
    y = dws.bevpool_qk_norm_rope(x, x, pos_t, rope, weight, weight, EPS)
    torch.autograd.backward(y, [dq, dk])
    g = dws.bevpool_qk_norm_rope_backward(dq.contiguous(), dk.contiguous(), x.detach(), x.detach(),
                                          pos_t, rope, w[0], w[0], EPS)
    assert torch.equal(x.grad, g[0] + g[1]) and torch.equal(weight.grad, g[2] + g[3])


def test_gradient_against_differences():
    """Through the graph, in fp32: a step of 2^-6 leaves h^2 f''' / 6, below 2e-4
    here (third derivatives under 5), and rounding of 1e-6 * |loss terms| / h."""
    rope, pos_t, _, _, qkv, w, dy = _case(105, n=2, hq=2, hk=1, dim=32, sections=(8, 8), dtype="f32")
    x, weight = (2 * qkv[:, :2]).clone().requires_grad_(), w[0].clone().requires_grad_()

    def loss(x, weight):
        return (dws.bevpool_qk_norm_rope(x, None, pos_t, rope, weight, None, EPS)[0].double() *
                dy[0]).sum()

    loss(x, weight).backward()
    h = 2.0 ** -6
    for t in (x, weight):
        for i in range(0, t.numel(), 7):
            ends = []
            for step in (h, -h):
                moved = t.detach().clone()
                moved.view(-1)[i] += step
                with torch.no_grad():
                    ends.append(float(loss(moved, weight) if t is x else loss(x, moved)))
            assert abs((ends[0] - ends[1]) / (2 * h) - float(t.grad.view(-1)[i])) < 3e-4, i


def test_without_weights_and_without_rotation():
    """No weight: the inputs are not kept, and may change before the backward
    pass.  No rotation and no weight: the gradient itself."""
    rope, pos_t, _, _, qkv, _, dy = _case(106)
    leaf = qkv[:, :4].clone().requires_grad_()
    x = leaf * 1
    y, _ = dws.bevpool_qk_norm_rope(x, None, pos_t, rope)
    x.detach().zero_()
    y.backward(dy[0])
    want = dws.bevpool_qk_norm_rope_backward(dy[0], None, None, None, pos_t, rope)[0]
    assert torch.equal(leaf.grad, want)
    leaf.grad = None
    dws.bevpool_qk_norm_rope(leaf, None, None, None)[0].backward(dy[0])
    assert torch.equal(leaf.grad, dy[0])


def test_inputs_that_change_before_the_backward_pass():
    rope, pos_t, _, _, qkv, w, dy = _case(107)
    leaf = qkv[:, :4].clone().requires_grad_()
    x, pos = leaf * 1, pos_t.clone()
    y, _ = dws.bevpool_qk_norm_rope(x, None, pos, rope, w[0], None, EPS)
    x.detach().add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(dy[0])
    y, _ = dws.bevpool_qk_norm_rope(leaf, None, pos, rope, w[0], None, EPS)
    pos.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(dy[0])


def test_on_another_stream():
    rope, pos_t, _, _, qkv, w, dy = _case(108, n=3000)
    leaf = qkv.clone().requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = dws.bevpool_qk_norm_rope(leaf[:, :4], leaf[:, 4:6], pos_t, rope, *w, EPS, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.autograd.backward(y, dy)
    torch.cuda.synchronize()
    g = dws.bevpool_qk_norm_rope_backward(*dy, qkv[:, :4], qkv[:, 4:6], pos_t, rope, *w, EPS)
    assert torch.equal(leaf.grad[:, :4], g[0]) and torch.equal(leaf.grad[:, 4:6], g[1])


def test_no_tokens():
    e = torch.empty((0, 2, 32), dtype=torch.bfloat16, device=dev(), requires_grad=True)
    w = torch.ones(32, dtype=torch.bfloat16, device=dev(), requires_grad=True)
    y, _ = dws.bevpool_qk_norm_rope(e, None, None, None, w)
    y.sum().backward()
    assert e.grad.shape == e.shape and (w.grad == 0).all()


def test_refusals(monkeypatch):
    rope, pos_t, _, _, qkv, w, dy = _case(109)
    q, k = qkv[:, :4].clone(), qkv[:, 4:6].clone()
    leaf, weight = q.clone().requires_grad_(), w[0].clone().requires_grad_()
    turn = dws.bevpool_qk_norm_rope
    for kw in (dict(q_out=torch.empty_like(q)), dict(k_out=torch.empty_like(k))):
        with pytest.raises(RuntimeError, match="not differentiable"):
            turn(leaf, k, pos_t, rope, **kw)
        with pytest.raises(RuntimeError, match="not differentiable"):
            turn(q, k, pos_t, rope, weight, **kw)
    with pytest.raises(RuntimeError, match="not differentiable"):
        turn(q, None, pos_t, rope, q_out=leaf)
    y, _ = turn(leaf, None, pos_t, rope, w[0])
    with pytest.raises(RuntimeError):                          # no second derivative
        g, = torch.autograd.grad(y, leaf, dy[0].clone().requires_grad_(), create_graph=True)
        g.sum().backward()
    back = dws.bevpool_qk_norm_rope_backward
    with pytest.raises(RuntimeError, match="second derivative"):
        back(dy[0].clone().requires_grad_(), None, q, None, pos_t, rope, w[0])
    assert back(dy[0], None, leaf, None, pos_t, rope, weight)[0].requires_grad is False

    b = Batch(np.random.default_rng(110), [30, 7], [9, 3], 2, 64, 16, "bf16", "bf16")
    append, attend = dws.bevpool_kv_append, dws.bevpool_paged_attention
    pos = pos_t
    with pytest.raises(RuntimeError, match="no gradient"):
        append(k.clone().requires_grad_(), k, b.pool, b.batch, pos, rope)
    with pytest.raises(RuntimeError, match="no gradient"):
        append(k, k.clone().requires_grad_(), b.pool, b.batch, pos, rope)
    with pytest.raises(RuntimeError, match="no gradient"):
        append(k, k, b.pool, b.batch, pos, rope, q=leaf)
    with pytest.raises(RuntimeError, match="no gradient"):
        append(k, k, b.pool, b.batch, pos, rope, k_weight=weight)
    with pytest.raises(RuntimeError, match="no gradient"):
        attend(leaf, b.pool, b.batch)
    with pytest.raises(RuntimeError, match="no gradient"):
        attend(q, dws.PagedCache(b.kt.clone().requires_grad_(), b.vt), b.batch)
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            qt = append(k, k, b.pool, b.batch, pos, rope, q=leaf, q_weight=weight)
            assert torch.isfinite(attend(qt, b.pool, b.batch)).all()
            assert torch.equal(turn(leaf, k, pos_t, rope, weight, q_out=torch.empty_like(q))[0],
                               turn(q, k, pos_t, rope, w[0])[0])
    # a captured call of its own is the plain one
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="not captured"):
        turn(leaf, k, pos_t, rope)
    turn(q, k, pos_t, rope)
