"""Attention where the size of the scores decides: very large ones, whose
softmax is one key, and many small weights beside a large one."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from token_util import DT, Batch, dev, host

pytestmark = pytest.mark.gpu


def _ranks(rng, n, cache):
    """n distinct positive values that the type holds, in any order; e4m3 has
    120 of them, and zeros behind the first key."""
    if cache == "e4m3":
        v = torch.arange(1, 121, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        a = np.zeros(n)
        at = np.concatenate([[0], 1 + rng.permutation(n - 1)[:119]])
        a[at[:len(v)]] = rng.permutation(v)[:len(at)]
        return a
    r = rng.permutation(n)
    if cache == "f16":
        return 32.0 * (r + 1)                       # up to 65504
    return (128.0 + r % 128) * 2.0 ** (20 + r // 128)


# new, ctx, hq, hk, table entries past the sequence
ONE_KEY = [([1], [700], 4, 2, 0), ([1, 1], [1900, 30], 8, 1, 600), ([100], [400], 2, 2, 0),
           ([40, 3], [1900, 500], 4, 2, 0), ([300], [1500], 3, 1, 0), ([90], [1900], 64, 2, 0)]


@pytest.mark.parametrize("dtype,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"),
                                         ("bf16", "e4m3")])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("case", ONE_KEY, ids=str)
def test_attention_of_one_key(case, dim, dtype, cache):
    """Scores of up to 2^40 (fp16) and more that differ by far more than the
    exponential holds: the output is the best key's value, exactly."""
    new, ctx, hq, hk, wide = case
    rng = np.random.default_rng(71)
    b = Batch(rng, new, ctx, hk, dim, 32, dtype, cache, wide=wide)
    q = rng.uniform(4.0, 15.9, b.n * hq)            # 2^4 to 2^16
    q = np.exp2(q) * (1e9 if dtype == "bf16" else 1.0)
    if cache != "e4m3":
        q *= rng.choice([-1.0, 1.0], q.shape)
    qt = torch.from_numpy(q.reshape(b.n, hq, 1)).to(DT[dtype])
    q = qt.double().numpy()[..., 0]
    qt = qt.expand(b.n, hq, dim).contiguous().to(dev())
    v = host(b.vt)
    want = np.zeros((b.n, hq, dim))
    kt = b.kt.cpu()
    for s, kv in enumerate(b.kv):
        j = np.arange(kv)
        pages, slots = b.table[s, j // 32], j % 32
        for g in range(hk):
            a = _ranks(rng, kv, cache)
            kt[pages, g, slots] = torch.from_numpy(a)[:, None].expand(kv, dim).to(kt.dtype)
            for t in range(b.offsets[s], b.offsets[s + 1]):
                see = kv - b.offsets[s + 1] + t + 1
                for h in range(g * hq // hk, (g + 1) * hq // hk):
                    best = np.argmax(a[:see] * q[t, h])
                    want[t, h] = v[pages[best], g, slots[best]]
    b.kt.copy_(kt)
    got = dws.bevpool_paged_attention(qt, b.pool, b.batch)
    want = torch.from_numpy(want * (b.v_scale if cache == "e4m3" else 1.0))
    if cache == "e4m3":                             # code * scale, in fp32, then rounded
        want = want.float()
        off = (got.cpu().double() - want.double()).abs()
        assert (off <= want.abs().double() * (torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -22)).all()
    else:
        assert torch.equal(got.cpu(), want.to(DT[dtype]))


@pytest.mark.parametrize("dim,cache", [(64, "f16"), (128, "e4m3")])
@pytest.mark.parametrize("n,hq,hk", [(8192, 8, 8), (2, 16, 8)])
def test_attention_many_small_weights(n, hq, hk, dim, cache):
    """One key of weight 1 and value 0, and 2^16 of weight 2^-27 and value 1,
    which fp16 alone would round to 0.  Weights reach the product with v as
    fp16 numbers 2^7 times as large, so one under 2^-21 is off by up to 2^-32
    and the sum by 2^16 * 2^-32; the rest are a few roundings of it."""
    keys, page = 65536, 64
    rng = np.random.default_rng(72)
    k_scale, v_scale = (0.5, 0.25) if cache == "e4m3" else (1.0, 1.0)
    kt = torch.zeros((keys // page, hk, page, dim), device=dev())
    vt = torch.full_like(kt, 1.0 / v_scale)
    kt[0, :, 0, 0] = 16.0 / k_scale
    vt[0, :, 0] = 0.0
    pool = dws.PagedCache(kt.to(DT[cache]), vt.to(DT[cache]), k_scale, v_scale)
    del kt, vt
    batch = dws.PagedBatch(torch.tensor([0, n], dtype=torch.int32, device=dev()),
                           torch.tensor([keys], dtype=torch.int32, device=dev()),
                           torch.arange(keys // page, dtype=torch.int32, device=dev())[None])
    q = torch.zeros((n, hq, dim), dtype=torch.float16, device=dev())
    q[..., 0] = 1.0
    got = dws.bevpool_paged_attention(q, pool, batch, 27 * np.log(2.0) / 16, causal=False)
    tail = (keys - 1) * 2.0 ** -27
    want = tail / (1 + tail)
    # the scale is an fp32 number and so is its product with log2 e: 27 of them are within 2^-18
    slack = keys * 2.0 ** -32 + want * (2.0 ** -11 + 2.0 ** -18 + 2.0 ** -16)
    off = (got.double() - want).abs().max().item()
    assert off <= slack, (off, slack, want)
