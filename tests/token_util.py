"""Helpers of the token operators' GPU tests: inputs, batches over a paged
cache, and error bounds.  Bounds are derived here, before any kernel ran:

u(t) is half a step of the output type (bf16 2^-8, fp16 2^-11, fp32 2^-24,
e4m3 2^-4) and e = 2^-24 that of fp32.

Norm and rotation.  The mean square of dim positive terms is within dim * e of
itself, its root's reciprocal within (dim / 2 + 6) e; two products follow.  An
angle is right to 2^-22 (half a turn's fraction rounded to fp32, pi * 2^-25,
and a few units of the sine), so a rotated coordinate is within
(|a| + |b|) * (dim / 2 + 16) e of its value; the store adds u |y|.

Attention.  A score is a sum of dim products, within (dim + 4) e * spread of
its value (spread = sum |q k| scale; the product with scale * log2 e and the
difference to the maximum, at most 4 spread, add the 4), so a weight is within
w * d with d = 2 (dim + 8) e spread + 2^-21 (the exponential and the rescales).
Weights are rounded to the token type before they meet v (u w), but not in the
softmax's sum; a sum of n terms adds n e.  So the output is within
mag * (u + 2 d + 2 n e + 2^-20) with mag = sum w |v|, and the store adds
u |out|.  fp16 weights under 2^-14 are rounded to 2^-25 of the largest: n 2^-25
max |v| more.
"""
from __future__ import annotations

import numpy as np
import torch

import depth_weighted_scatter_amd as dws

E32 = 2.0 ** -24
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}
# half the smallest subnormal step
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
      "e4m3": torch.float8_e4m3fn}


def dev():
    return torch.device("cuda:0")


def values(rng, shape, dtype, scale=1.0):
    """Random values of dtype on the GPU, and the same in float64 on the host."""
    t = torch.from_numpy(rng.standard_normal(shape) * scale).to(DT[dtype])
    return t.to(dev()), t.double().numpy()


def host(t):
    return t.detach().double().cpu().numpy()


def make_rope(rng, sections, n, far=1000):
    half = sum(sections)
    f = (10000.0 ** (-np.arange(half) / max(half, 1))).astype(np.float32)
    pos = rng.integers(-far, far + 1, (len(sections), n)).astype(np.int32)
    return (torch.from_numpy(pos).to(dev()), pos,
            torch.from_numpy(f).to(dev()) if half else None, f)


def packed(rng, n, heads, dim, dtype, stride_extra=0):
    """Token tensors that are slices of one buffer, with their host values."""
    total = sum(heads) * dim + stride_extra
    buf, h = values(rng, (n, total), dtype)
    got, at = [], 0
    for k in heads:
        got.append((buf[:, at:at + k * dim].view(n, k, dim),
                    h[:, at:at + k * dim].reshape(n, k, dim)))
        at += k * dim
    return got


def turned_bound(n64, half, adjacent, dim, dtype, y):
    """Bound on a rotated coordinate's error, from the normed row n64."""
    part = np.abs(n64).copy()
    if half:
        if adjacent:
            s = part[..., 0:2 * half:2] + part[..., 1:2 * half:2]
            part[..., 0:2 * half:2] = part[..., 1:2 * half:2] = s
        else:
            s = part[..., :half] + part[..., half:2 * half]
            part[..., :half] = part[..., half:2 * half] = s
    # the store rounds the computed value, itself within the first term of y
    err = part * (dim / 2 + 16) * E32
    return err * (1 + U[dtype]) + U[dtype] * np.abs(y) + TINY[dtype]


def within(got, want, bound, label=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (label, got.shape, want.shape)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= bound)
    bad &= ~(np.isnan(got) & np.isnan(want)) & ~((got == want) & np.isinf(got))
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{label}: {bad.sum()} of {bad.size} off, first at {at}: got "
                             f"{got[at]}, want {want[at]} +- {np.broadcast_to(bound, got.shape)[at]}")


class Batch:
    """Sequences with `new` new tokens and `ctx` cached ones each, their pages
    scattered over a pool whose every unused slot holds NaN."""

    def __init__(self, rng, new, ctx, hk, dim, page, dtype, cache, lead=0, tail=0, spare=3,
                 k_scale=0.03, v_scale=0.02, wide=0, fill=True):
        new, ctx = np.array(new), np.array(ctx)
        self.new, self.kv = new, new + ctx
        self.page, self.hk, self.dim, self.dtype, self.cache = page, hk, dim, dtype, cache
        self.n = lead + int(new.sum()) + tail
        self.offsets = (lead + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        need = np.maximum(-(-self.kv // page), 0)
        self.n_pages = int(need.sum()) + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(new), int(need.max(initial=0)) + wide), -1, np.int32)
        at = 0
        for s, c in enumerate(need):
            self.table[s, :c] = order[at:at + c]
            at += c
        shape = (self.n_pages, hk, page, dim)
        self.k_scale, self.v_scale = (k_scale, v_scale) if cache == "e4m3" else (1.0, 1.0)
        live = np.zeros((self.n_pages, page), bool)
        if fill:
            for s, v in enumerate(self.kv):
                j = np.arange(max(int(v), 0))
                live[self.table[s, j // page], j % page] = True
        self.live = live[:, None, :, None]
        parts = []
        for scale in (self.k_scale, self.v_scale):
            x = torch.from_numpy(rng.standard_normal(shape) / scale).clamp_(-448, 448)
            x = torch.where(torch.from_numpy(np.broadcast_to(self.live, shape).copy()), x, torch.nan)
            parts.append(x.to(DT[cache]))
        self.k0, self.v0 = (np.where(self.live, host(x) * scale, np.nan)
                            for x, scale in zip(parts, (self.k_scale, self.v_scale)))
        self.kt, self.vt = (x.to(dev()) for x in parts)
        self.gpu()

    def gpu(self):
        t = [torch.from_numpy(np.ascontiguousarray(a)).to(dev())
             for a in (self.offsets, self.kv.astype(np.int32), self.table)]
        self.batch = dws.PagedBatch(*t)
        self.pool = dws.PagedCache(self.kt, self.vt, self.k_scale, self.v_scale)
