"""CPU oracle of the token operators -- TEST INFRASTRUCTURE ONLY.

Plain numpy in float64, straight from the definitions: RMS norm and rotation
by positions of several axes, their gradient, the append to a paged cache and
attention over it.  Shares nothing with the product library.  Pinned by
tests/test_tokens_oracle.py.
"""
from __future__ import annotations

import numpy as np


def turn(x, positions, inv_freq, sections, adjacent, sign=1.0):
    """Rotate each pair of x [n, heads, dim] by sign * position * inv_freq."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    half = sum(sections)
    pair = 0
    for axis, count in enumerate(sections):
        for _ in range(count):
            a, b = (2 * pair, 2 * pair + 1) if adjacent else (pair, pair + half)
            th = sign * positions[axis].astype(np.float64) * np.float64(inv_freq[pair])
            c, s = np.cos(th)[:, None], np.sin(th)[:, None]
            y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
            y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
            pair += 1
    return y


def norm(x, w, eps):
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return np.asarray(w, np.float64) * x * r


def norm_turn(x, w, eps, positions, inv_freq, sections, adjacent):
    return turn(norm(x, w, eps), positions, inv_freq, sections, adjacent)


def norm_turn_backward(dy, x, w, eps, positions, inv_freq, sections, adjacent):
    """(dx, dw) with dw None where w is."""
    g = turn(dy, positions, inv_freq, sections, adjacent, -1.0)
    if w is None:
        return g, None
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1))
    dx = r * (w * g - x * r * r * (x * w * g).mean(-1, keepdims=True))
    return dx, dw


def places(offsets, lengths, max_pages, page, n_tokens):
    """(sequence, place) of every token, (-1, 0) outside all of them.  A place
    may be negative or past the table; offsets may name tokens that are not
    there."""
    seq, place = np.full(n_tokens, -1), np.zeros(n_tokens, np.int64)
    for s in range(len(lengths)):
        b, e = int(offsets[s]), int(offsets[s + 1])
        for t in range(max(b, 0), min(e, n_tokens)):
            seq[t], place[t] = s, int(lengths[s]) - (e - b) + t - b
    return seq, place


def append(k, v, k_cache, v_cache, offsets, lengths, table):
    """Values at their slots, in float64 copies of the caches; a second pair
    says which slots were written."""
    n_pages, heads, page, _ = k_cache.shape
    kc, vc = k_cache.astype(np.float64), v_cache.astype(np.float64)
    hit = np.zeros((n_pages, page), bool)
    seq, place = places(offsets, lengths, table.shape[1], page, k.shape[0])
    for t in range(k.shape[0]):
        p = int(place[t])
        if seq[t] < 0 or p < 0 or p >= table.shape[1] * page:
            continue
        at = int(table[seq[t], p // page])
        if at < 0 or at >= n_pages:
            continue
        kc[at, :, p % page], vc[at, :, p % page] = k[t], v[t]
        hit[at, p % page] = True
    return kc, vc, hit


def attention(q, k_cache, v_cache, offsets, lengths, table, scale, causal, window):
    """out [n, heads, dim] with NaN rows outside the sequences, and for the
    error bound: sum of weight * |v| (like out), the largest sum of |q k| *
    scale among the keys seen, and the number of keys seen ([n, heads])."""
    q = np.asarray(q, np.float64)
    n, hq, dim = q.shape
    n_pages, hk, page, _ = k_cache.shape
    out = np.full(q.shape, np.nan)
    mag, spread = np.zeros(q.shape), np.zeros((n, hq))
    seen_n = np.zeros((n, hq), np.int64)
    for s in range(len(lengths)):
        b, e = int(offsets[s]), int(offsets[s + 1])
        kv = min(max(int(lengths[s]), 0), table.shape[1] * page)
        j = np.arange(kv)
        pages = table[s, j // page].astype(np.int64) if kv else np.zeros(0, np.int64)
        there = (pages >= 0) & (pages < n_pages)
        j, pages = j[there], pages[there]
        k = k_cache[pages, :, j % page].astype(np.float64)        # [keys, hk, dim]
        v = v_cache[pages, :, j % page].astype(np.float64)
        for t in range(max(b, 0), min(e, n)):
            p = int(lengths[s]) - (e - b) + t - b
            see = np.ones(j.shape, bool)
            if causal:
                see &= j <= p
            if window > 0:
                see &= j > p - window
            for h in range(hq):
                if not see.any():
                    out[t, h] = 0.0
                    continue
                g = h // (hq // hk)
                ks, vs = k[see, g], v[see, g]
                x = ks @ q[t, h] * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                with np.errstate(invalid="ignore"):
                    out[t, h] = w @ vs
                    mag[t, h] = w @ np.abs(vs)
                spread[t, h] = (np.abs(ks) @ np.abs(q[t, h])).max() * scale
                seen_n[t, h] = see.sum()
    return out, mag, spread, seen_n
