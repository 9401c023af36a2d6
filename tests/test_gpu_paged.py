"""The append to a paged cache and attention over it against the float64
oracle (bounds derived in token_util), and the token operators in a row."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from oracle import tokens as ref
from token_util import (DT, E32, TINY, U, Batch, dev, host, make_rope, packed, turned_bound, values,
                        within)

pytestmark = pytest.mark.gpu
EPS = 1e-6


# ---- append -------------------------------------------------------------------------------
def _codes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _check_append(b, got, before, k64, v64, n64, half, adjacent, label=""):
    kc, vc, hit = ref.append(k64, v64, b.k0, b.v0, b.offsets, b.kv, b.table)
    nb, _, _ = ref.append(np.abs(n64), np.abs(v64), 0 * b.k0, 0 * b.v0, b.offsets, b.kv, b.table)
    for name, t, old, want, n, scale in (("k", b.kt, before[0], kc, nb, b.k_scale),
                                         ("v", b.vt, before[1], vc, None, b.v_scale)):
        same = _codes(t).cpu().view(torch.uint8) == _codes(old).cpu().view(torch.uint8)
        rest = ~np.broadcast_to(hit[:, None, :, None], want.shape)
        assert same.numpy().reshape(*want.shape, -1)[rest].all(), f"{label} {name}: other slots"
        z = want / scale
        if b.cache == "e4m3":
            z = np.clip(z, -448, 448)
        u, tiny = U[b.cache], TINY[b.cache]
        err = u * np.abs(z) + tiny
        if n is not None:
            err = turned_bound(np.where(rest, 0, n), half, adjacent, b.dim, "f32", 0 * n) / scale * \
                (1 + u) + err
        err = err + 2 * E32 * np.abs(z)              # the division
        on = ~rest
        within(host(t)[on], z[on], err[on], f"{label} {name}")


APPEND = [
    # new, ctx, hq, hk, dim, page, sections, adjacent
    ([1], [0], 2, 1, 64, 16, (32,), False),
    ([1, 1, 1], [0, 15, 16], 4, 2, 128, 16, (16, 24, 24), False),
    ([17, 0, 33, 1], [5, 9, 0, 64], 3, 3, 80, 32, (8, 16, 16), True),
    ([100], [28], 0, 2, 96, 64, (24, 24), False),
    ([5, 70], [250, 3], 8, 1, 256, 128, (32, 48, 48), True),
    ([3] * 70, list(range(70)), 2, 1, 32, 16, (8,), False),
    ([2, 300], [600, 1], 2, 2, 16, 256, (), False),
]


@pytest.mark.parametrize("dtype,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"),
                                         ("bf16", "e4m3")])
@pytest.mark.parametrize("case", APPEND, ids=str)
@pytest.mark.parametrize("norm", [True, False])
def test_append(case, dtype, cache, norm):
    new, ctx, hq, hk, dim, page, sections, adjacent = case
    rng = np.random.default_rng(11)
    b = Batch(rng, new, ctx, hk, dim, page, dtype, cache, lead=2, tail=3, wide=1)
    pos_t, pos, f_t, f = make_rope(rng, sections, b.n)
    rope = dws.Rope(f_t, sections, int(adjacent))
    parts = packed(rng, b.n, ([hq] if hq else []) + [hk, hk], dim, dtype)
    q, k, v = parts if hq else [(None, None)] + parts
    w = [values(rng, (dim,), dtype) if norm else (None, None) for _ in range(2)]
    before = b.kt.clone(), b.vt.clone()
    out = torch.full((b.n, hq, dim), 9.0, dtype=DT[dtype], device=dev()) if hq else None
    got = dws.bevpool_kv_append(k[0], v[0], b.pool, b.batch, pos_t, rope, q=q[0],
                                q_weight=w[0][0] if hq else None, k_weight=w[1][0], eps=EPS,
                                q_out=out)
    torch.cuda.synchronize()
    n64 = ref.norm(k[1], w[1][1], EPS)
    _check_append(b, got, before, ref.turn(n64, pos, f, sections, adjacent), v[1], n64,
                  sum(sections), adjacent)
    if not hq:
        assert got is None
        return
    nq = ref.norm(q[1], w[0][1], EPS)
    want = ref.turn(nq, pos, f, sections, adjacent)
    inside = slice(int(b.offsets[0]), int(b.offsets[-1]))
    within(host(got)[inside], want[inside],
           turned_bound(nq, sum(sections), adjacent, dim, dtype, want)[inside], "q")
    assert (got[:inside.start] == 9).all() and (got[inside.stop:] == 9).all()


def test_append_drops_what_has_no_slot():
    """Pages outside the pool, places past the table, and negative ones (more
    new tokens than the sequence has) are dropped; queries are still turned."""
    rng = np.random.default_rng(12)
    b = Batch(rng, [40, 20, 6], [8, 0, 10], 2, 64, 16, "bf16", "bf16")
    b.table[0, 1] = -1
    b.table[0, 2] = b.n_pages
    b.kv[1] = 12                       # 20 new tokens in a sequence of 12
    b.kv[2] = 50                       # past the table's 48 places; its last pages are not there
    b.gpu()
    pos_t, pos, f_t, f = make_rope(rng, (32,), b.n)
    k, v = packed(rng, b.n, [2, 2], 64, "bf16")
    q = values(rng, (b.n, 2, 64), "bf16")
    before = b.kt.clone(), b.vt.clone()
    got = dws.bevpool_kv_append(k[0], v[0], b.pool, b.batch, pos_t, dws.Rope(f_t, (32,)), q=q[0])
    torch.cuda.synchronize()
    _check_append(b, got, before, ref.turn(k[1], pos, f, (32,), False), v[1], k[1], 32, False)
    want = ref.turn(q[1], pos, f, (32,), False)
    within(host(got), want, turned_bound(q[1], 32, False, 64, "bf16", want))


@pytest.mark.parametrize("dim", [16, 128])
@pytest.mark.parametrize("empty", [3, 90])
def test_append_many_empty_sequences(dim, empty):
    """Sequences without new tokens between the tokens of one wave, fewer and
    more than it has lanes."""
    rng = np.random.default_rng(14)
    new = [2] + [0] * empty + [5, 0, 0, 1, 60] + [0] * empty
    b = Batch(rng, new, [3 * i % 40 for i in range(len(new))], 2, dim, 16, "bf16", "bf16", lead=3,
              tail=2)
    k, v = packed(rng, b.n, [2, 2], dim, "bf16")
    before = b.kt.clone(), b.vt.clone()
    got = dws.bevpool_kv_append(k[0], v[0], b.pool, b.batch, None, None)
    torch.cuda.synchronize()
    _check_append(b, got, before, k[1], v[1], k[1], 0, False)
    q = values(rng, (b.n, 2, dim), "bf16")
    _check_attention(b, q, 2, k=host(b.kt), v=host(b.vt))


@pytest.mark.parametrize("scale", [2.0 ** -64, 0.013, 2.0 ** 64])
def test_append_e4m3_range(scale):
    """Values past 448 scales are cut, infinities too, NaN stays NaN."""
    rng = np.random.default_rng(13)
    b = Batch(rng, [16], [0], 1, 16, 16, "bf16", "e4m3", k_scale=scale, v_scale=scale)
    k, v = packed(rng, 16, [1, 1], 16, "bf16")
    v[0].mul_(scale * 200)
    v[0][0, 0, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    v64 = host(v[0]) / scale
    dws.bevpool_kv_append(k[0], v[0], b.pool, b.batch, None, None)
    got = host(b.vt)[b.table[0, 0], 0]
    want = np.clip(v64[:, 0], -448, 448)
    within(got, want, U["e4m3"] * np.abs(want) + TINY["e4m3"])
    assert got[0, 0] == 448 and got[0, 1] == -448 and np.isnan(got[0, 2])


# ---- attention ----------------------------------------------------------------------------
def _check_attention(b, q, hq, scale=None, causal=True, window=0, out=None, label="", stream=None,
                     workspace=None, k=None, v=None):
    sc = b.dim ** -0.5 if scale is None else scale
    want, mag, spread, seen = ref.attention(q[1], b.k0 if k is None else k, b.v0 if v is None else v,
                                            b.offsets, b.kv, b.table, sc, causal, window)
    got = dws.bevpool_paged_attention(q[0], b.pool, b.batch, scale, causal, window, out=out,
                                      workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    u = U["f16" if b.cache == "e4m3" else b.dtype]
    d = 2 * (b.dim + 8) * E32 * spread + 2.0 ** -21
    rel = (u + 2 * d + 2 * seen * E32 + 2.0 ** -20)[..., None]
    vmax = np.nanmax(np.abs(np.where(np.isfinite(b.v0), b.v0, 0)), initial=0.0)
    err = mag * rel * (1 + U[b.dtype]) + U[b.dtype] * np.abs(want) + TINY[b.dtype]
    if u == U["f16"]:
        err = err + (seen * 2.0 ** -25)[..., None] * vmax
    inside = ~np.isnan(want).all((1, 2))
    within(host(got)[inside], want[inside], err[inside], label)
    return got


ATTEND = [
    # new, ctx, hq, hk, dim, page
    ([1], [0], 1, 1, 64, 16),
    ([1], [1], 4, 1, 128, 16),
    ([1], [510], 8, 2, 64, 16),
    ([1, 1, 1, 1], [0, 15, 16, 300], 8, 2, 128, 32),
    ([1] * 70, [7 * i for i in range(70)], 3, 1, 80, 16),
    ([1, 1], [2500, 31], 16, 1, 96, 64),
    ([2, 3], [40, 500], 32, 1, 128, 128),
    ([5], [0], 2, 2, 16, 16),
    ([33], [31], 4, 4, 32, 16),
    ([64], [64], 2, 1, 64, 64),
    ([130], [70], 5, 5, 80, 32),
    ([100, 0, 1, 29], [0, 50, 333, 64], 6, 2, 128, 16),
    ([257], [300], 4, 1, 128, 256),
    ([70], [600], 7, 1, 256, 64),
    ([19, 1], [3, 900], 2, 1, 256, 16),
    ([41], [77], 3, 3, 144, 16),
    ([300, 1, 1], [10, 1300, 5], 2, 2, 48, 32),
]


@pytest.mark.parametrize("dtype,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"),
                                         ("bf16", "e4m3")])
@pytest.mark.parametrize("case", ATTEND, ids=str)
@pytest.mark.parametrize("mask", ["causal", "all", "window", "window_all"])
def test_attention(case, dtype, cache, mask):
    new, ctx, hq, hk, dim, page = case
    rng = np.random.default_rng(21)
    b = Batch(rng, new, ctx, hk, dim, page, dtype, cache)
    q = values(rng, (b.n, hq, dim), dtype, 1.5)
    _check_attention(b, q, hq, causal=mask in ("causal", "window"),
                     window=37 if "window" in mask else 0)


def test_attention_long_context_single_tokens():
    """Contexts that are split over many blocks, beside short ones."""
    rng = np.random.default_rng(22)
    for new, ctx, hq, hk, dim, cache in (([1, 1, 1], [20000, 3, 9000], 4, 1, 64, "f16"),
                                         ([1], [33000], 2, 2, 128, "e4m3"),
                                         ([2, 8], [15000, 7000], 8, 2, 128, "f16")):
        b = Batch(rng, new, ctx, hk, dim, 64, "f16", cache)
        q = values(rng, (b.n, hq, dim), "f16", 2.0)
        _check_attention(b, q, hq)
        _check_attention(b, q, hq, window=5000)


def test_attention_chunk_over_a_long_context():
    rng = np.random.default_rng(23)
    b = Batch(rng, [150], [6000], 1, 128, 32, "bf16", "bf16")
    q = values(rng, (b.n, 2, 128), "bf16", 2.0)
    _check_attention(b, q, 2)


def test_attention_rows_without_keys():
    """Empty caches, more new tokens than cached ones, pages that are not
    there, and a window that holds only missing pages: those rows are 0."""
    rng = np.random.default_rng(24)
    b = Batch(rng, [4, 40, 3, 1], [0, 0, 60, 70], 2, 64, 16, "bf16", "bf16")
    b.kv[0] = 0
    b.kv[1] = 25                                  # its first 15 tokens see nothing
    b.table[2, 1:3] = -1
    b.table[3, 3:] = b.n_pages + 5
    b.gpu()
    q = values(rng, (b.n, 4, 64), "bf16")
    got = _check_attention(b, q, 4)
    assert (got[:4 + 15] == 0).all() and (got[19:44] != 0).any(-1).all()
    got = _check_attention(b, q, 4, window=3)
    assert (got[-1] == 0).all()                    # its last 23 places are on no page
    b.kv[:] = [-5, -1, 0, -(2 ** 31)]
    b.gpu()
    for causal in (True, False):
        assert (dws.bevpool_paged_attention(q[0], b.pool, b.batch, causal=causal) == 0).all()


def test_attention_leaves_other_rows():
    rng = np.random.default_rng(25)
    b = Batch(rng, [3, 0, 50], [9, 4, 100], 1, 64, 16, "f16", "f16", lead=5, tail=7, wide=3)
    q = values(rng, (b.n, 2, 64), "f16")
    buf = torch.full((b.n, 5, 64), 3.0, dtype=torch.float16, device=dev())
    got = _check_attention(b, q, 2, out=buf[:, 1:3])
    assert (got[:5] == 3).all() and (got[-7:] == 3).all()
    assert (buf[:, 0] == 3).all() and (buf[:, 3:] == 3).all()


@pytest.mark.parametrize("new,ctx", [([1], [200]), ([48], [152]), ([200], [100])])
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), -float("inf")])
def test_attention_hidden_non_finite_values(new, ctx, bad):
    """Infinities and NaN in keys and values that a row does not see leave no
    trace in it; rows that see them get them."""
    rng = np.random.default_rng(26)
    b = Batch(rng, new, ctx, 1, 64, 16, "bf16", "bf16")
    q = values(rng, (b.n, 2, 64), "bf16")
    kv, n = int(b.kv[0]), int(new[0])
    page, slot = b.table[0, (kv - 1) // 16], (kv - 1) % 16
    k, v = b.k0.copy(), b.v0.copy()
    v[page, 0, slot, 5] = bad                # the last place: seen by the last token alone
    b.vt[page, 0, slot, 5] = bad
    first = b.table[0, 0]                    # the first place: outside the window of all
    k[first, 0, 0, :] = v[first, 0, 0, :] = bad
    b.kt[first, 0, 0], b.vt[first, 0, 0] = bad, bad
    got = _check_attention(b, q, 2, window=kv - n, k=k, v=v)
    assert torch.isfinite(got[:-1]).all()
    assert not torch.isfinite(got[-1, :, 5]).any()
    rest = torch.cat([got[-1, :, :5], got[-1, :, 6:]], -1)
    assert torch.isfinite(rest).all()


def test_attention_scale_and_large_scores():
    rng = np.random.default_rng(27)
    b = Batch(rng, [1, 80], [300, 40], 2, 128, 32, "bf16", "bf16")
    q = values(rng, (b.n, 4, 128), "bf16", 20.0)
    for scale in (1.0, 1e-4, 0.0883883):
        _check_attention(b, q, 4, scale=scale)


def test_attention_strided_queries():
    rng = np.random.default_rng(28)
    b = Batch(rng, [37, 1], [60, 90], 2, 80, 16, "f16", "f16")
    q, _ = packed(rng, b.n, [6, 4], 80, "f16")
    _check_attention(b, q, 6)


def test_attention_shared_pages():
    """Two sequences that read the same pages, and one page twice in a table."""
    rng = np.random.default_rng(29)
    b = Batch(rng, [1, 1, 20], [100, 100, 28], 1, 64, 16, "bf16", "bf16")
    b.table[1] = b.table[0]
    b.table[2, 1] = b.table[2, 0]
    b.gpu()
    q = values(rng, (b.n, 2, 64), "bf16")
    _check_attention(b, q, 2)


def test_attention_cache_past_32_bits():
    """Pages whose offset passes 2^32 bytes and 2^32 elements."""
    rng = np.random.default_rng(30)
    hk, dim, page = 8, 256, 256
    n_pages = (1 << 32) // (hk * dim * page) + 40
    kt, vt = (torch.zeros((n_pages, hk, page, dim), dtype=torch.bfloat16, device=dev())
              for _ in range(2))
    b = Batch(rng, [1, 30], [700, 300], hk, dim, page, "bf16", "bf16")
    ids = np.array([n_pages - 1 - 5 * i for i in range(b.n_pages)], np.int32)
    for i, at in enumerate(ids):
        kt[at], vt[at] = b.kt[i], b.vt[i]
    small = b.table.copy()
    q = values(rng, (b.n, hk, dim), "bf16")
    want = _check_attention(b, q, hk)
    b.table = np.where(small >= 0, ids[small], -1).astype(np.int32)
    b.kt, b.vt = kt, vt
    b.gpu()
    got = dws.bevpool_paged_attention(q[0], b.pool, b.batch)
    assert torch.equal(got, want)
    # and the append writes there
    pos_t, _, f_t, _ = make_rope(rng, (128,), b.n)
    k, v = packed(rng, b.n, [hk, hk], dim, "bf16")
    dws.bevpool_kv_append(k[0], v[0], b.pool, b.batch, pos_t, dws.Rope(f_t, (128,)))
    at = int(b.kv[0]) - 1
    assert torch.equal(vt[int(b.table[0, at // page]), :, at % page], v[0][0])


def test_attention_same_bits_and_overlapping_calls():
    """Two calls at once on two streams, each with its own workspace, give
    what one gives alone, every time."""
    rng = np.random.default_rng(31)
    b = Batch(rng, [1, 1, 40], [9000, 100, 2000], 2, 128, 64, "bf16", "bf16")
    q = values(rng, (b.n, 8, 128), "bf16")
    want = dws.bevpool_paged_attention(q[0], b.pool, b.batch)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [dws.bevpool_paged_attention(q[0], b.pool, b.batch, stream=s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("dim,dtype,cache", [(64, "f16", "f16"), (80, "bf16", "e4m3"),
                                             (96, "f16", "e4m3"), (128, "bf16", "bf16"),
                                             (128, "f16", "e4m3"), (48, "bf16", "bf16"),
                                             (112, "f16", "f16")])
@pytest.mark.parametrize("mask", ["causal", "all", "window"])
def test_attention_many_rows(dim, dtype, cache, mask):
    """Enough rows for tiles of 256: 15616 a key head are 122 tiles of 128 or 61
    of 256, for each of four key heads, on 256 CUs.  The last of a sequence is
    not full.  Some heads of two key heads against the oracle."""
    rng = np.random.default_rng(33)
    new, ctx, hq, hk, page = [573, 3, 400], [95, 300, 41], 64, 4, 32
    b = Batch(rng, new, ctx, hk, dim, page, dtype, cache)
    q = values(rng, (b.n, hq, dim), dtype, 1.5)
    causal, window = mask != "all", 150 if mask == "window" else 0
    got = dws.bevpool_paged_attention(q[0], b.pool, b.batch, causal=causal, window=window)
    torch.cuda.synchronize()
    assert torch.isfinite(got).all()
    for g, heads in ((2, slice(33, 48, 7)), (0, slice(0, 16, 15))):
        # the heads picked share key head g, so the oracle gets that one alone
        want, mag, spread, seen = ref.attention(q[1][:, heads], b.k0[:, g:g + 1], b.v0[:, g:g + 1],
                                                b.offsets, b.kv, b.table, dim ** -0.5, causal, window)
        u = U["f16" if cache == "e4m3" else dtype]
        rel = (u + 4 * (dim + 8) * E32 * spread + 2.0 ** -20 + 2 * seen * E32 + 2.0 ** -20)[..., None]
        err = mag * rel * (1 + U[dtype]) + U[dtype] * np.abs(want) + TINY[dtype]
        if u == U["f16"]:
            err = err + (seen * 2.0 ** -25)[..., None] * np.nanmax(np.abs(b.v0))
        within(host(got[:, heads]), want, err, f"key head {g}")


@pytest.mark.parametrize("dim,cache", [(128, "bf16"), (256, "bf16"), (256, "e4m3"), (64, "e4m3")])
def test_attention_few_blocks_in_splits(dim, cache):
    """Tiles of many rows whose keys are cut over blocks: those of a sequence
    that ends early have no key in the later ones."""
    rng = np.random.default_rng(34)
    b = Batch(rng, [40, 90, 2], [4100, 30, 0], 2, dim, 64, "bf16", cache)
    q = values(rng, (b.n, 6, dim), "bf16", 1.5)
    _check_attention(b, q, 6)
    _check_attention(b, q, 6, causal=False, window=2000)


@pytest.mark.parametrize("new,ctx,hq,cache", [([1], [40000], 64, "bf16"), ([30], [20000], 6, "e4m3"),
                                              ([1, 50], [17000, 10], 48, "bf16")])
def test_attention_few_blocks_in_many_splits(new, ctx, hq, cache):
    """One or two tiles of more than 32 rows over long contexts: more than 16
    splits of each."""
    rng = np.random.default_rng(38)
    b = Batch(rng, new, ctx, 1, 64, 64, "bf16", cache)
    q = values(rng, (b.n, hq, 64), "bf16", 1.5)
    _check_attention(b, q, hq)


@pytest.mark.parametrize("new,ctx", [([1], [200]), ([48], [152]), ([200], [100])])
def test_attention_hidden_nan_codes(new, ctx):
    """The same of e4m3 caches, whose one value that is not finite is NaN."""
    rng = np.random.default_rng(35)
    b = Batch(rng, new, ctx, 1, 128, 16, "f16", "e4m3")
    q = values(rng, (b.n, 2, 128), "f16")
    kv, n = int(b.kv[0]), int(new[0])
    page, slot, first = b.table[0, (kv - 1) // 16], (kv - 1) % 16, b.table[0, 0]
    k, v = b.k0.copy(), b.v0.copy()
    v[page, 0, slot, 5] = k[first, 0, 0, :] = v[first, 0, 0, :] = np.nan
    _codes(b.vt)[page, 0, slot, 5] = 0x7f
    _codes(b.kt)[first, 0, 0], _codes(b.vt)[first, 0, 0] = 0xff, 0x7f
    got = _check_attention(b, q, 2, window=kv - n, k=k, v=v)
    assert torch.isfinite(got[:-1]).all() and torch.isnan(got[-1, :, 5]).all()
    assert torch.isfinite(got[-1, :, :5]).all() and torch.isfinite(got[-1, :, 6:]).all()


def test_attention_graphs_that_share_a_workspace():
    """Two graphs captured with one workspace, replayed in turn on one stream
    with eager calls between them."""
    rng = np.random.default_rng(36)
    b = Batch(rng, [1, 40], [9000, 2000], 2, 64, 64, "bf16", "bf16")
    q = [values(rng, (b.n, 4, 64), "bf16")[0] for _ in range(2)]
    need = dws.bevpool_paged_attention_workspace_size(b.n, 2, 4, 2, 64, 64, b.table.shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    want = [dws.bevpool_paged_attention(x, b.pool, b.batch) for x in q]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in q:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(dws.bevpool_paged_attention(x, b.pool, b.batch, workspace=ws))
    for _ in range(3):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        eager = dws.bevpool_paged_attention(q[0], b.pool, b.batch, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
        assert torch.equal(eager, want[0])


def test_attention_empty_and_wide_batches():
    """No sequences, no tokens, a table of no pages, and one far wider than the
    sequences need."""
    rng = np.random.default_rng(39)
    b = Batch(rng, [1, 40], [70, 30], 2, 64, 16, "bf16", "bf16")
    q = values(rng, (b.n, 4, 64), "bf16")
    none = torch.empty(0, dtype=torch.int32, device=dev())
    zero = torch.zeros(1, dtype=torch.int32, device=dev())
    out = torch.full_like(q[0], 5.0)
    empty = dws.PagedBatch(zero, none, none.view(0, 4))
    assert (dws.bevpool_paged_attention(q[0], b.pool, empty, out=out) == 5).all()
    got = dws.bevpool_paged_attention(q[0][:0], b.pool, b.batch)
    assert got.shape == (0, 4, 64)
    no_pages = dws.PagedBatch(b.batch.q_offsets, b.batch.kv_lengths, none.view(2, 0))
    assert (dws.bevpool_paged_attention(q[0], b.pool, no_pages) == 0).all()
    before = b.kt.clone()
    kv = values(rng, (b.n, 2, 64), "bf16")[0]
    dws.bevpool_kv_append(kv, kv, b.pool, no_pages, None, None)
    dws.bevpool_kv_append(kv, kv, b.pool, empty, None, None)
    dws.bevpool_kv_append(kv[:0], kv[:0], b.pool, b.batch, None, None)
    assert torch.equal(_codes(b.kt).view(torch.int16), _codes(before).view(torch.int16))
    wide = np.full((2, 20000), -1, np.int32)
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    b.gpu()
    _check_attention(b, q, 4)


def test_attention_refusals():
    rng = np.random.default_rng(37)
    b = Batch(rng, [3, 40], [4, 9000], 2, 64, 16, "bf16", "bf16")
    q = values(rng, (b.n, 4, 64), "bf16")[0]
    call = dws.bevpool_paged_attention
    with pytest.raises(TypeError):
        call(q.cpu(), b.pool, b.batch)
    with pytest.raises((TypeError, ValueError, dws.BevPoolError)):
        call(q.float(), b.pool, b.batch)                       # fp32 tokens
    with pytest.raises((TypeError, ValueError, dws.BevPoolError)):
        call(q.half(), b.pool, b.batch)                        # an fp16 query, a bf16 cache
    with pytest.raises((ValueError, dws.BevPoolError)):
        call(q[:, :3], b.pool, b.batch)                        # 3 heads on 2
    with pytest.raises(ValueError):
        call(q[:, :, :32], b.pool, b.batch)
    with pytest.raises(ValueError):
        call(q.transpose(0, 1), b.pool, b.batch)
    with pytest.raises(dws.BevPoolError):
        call(q, b.pool, b.batch, window=-1)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises((ValueError, dws.BevPoolError)):
            call(q, b.pool, b.batch, scale)
    need = dws.bevpool_paged_attention_workspace_size(b.n, 2, 4, 2, 64, 16, b.table.shape[1])
    with pytest.raises(dws.BevPoolError):
        call(q, b.pool, b.batch, workspace=torch.empty(need - 256, dtype=torch.uint8, device=dev()))
    with pytest.raises(TypeError):
        call(q, b.pool, b.batch, workspace=torch.empty(need, device=dev()))
    with pytest.raises(ValueError):
        call(q, b.pool, b.batch, out=torch.empty_like(q)[:, :2])
    with pytest.raises(ValueError):                            # a cache of another shape
        dws.PagedCache(b.kt, b.vt[:1])


# ---- in a row -----------------------------------------------------------------------------
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_frames_then_steps(cache):
    """Three frames of BEV tokens (all of a frame see each other and the
    earlier frames), then single tokens, through append and attention, against
    the oracle's own cache; the steps once eagerly and once as a graph that is
    replayed with the batch's arrays rewritten between replays."""
    rng = np.random.default_rng(41)
    hq, hk, dim, page, sections = 4, 2, 64, 16, (8, 12, 12)
    rows, cols, frames, steps, seqs = 5, 9, 3, 4, 2
    cells = rows * cols
    total = frames * cells + steps
    width = -(-total // page)
    k_scale, v_scale = (0.02, 0.015) if cache == "e4m3" else (1.0, 1.0)
    kt, vt = (torch.full((seqs * width, hk, page, dim), float("nan"), device=dev()).to(DT[cache])
              for _ in range(2))
    pool = dws.PagedCache(kt, vt, k_scale, v_scale)
    table = rng.permutation(seqs * width).astype(np.int32).reshape(seqs, width)
    _, _, f_t, f = make_rope(rng, sections, 1)
    rope = dws.Rope(f_t, sections)
    wq, wk = values(rng, (dim,), "bf16"), values(rng, (dim,), "bf16")

    def to(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev())

    def check(got, q_turned, lens, n, causal):
        b = Batch.__new__(Batch)
        b.offsets, b.kv, b.table = np.arange(seqs + 1) * n, np.full(seqs, lens), table
        b.dim, b.dtype, b.cache = dim, "bf16", cache
        k64, v64 = host(kt) * k_scale, host(vt) * v_scale
        want, mag, spread, seen = ref.attention(host(q_turned), k64, v64, b.offsets, b.kv, table,
                                                dim ** -0.5, causal, 0)
        u = U["f16" if cache == "e4m3" else "bf16"]
        rel = (u + 4 * (dim + 8) * E32 * spread + 2.0 ** -20 + 2 * seen * E32 + 2.0 ** -20)[..., None]
        within(host(got), want, mag * rel * (1 + U["bf16"]) + U["bf16"] * np.abs(want) +
               (seen * 2.0 ** -25)[..., None] * np.nanmax(np.abs(v64)), "out")

    def step_inputs(n, start, frame):
        parts = packed(rng, seqs * n, [hq, hk, hk], dim, "bf16")
        i = np.arange(n)
        point = np.stack([np.full(n, frame), i // cols, i % cols]).astype(np.int32)
        return parts, np.concatenate([point] * seqs, 1), np.full(seqs, start + n, np.int32)

    done = 0
    for frame in range(frames):
        (q, k, v), point, lens = step_inputs(cells, done, frame)
        done += cells
        batch = dws.PagedBatch(to(np.arange(seqs + 1, dtype=np.int32) * cells), to(lens), to(table))
        qt = dws.bevpool_kv_append(k[0], v[0], pool, batch, to(point), rope, q=q[0],
                                   q_weight=wq[0], k_weight=wk[0])
        nq = ref.norm(q[1], wq[1], 1e-6)
        want = ref.turn(nq, point, f, sections, False)
        within(host(qt), want, turned_bound(nq, 32, False, dim, "bf16", want), "q")
        # the turned queries of the other entry point are the same
        same = dws.bevpool_qk_norm_rope(q[0], None, to(point), rope, wq[0])[0]
        assert torch.equal(same, qt)
        got = dws.bevpool_paged_attention(qt, pool, batch, causal=False)
        check(got, qt, done, cells, False)

    lens_t, pos_t = to(np.zeros(seqs, np.int32)), to(np.zeros((3, seqs), np.int32))
    batch = dws.PagedBatch(to(np.arange(seqs + 1, dtype=np.int32)), lens_t, to(table))
    (q, k, v), _, _ = step_inputs(1, done, frames)

    def step():
        qt = dws.bevpool_kv_append(k[0], v[0], pool, batch, pos_t, rope, q=q[0], q_weight=wq[0],
                                   k_weight=wk[0])
        return qt, dws.bevpool_paged_attention(qt, pool, batch)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lens_t.fill_(done + 1)
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(steps):
        parts, point, lens = step_inputs(1, done, frames + i)
        for dst, src in zip((q, k, v), parts):
            dst[0].copy_(src[0])
        lens_t.copy_(to(lens))
        pos_t.copy_(to(point))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in captured]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(replayed, eager)), i
        done += 1
        check(eager[1], eager[0], done, 1, True)
