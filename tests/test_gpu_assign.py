"""The pages of a step against the oracle: whole numbers, all equal."""
import numpy as np
import pytest
import torch

import depth_weighted_scatter_amd as dws
from depth_weighted_scatter_amd import tokens
from oracle import tokens as ref
from token_util import dev

pytestmark = pytest.mark.gpu


def to(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


class Pool:
    """Sequences with kv cached tokens each, pages anywhere in the pool, junk in
    the table and the list where nothing is kept."""

    def __init__(self, rng, kv, page, width=None, spare=10, capacity=None, separate=False):
        self.kv, self.page = np.array(kv, np.int32).reshape(-1), page
        need = np.maximum(-(-self.kv.astype(np.int64) // page), 0)
        width = int(need.max(initial=0)) + 4 if width is None else width
        fits = np.minimum(need, width)
        self.n_pages = int(fits.sum()) + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = rng.integers(-5, 10 ** 6, (len(self.kv), width)).astype(np.int32)
        at = 0
        for s, c in enumerate(fits):
            self.table[s, :c] = order[at:at + c]
            at += c
        self.count = self.n_pages - at
        self.free = rng.integers(-5, 10 ** 6, capacity or self.n_pages).astype(np.int32)
        self.free[:self.count] = order[at:]
        self.separate = separate
        self.gpu()

    def gpu(self):
        extra = {}
        if self.separate:
            extra = dict(next_lengths=torch.full((len(self.kv),), 77, dtype=torch.int32, device=dev()),
                         next_free=torch.full((1,), 77, dtype=torch.int32, device=dev()))
        self.pages = dws.PageTable(to(self.table), to(self.kv), to(self.free), to([self.count]),
                                   self.page, self.n_pages, **extra)

    def want(self, new, keep, n_tokens):
        return ref.assign_pages(new, keep, self.kv, self.table, self.free, self.count, self.page,
                                self.n_pages, n_tokens)

    def step(self, new, keep, n_tokens, **kw):
        return dws.bevpool_assign_pages(to(new), self.pages, n_tokens,
                                        keep_lengths=None if keep is None else to(keep), **kw)

    def compare(self, got, want):
        p = self.pages
        for name, t, w in (("status", got[2], [want["status"]]), ("offsets", p.q_offsets, want["offsets"]),
                           ("lengths", p.next_lengths, want["lengths"]),
                           ("count", p.next_free, [want["count"]]), ("table", p.block_table, want["table"]),
                           ("free", p.free_pages, want["free"]), ("places", got[1], want["places"]),
                           ("slots", got[0], want["slots"])):
            assert np.array_equal(t.cpu().numpy(), np.asarray(w)), name
        if self.separate:
            assert np.array_equal(p.kv_lengths.cpu().numpy(), self.kv) and int(p.free_count) == self.count


def lengths(rng, n, kv_most, new_most, kind):
    kv = rng.integers(0, kv_most + 1, n)
    new = rng.integers(0, new_most + 1, n)
    if kind == "grow":
        return kv, new, None
    if kind == "drop":
        return kv, np.zeros(n, int), rng.integers(0, kv + 1)
    keep = np.where(rng.random(n) < 0.5, rng.integers(0, kv + 1), kv)
    return kv, new * (rng.random(n) < 0.7), keep


SIZES = [(1, 0, 1, 16), (1, 1, 1, 16), (1, 300, 40, 16), (3, 16, 16, 16), (64, 500, 1, 16),
         (65, 100, 3, 32), (1000, 60, 5, 16), (1025, 40, 2, 64), (3000, 300, 9, 256), (5, 900, 5000, 64),
         (200, 3000, 700, 128), (5003, 50, 3, 16), (20001, 30, 2, 32)]


@pytest.mark.parametrize("n,kv_most,new_most,page", SIZES)
@pytest.mark.parametrize("kind", ["grow", "drop", "mixed"])
@pytest.mark.parametrize("separate", [False, True])
def test_steps(n, kv_most, new_most, page, kind, separate):
    rng = np.random.default_rng(201)
    kv, new, keep = lengths(rng, n, kv_most, new_most, kind)
    p = Pool(rng, kv, page, int(-(-(kv_most + new_most) // page)) + 1,
             spare=int((-(-new // page) + 1).sum()) + 3, separate=separate)
    n_tokens = int(new.sum()) + 5
    want = p.want(new, keep, n_tokens)
    assert want["status"] == 0
    p.compare(p.step(new, keep, n_tokens), want)


def test_exactly_enough_tokens_and_pages():
    rng = np.random.default_rng(202)
    p = Pool(rng, [16, 31, 0], 16, 8, spare=4)
    want = p.want([17, 2, 16], None, 35)
    assert want["status"] == 0 and want["count"] == 0
    p.compare(p.step([17, 2, 16], None, 35), want)


@pytest.mark.parametrize("separate", [False, True])
@pytest.mark.parametrize("n", [3, 1500])
@pytest.mark.parametrize("why", ["pages", "tokens", "table", "table_before", "list"])
def test_refused_steps(why, n, separate):
    """The step is refused as a whole, and the calls that read the batch do
    nothing."""
    rng = np.random.default_rng(203)
    kv = rng.integers(0, 60, n)
    kv[n // 2] = 60
    new, keep, n_tokens = np.full(n, 20), None, 20 * n + 3
    spare, width, capacity = 2 * n, 6, None
    if why == "pages":
        spare = n // 2
    elif why == "tokens":
        n_tokens = 20 * n - 1
    elif why == "table":
        width = 4
    elif why == "table_before":
        kv[n // 2], keep, width = 97, np.zeros(n, int), 6
    else:
        # every slot of the list is filled, and a page comes back
        new, keep = np.zeros(n, int), np.maximum(kv - 16, 0)
    p = Pool(rng, kv, 16, width, spare, capacity, separate)
    if why == "list":
        p.free, p.n_pages = p.free[:p.count].copy(), p.n_pages
        p.gpu()
    want = p.want(new, keep, n_tokens)
    assert want["status"] > 0 if why == "pages" else want["status"] == -1
    p.compare(p.step(new, keep, n_tokens), want)
    assert not p.pages.q_offsets.any()


def test_lengths_out_of_range():
    """Negative lengths count as 0, kept ones beyond the cached as all."""
    rng = np.random.default_rng(204)
    p = Pool(rng, [-5, 20, 40, 33, -(2 ** 31)], 16, 8)
    new, keep = [3, -7, -(2 ** 31), 5, 1], [9, 2 ** 31 - 1, -3, -(2 ** 31), 2 ** 31 - 1]
    want = p.want(new, keep, 12)
    assert want["lengths"].tolist() == [3, 20, 0, 5, 1] and want["status"] == 0
    p.compare(p.step(new, keep, 12), want)


def test_totals_past_32_bits():
    """Thousands of requests for 2^31 - 1 tokens, and a count that is no count."""
    rng = np.random.default_rng(205)
    p = Pool(rng, [5] * 3000, 16, 8)
    new = np.full(3000, 2 ** 31 - 1)
    p.compare(p.step(new, None, 7), p.want(new, None, 7))
    for count in (-4, 10 ** 9):
        p = Pool(rng, [5] * 3, 16, 8)
        p.count = count
        p.gpu()
        p.compare(p.step([40, 40, 40], None, 130), p.want([40, 40, 40], None, 130))


def test_more_tokens_than_31_bits_hold():
    """Room for 2^31 - 1 tokens, pages for all that are asked for, and 3 x 2^30 of
    them: the step is refused (slots and places are not asked for)."""
    n, page, width, listed = 3, 256, 2 ** 22, 3 * 2 ** 22 + 5
    table, kv, new = to(np.zeros((n, width))), to([0] * n), to([2 ** 30] * n)
    free = torch.arange(listed, dtype=torch.int32, device=dev())
    count, offsets, status = to([listed]), to([7] * (n + 1)), to([9])
    ws = torch.empty(dws.bevpool_assign_pages_workspace_size(n), dtype=torch.uint8, device=dev())
    before = free.clone()
    for lengths, want in (([2 ** 30] * 3, -1), ([2 ** 30, 2 ** 30, 0], -1), ([2 ** 30, 2 ** 30 - 1, 0], 0)):
        new.copy_(to(lengths))
        rc = tokens._lib().bevpool_assign_pages(
            new.data_ptr(), None, kv.data_ptr(), kv.data_ptr(), n, table.data_ptr(), width, 1000, page,
            free.data_ptr(), listed, count.data_ptr(), count.data_ptr(), offsets.data_ptr(), None, None,
            2 ** 31 - 1, status.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0 and int(status) == want
        assert torch.equal(free, before)
        if want:
            assert not offsets.any() and not kv.any() and not table.any() and int(count) == listed
    assert kv.tolist() == lengths and offsets.tolist() == [0, 2 ** 30, 2 ** 31 - 1, 2 ** 31 - 1]
    assert int(count) == listed - 2 ** 23
    assert torch.equal(table[:2].reshape(-1), before.flip(0)[:2 ** 23])


def test_wide_table_tokens():
    """2^30 places a row, and new tokens at its very end."""
    rng = np.random.default_rng(206)
    width = 2 ** 22
    p = Pool(rng, [100, 0], 256, width, spare=20)
    far = 2 ** 30 - 10
    p.kv[1] = far
    p.table[1, -1] = 4
    p.gpu()
    want = p.want([30, 10], None, 40)
    assert want["places"][-1] == 2 ** 30 - 1 and want["slots"][-1] == 4 * 256 + 255
    p.compare(p.step([30, 10], None, 40), want)
    p.kv = np.array([130, far], np.int32)
    p.table, p.free, p.count = want["table"], want["free"], want["count"]
    p.gpu()
    want = p.want([1, 11], None, 40)
    assert want["status"] == -1
    p.compare(p.step([1, 11], None, 40), want)


def test_pages_that_are_none():
    """Numbers outside the pool in the table and the list are copied; their
    tokens have no slot."""
    rng = np.random.default_rng(207)
    p = Pool(rng, [20, 20, 40], 16, 6)
    p.table[0, 1], p.table[2, 2], p.free[p.count - 1], p.free[p.count - 2] = -1, p.n_pages, -7, 2 ** 30
    p.gpu()
    want = p.want([20, 20, 0], [20, 20, 3], 45)
    assert (want["slots"][:40] == -1).any()
    p.compare(p.step([20, 20, 0], [20, 20, 3], 45), want)


def test_empty_calls():
    rng = np.random.default_rng(208)
    p = Pool(rng, [], 16, 4, spare=3)
    p.compare(p.step([], None, 6), p.want([], None, 6))
    p = Pool(rng, [17, 3], 16, 4)
    p.compare(p.step([0, 0], None, 0), p.want([0, 0], None, 0))
    p = Pool(rng, [0, 0], 16, 0, spare=3)
    p.compare(p.step([0, 0], None, 3), p.want([0, 0], None, 3))
    p.compare(p.step([0, 1], None, 3), p.want([0, 1], None, 3))
    p = Pool(rng, [0, 0], 16, 4, spare=3, capacity=3)
    p.free, p.count = p.free[:0], 0
    p.gpu()
    p.compare(p.step([0, 1], None, 3), p.want([0, 1], None, 3))


@pytest.mark.parametrize("n,new_most", [(40, 4), (600, 30)])
def test_many_steps_eager_and_replayed(n, new_most):
    """A stream of steps in place, each checked; the second half replays one
    captured call, with the requests rewritten between the replays."""
    rng = np.random.default_rng(209)
    p = Pool(rng, rng.integers(0, 100, n), 16, 20, spare=n * 12)
    n_tokens = n * new_most
    new_t, keep_t = to(np.zeros(n)), to(np.zeros(n))
    out = [torch.zeros(n_tokens, dtype=torch.int32, device=dev()) for _ in range(2)]
    out.append(torch.zeros(1, dtype=torch.int32, device=dev()))

    def call():
        return dws.bevpool_assign_pages(new_t, p.pages, n_tokens, keep_lengths=keep_t, slots=out[0],
                                        places=out[1], status=out[2])

    graph = None
    for i in range(12):
        kv = p.kv
        keep = np.where(rng.random(n) < 0.3, rng.integers(0, kv + 1), kv)
        new = np.minimum(rng.integers(0, new_most + 1, n), 320 - keep)
        want = p.want(new, keep, n_tokens)
        assert want["status"] == 0
        if i == 6:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
        new_t.copy_(to(new))
        keep_t.copy_(to(keep))
        if graph is None:
            call()
        else:
            graph.replay()
        torch.cuda.synchronize()
        p.compare(out, want)
        p.kv, p.table, p.free, p.count = want["lengths"].astype(np.int32), want["table"], want["free"], \
            want["count"]


def test_two_tables_at_once():
    """Two steps on two streams, each with what is its own."""
    rng = np.random.default_rng(210)
    pools = [Pool(rng, rng.integers(0, 300, n), 32, 40, spare=4 * n, separate=True) for n in (900, 1100)]
    new = [rng.integers(0, 30, len(p.kv)) for p in pools]
    wants = [p.want(x, None, 40000) for p, x in zip(pools, new)]
    streams = [torch.cuda.Stream() for _ in pools]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [p.step(x, None, 40000, stream=s) for p, x, s in zip(pools, new, streams)]
        torch.cuda.synchronize()
        for p, g, w in zip(pools, got, wants):
            p.compare(g, w)


def test_refusals():
    rng = np.random.default_rng(211)
    p = Pool(rng, [5, 40], 16, 8)
    new = to([1, 1])
    call = dws.bevpool_assign_pages
    with pytest.raises(TypeError):
        call(new.cpu(), p.pages, 4)
    with pytest.raises(TypeError):
        call(new, p.pages.batch, 4)
    with pytest.raises(TypeError):
        call(new.long(), p.pages, 4)
    with pytest.raises(ValueError):
        call(new[:1], p.pages, 4)
    with pytest.raises(ValueError):
        call(new, p.pages, -1)
    with pytest.raises(ValueError):
        call(new, p.pages, 4, slots=to([0] * 3))
    with pytest.raises(ValueError):
        call(new, p.pages, 4, places=to([0] * 8)[::2])
    with pytest.raises(TypeError):
        call(new, p.pages, 4, keep_lengths=new.float())
    with pytest.raises(ValueError):
        call(new, p.pages, 4, status=to([0, 0]))
    with pytest.raises(dws.BevPoolError):
        call(new, p.pages, 4, workspace=torch.empty(100, dtype=torch.uint8, device=dev()))
    t = p.pages
    with pytest.raises(ValueError):
        dws.PageTable(t.block_table, t.kv_lengths[:1], t.free_pages, t.free_count, 16)
    with pytest.raises(ValueError):
        dws.PageTable(t.block_table, t.kv_lengths, t.free_pages, t.free_pages, 16)
    with pytest.raises(TypeError):
        dws.PageTable(t.block_table, t.kv_lengths, t.free_pages.long(), t.free_count, 16)
    with pytest.raises(dws.BevPoolError):
        call(new, dws.PageTable(t.block_table, t.kv_lengths, t.free_pages, t.free_count, 24), 4)


def test_versions():
    rng = np.random.default_rng(212)
    p = Pool(rng, [5, 40], 16, 8, separate=True)
    new, slots = to([1, 1]), to([0] * 4)
    t = p.pages
    seen = (new, t.kv_lengths, t.free_count, slots, t.block_table, t.free_pages, t.q_offsets,
            t.next_lengths, t.next_free)
    before = [x._version for x in seen]
    dws.bevpool_assign_pages(new, t, 4, slots=slots)
    assert [x._version - v for x, v in zip(seen, before)] == [0, 0, 0, 1, 1, 1, 1, 1, 1]
