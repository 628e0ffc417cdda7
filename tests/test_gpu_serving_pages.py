"""Page management on the GPU against the list form: tables, lengths, counts, status and
every byte of the cache equal."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_serving_kv import bsq, dev_cache, i32, random_cache, same_cache  # noqa: F401

pytestmark = pytest.mark.gpu


def scene(rng, seqs, empty, pages, width, most, heads=2, D=64, spare_table=0):
    """Sequences with random pages, `empty` empty slots behind them."""
    lens = [int(x) for x in rng.integers(0, most + 1, seqs)] + [0] * empty
    order = list(rng.permutation(pages))
    table = rng.integers(-5, pages + 5, (seqs + empty, width + spare_table))
    refs = np.zeros(pages, int)
    for s in range(seqs):
        for k in range(R.pages_of(lens[s])):
            table[s, k] = order.pop()
            refs[table[s, k]] = 1
    return lens, table, refs, random_cache(rng, pages, heads, D)


class Both:
    """The device's state and the reference's."""

    def __init__(self, bsq, lens, table, refs, cache, pad=0):
        self.bsq, self.cache = bsq, cache
        self.pool = R.Pool(table.tolist(), lens, refs.tolist())
        self.wide = torch.full((table.shape[0], table.shape[1] + pad), -7, dtype=torch.int32,
                               device="cuda")
        self.table = self.wide[:, :table.shape[1]]
        self.table.copy_(i32(table))
        self.lens, self.refs, self.d = i32(lens), i32(refs), dev_cache(bsq, cache)

    def same(self):
        torch.cuda.synchronize()
        assert self.lens.tolist() == self.pool.lens
        assert self.refs.tolist() == self.pool.refs
        for s, n in enumerate(self.pool.lens):               # entries past the end mean nothing
            m = R.pages_of(max(n, 0))
            assert self.table[s, :m].tolist() == self.pool.table[s][:m], s
        assert torch.all(self.wide[:, self.table.shape[1]:] == -7)
        same_cache(self.d, self.cache)

    def fork(self, parents, children):
        st = self.bsq.kv_pages_fork(self.d, self.table, self.lens, self.refs, i32(parents), i32(children))
        assert st.tolist() == self.pool.fork(parents, children, self.cache)
        self.same()

    def reserve(self, slots, add):
        st = self.bsq.kv_pages_reserve(self.table, self.lens, self.refs, i32(slots), i32(add))
        assert st.tolist() == self.pool.reserve(slots, add)
        self.same()

    def free(self, slots):
        self.bsq.kv_pages_free(self.table, self.lens, self.refs, i32(slots))
        self.pool.free(slots)
        self.same()

    def compact(self, inplace):
        if inplace:
            kw = dict(table_out=self.table, refcounts_out=self.refs)
        else:
            kw = {}
        t, r, n = self.bsq.kv_pages_compact(self.d, self.table, self.lens, self.refs, **kw)
        assert n.tolist() == [self.pool.compact(self.cache)]
        if not inplace:
            self.table.copy_(t)
            self.refs = r
        self.same()


@pytest.mark.parametrize("heads,D", [(1, 64), (3, 128), (2, 256)])
def test_a_life_of_pages(bsq, heads, D):  # noqa: F811
    """Fork, lengthen, free, fork again, compact: shared and single pages, slots reused."""
    rng = np.random.default_rng(heads)
    b = Both(bsq, *scene(rng, 5, 6, 60, 6, 300, heads, D), pad=3)
    b.fork([0, 1, 2, 0], [5, 6, 7, 8])
    b.reserve([0, 5, 8, 6], [1, 64, 63, 0])
    b.free([0, 6])
    b.fork([5, 8], [0, 6])
    b.compact(False)
    b.free([1, 2, 3])
    b.compact(True)
    b.reserve([1, 2], [200, 64])
    b.compact(True)
    b.free(list(range(11)))
    assert b.refs.sum().item() == 0
    b.compact(False)


@pytest.mark.parametrize("pages_left", [0, 1, 3])
def test_not_enough_pages(bsq, pages_left):  # noqa: F811
    """Requests are served in order until the pages end; what fails changes nothing."""
    rng = np.random.default_rng(7)
    lens, table, refs, cache = scene(rng, 6, 6, 40, 8, 0)
    lens[:6] = [65, 130, 64, 10, 0, 200]
    free = list(rng.permutation(40))
    for s in range(6):
        for k in range(R.pages_of(lens[s])):
            table[s, k] = free.pop()
            refs[table[s, k]] = 1
    for p in free[pages_left:]:
        refs[p] = 9
    b = Both(bsq, lens, table, refs, cache)
    b.fork([0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11])
    b = Both(bsq, lens, table, refs, cache)
    b.reserve([2, 0, 3, 1, 5, 4], [64, 63, 64, 130, 0, 200])


def test_requests_that_cannot_be(bsq):  # noqa: F811
    """Slots outside the table, negative lengths and growth, tables too short."""
    rng = np.random.default_rng(8)
    b = Both(bsq, *scene(rng, 3, 3, 30, 4, 256))
    b.reserve([-1, 3, 99, 4, 5], [5, 257, 3, -2, 256])
    b.fork([0, -3, 77, 1], [3, 4, 5, 6])
    b.free([-1, 6, 1, 1])                                    # named twice: freed once
    assert min(b.refs.tolist()) == 0
    b.fork([], [])
    b.reserve([], [])
    b.free([])


@pytest.mark.parametrize("n", [1025, 3000])
def test_more_requests_than_threads(bsq, n):  # noqa: F811
    rng = np.random.default_rng(n)
    lens, table, refs, cache = scene(rng, n, n, 2 * n + 50, 3, 70, 1, 64)
    b = Both(bsq, lens, table, refs, cache)
    b.fork(list(range(n)), [n + (7 * i) % n for i in range(n)] if n % 7 else list(range(n, 2 * n)))
    b.reserve([(11 * i) % (2 * n) for i in range(2 * n)], [int(x) for x in rng.integers(0, 60, 2 * n)])
    b.free(list(range(0, 2 * n, 3)))
    b.compact(True)


@pytest.mark.parametrize("pages", [1, 63, 4096, 4097, 20001])
def test_pools_of_many_sizes(bsq, pages):  # noqa: F811
    """The walk over the counts, a step of 4096 at a time; needs of many pages at once."""
    rng = np.random.default_rng(pages)
    refs = (rng.random(pages) < 0.6).astype(int)
    S, M = 6, max(2, pages // 3)
    table = np.zeros((S, M), int)
    cache = R.Cache(pages, 1, 64)
    cache.ks[:] = rng.integers(0, 255, cache.ks.shape)
    cache.k[:, 0, 0, 0, 0] = np.arange(pages) % 251
    b = Both(bsq, [0] * S, table, refs, cache)
    want = int((refs == 0).sum())
    b.reserve(list(range(S)), [64 * (want // 4) + 1, 0, 5, 64 * (want // 3), 64 * want, 1])
    b.free([0])
    b.compact(True)


def test_copy(bsq):  # noqa: F811
    rng = np.random.default_rng(4)
    for heads, D in ((1, 64), (5, 128)):
        c = random_cache(rng, 12, heads, D)
        d = dev_cache(bsq, c)
        src, dst = [3, 0, 11, 5, -1, 4, 12], [7, 1, 2, 5, 8, 99, 6]
        bsq.kv_pages_copy(d, i32(src), i32(dst))
        for s, t in zip(src, dst):
            if 0 <= s < 12 and 0 <= t < 12:
                for a in c.arrays():
                    a[t] = a[s]
        torch.cuda.synchronize()
        same_cache(d, c)


def test_copy_keeps_to_padded_pages(bsq):  # noqa: F811
    """Pages with gaps between them: the gaps' bytes stay."""
    k = torch.full((4, 64 * 64 + 48), 9, dtype=torch.uint8, device="cuda")
    v = torch.full((4, 64 * 64 + 48), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((4, 5), 9, dtype=torch.uint8, device="cuda")
    d = bsq.KvCache(k[:, :4096].unflatten(1, (1, 4, 64, 16)), v[:, :4096].unflatten(1, (1, 64, 64)),
                    s[:, 1:2], s[:, 3:4])
    for i, t in enumerate(d):
        t.copy_(torch.randint(0, 200, t.shape, dtype=torch.uint8, device="cuda") + i)
    bsq.kv_pages_copy(d, i32([2]), i32([1]))
    torch.cuda.synchronize()
    assert all(torch.equal(t[1], t[2]) for t in d)
    assert torch.all(k[:, 4096:] == 9) and torch.all(v[:, 4096:] == 9)
    assert torch.all(s[:, [0, 2, 4]] == 9)


def test_refusals(bsq):  # noqa: F811
    d = bsq.kv_cache(5, 1, 64)
    table, lens, refs = i32([[0, 1], [2, 3]]), i32([64, 3]), i32([1] * 5)
    with pytest.raises(bsq.BsqError):
        bsq.kv_pages_copy(d, i32([1, 2]), i32([3]))
    with pytest.raises(TypeError):
        bsq.kv_pages_copy(d, torch.zeros(1, device="cuda"), i32([3]))
    with pytest.raises(bsq.BsqError):
        bsq.kv_pages_fork(d, table, lens, refs[:4], i32([0]), i32([1]))
    with pytest.raises(bsq.BsqError):
        bsq.kv_pages_reserve(table, lens[:1], refs, i32([0]), i32([1]))
    with pytest.raises(TypeError):
        bsq.kv_pages_free(table.long(), lens, refs, i32([0]))
    with pytest.raises(bsq.BsqError):
        bsq.kv_pages_compact(d, table, lens, refs, table_out=table[:1])
    with pytest.raises(bsq.BsqError):
        bsq.kv_pages_compact(d, table, lens, refs,
                             workspace=torch.empty(32, dtype=torch.uint8, device="cuda"))
