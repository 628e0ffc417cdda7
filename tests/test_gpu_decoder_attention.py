"""Attention over the cache under masks of trees and sinks, on the GPU against the 64-bit
reference: every form of the kernels, rows that see nothing, pages that are not read."""
import numpy as np
import pytest
import torch

import decoder_ref as R
import serving_ref as S
from test_gpu_serving_kv import bsq, dev_cache, dev_rows, i32, make  # noqa: F401

pytestmark = pytest.mark.gpu


def call(bsq, c, q, off, lens, table, scale, window=0, sinks=0, masks=None, max_kv=None, dev=None,  # noqa: F811
         max_q=None, words=None, **kw):
    n = max_q or int(np.max(np.diff(np.asarray(off)), initial=0))
    if masks is not None:
        masks = torch.tensor(R.words(masks, words or (n + 63) // 64), device="cuda")
    return bsq.kv_cache_attention_masked(dev_rows(q), dev or dev_cache(bsq, c), i32(off), i32(lens),
                                         i32(table), n, int(max(lens)) if max_kv is None else max_kv,
                                         masks=masks, sinks=sinks, window=window, scale=scale,
                                         return_lse=True, **kw)


def check(bsq, c, q, off, lens, table, scale, window=0, sinks=0, masks=None, **kw):  # noqa: F811
    out, lse = call(bsq, c, q, off, lens, table, scale, window, sinks, masks, **kw)
    torch.cuda.synchronize()
    want, wlse, bo, bl, owned = R.attention(c, q, off, lens, table, scale, window, sinks, masks)
    o, z = out.double().cpu().numpy()[owned], lse.double().cpu().numpy()[owned]
    want, wlse, bo, bl = want[owned], wlse[owned], bo[owned], bl[owned]
    assert np.array_equal(np.isnan(o), np.isnan(want)) and np.array_equal(np.isnan(z), np.isnan(wlse))
    inf, ok = np.isinf(wlse), np.isfinite(wlse)
    assert np.array_equal(z[inf], wlse[inf])
    good = ~np.isnan(want)
    assert np.all(np.abs(o - want)[good] <= bo[good]), np.max((np.abs(o - want) / np.maximum(bo, 1e-300))[good & (bo > 0)])
    assert np.all(np.abs(z - wlse)[ok] <= bl[ok])
    return out, lse


def trees(seed, rows):
    rng = np.random.default_rng(seed)
    return [m for n in rows for m in R.random_tree(rng, n)]


# few columns, many columns (rows form) of both widths and every head width
FORMS = [(64, 2, 4), (128, 2, 8), (128, 1, 1), (256, 1, 4), (64, 3, 3), (128, 1, 7)]


@pytest.mark.parametrize("D,heads,hq", FORMS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 0), (70, 5), (3, 64), (200, 100), (64, 1000)])
def test_trees(bsq, D, heads, hq, window, sinks):  # noqa: F811
    rows = [1, 7, 33, 64, 2, 0]
    lens = [1, 300, 95, 64, 513, 12]
    c, q, off, table = make(D + hq, lens, rows, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5, window, sinks, trees(D + window, rows))


@pytest.mark.parametrize("D,heads,hq", FORMS)
@pytest.mark.parametrize("window,sinks", [(1, 1), (64, 4), (65, 63), (70, 64), (200, 65), (30, 1000),
                                          (5000, 7), (100, 0)])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1, 1], [5, 40, 3, 0, 2], [130, 2, 70, 64, 1]])
def test_sinks(bsq, D, heads, hq, window, sinks, rows):  # noqa: F811
    lens = [600, 129, 128, 64, 1]
    lens = [max(a, b) for a, b in zip(lens, rows)]
    c, q, off, table = make(D + sinks, lens, rows, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5, window, sinks)


@pytest.mark.parametrize("n", [63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("before", [0, 1, 37, 64, 100])
def test_trees_past_a_word(bsq, n, before):  # noqa: F811
    lens = [before + n, before + 3]
    c, q, off, table = make(n, lens, [n, 3], 1, 2, 64)
    check(bsq, c, q, off, lens, table, 0.125, 0, 0, trees(n + before, [n, 3]))
    check(bsq, c, q, off, lens, table, 0.125, 50, 3, trees(n + before, [n, 3]), words=9)


@pytest.mark.parametrize("heads,hq", [(2, 2), (1, 16)])
def test_chains_are_causal_attention(bsq, heads, hq):  # noqa: F811
    """A tree that is a chain is kv_cache_attention, with a window too; no masks at all are its
    kernels, bit for bit."""
    rows, lens = [1, 9, 40], [70, 300, 40]
    c, q, off, table = make(hq, lens, rows, heads, hq, 128)
    masks = [set(range(i + 1)) for n in rows for i in range(n)]
    d = dev_cache(bsq, c)
    for window in (0, 64, 150):
        a = call(bsq, c, q, off, lens, table, 0.1, window, 0, masks, dev=d)
        b = bsq.kv_cache_attention(dev_rows(q), d, i32(off), i32(lens), i32(table), 40, 300, scale=0.1,
                                   window=window, return_lse=True)
        s = call(bsq, c, q, off, lens, table, 0.1, window, 0, None, dev=d)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(s, b))
        assert torch.allclose(a[0].float(), b[0].float(), rtol=2 ** -7, atol=1e-3)
        check(bsq, c, q, off, lens, table, 0.1, window, 0, masks, dev=d)


def test_rows_that_see_little(bsq):  # noqa: F811
    """Empty masks, masks without the row itself, bits past the rows, all bits; with and without
    tokens before the rows, and more rows than tokens."""
    rows = [6, 6, 6, 70]
    lens = [6, 100, 3, 64]
    c, q, off, table = make(9, lens, rows, 2, 4, 64)
    rng = np.random.default_rng(4)
    masks = []
    for n in rows:
        for i in range(n):
            masks.append([set(), {0}, {n - 1}, set(range(128)), {i, n, n + 1, 127},
                          {int(x) for x in rng.integers(0, n, 3)}][i % 6])
    for window, sinks in ((0, 0), (4, 0), (4, 2), (1, 1), (90, 70)):
        out, lse = check(bsq, c, q, off, lens, table, 0.2, window, sinks, masks)
        assert bool((lse[0] == -float("inf")).all()) and not bool(out[0].any())


@pytest.mark.parametrize("tree", [False, True])
def test_nan_scales_reach_rows_that_see_them(bsq, tree):  # noqa: F811
    rows, lens = [3, 100], [400, 500]
    c, q, off, table = make(3, lens, rows, 2, 4, 64)
    c.ks[table[0][0], 0] = 255       # a page of sinks
    c.vs[table[1][2], 1] = 255       # in the gap: no row sees it
    c.vs[table[1][7], 0] = 255       # the rows' own page
    masks = trees(5, rows) if tree else None
    out, _ = check(bsq, c, q, off, lens, table, 0.125, 130, 10, masks)
    assert bool(out.isnan().any()) and not bool(out.isnan().all())
    check(bsq, c, q, off, lens, table, 0.125, 130, 0, masks)


def test_gap_is_not_read(bsq):  # noqa: F811
    """Pages and table entries between the sinks and the window may hold anything."""
    rows, lens = [1, 80, 1], [1000, 900, 70]
    c, q, off, table = make(8, lens, rows, 1, 4, 128)
    a = call(bsq, c, q, off, lens, table, 0.1, 100, 70)
    t2 = [list(r) for r in table]
    for p in range(2, 13):
        t2[0][p] = 10 ** 9
    for p in range(2, 11):
        t2[1][p] = -5
    b = call(bsq, c, q, off, lens, t2, 0.1, 100, 70)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("rows,D,heads,hq", [([1, 1], 128, 1, 8), ([20, 3], 64, 2, 2), ([100, 1], 128, 2, 4),
                                             ([60, 2], 256, 1, 2)])
@pytest.mark.parametrize("tree", [False, True])
def test_split_over_the_tokens(bsq, rows, D, heads, hq, tree):  # noqa: F811
    """Long sequences: runs of pages by several workgroups and their join, with the sinks in the
    first run; hints of the length that are wrong both ways."""
    lens = [9000, 260]
    c, q, off, table = make(D + hq, lens, rows, heads, hq, D)
    masks = trees(1, rows) if tree else None
    for window, sinks in ((0, 0), (6000, 100), (7000, 1)) if tree else ((6000, 100), (8000, 1)):
        for hint in (9000, 100, 200000):
            check(bsq, c, q, off, lens, table, D ** -0.5, window, sinks, masks, max_kv=hint)


@pytest.mark.parametrize("D,seqs,n,heads,hq", [
    (128, 33, 40, 16, 128),          # rows of 256 columns
    (128, 30, 20, 16, 128), (64, 33, 33, 16, 64), (256, 20, 33, 16, 64),   # rows of 128
    (128, 20, 9, 16, 64), (64, 65, 9, 4, 16), (128, 70, 5, 4, 20),         # blocks of 32 columns
    (128, 65, 3, 2, 12), (256, 30, 9, 8, 32)])                             # of 16
def test_forms_of_many_sequences(bsq, D, seqs, n, heads, hq):  # noqa: F811
    """Ragged lengths, equal ones among them, so that the longest-first order has ties."""
    rows = [n] * seqs
    lens = [n + 7 * (s * 13 % 17) for s in range(seqs)]
    c, q, off, table = make(2, lens, rows, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5, 0, 0, trees(3, rows))
    check(bsq, c, q, off, lens, table, D ** -0.5, 40, 4)


@pytest.mark.parametrize("D,heads,hq", [(128, 8, 32), (64, 8, 32)])
@pytest.mark.parametrize("seqs,n", [(64, 6), (48, 8), (32, 16)])
def test_batches_of_small_trees(bsq, D, heads, hq, seqs, n):  # noqa: F811
    """Blocks of 32 columns, fewer than 512; lengths in random order, some of one page
    or without tokens before the tree."""
    rows = [n - s % 3 for s in range(seqs)]
    lens = [r + (s * 37 % 23) * 13 for s, r in enumerate(rows)]
    c, q, off, table = make(5, lens, rows, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5, 0, 0, trees(4, rows))
    check(bsq, c, q, off, lens, table, D ** -0.5, 90, 5, trees(4, rows))
    check(bsq, c, q, off, lens, table, D ** -0.5, 40, 70)


@pytest.mark.parametrize("D,seqs,n,heads,hq", [(128, 65, 1, 8, 32), (64, 70, 1, 8, 16), (256, 80, 1, 8, 16),
                                               (128, 33, 2, 16, 64), (64, 33, 3, 16, 64)])
@pytest.mark.parametrize("longest", [300, 3300])
def test_batches_of_few_columns(bsq, D, seqs, n, heads, hq, longest):  # noqa: F811
    """One block of 16 columns a sequence and more workgroups than CUs: pages read past the caches,
    unsplit and in runs that a wave for each pair joins."""
    rows = [n] * seqs
    lens = [longest if s == 5 else n + (s * 29 % 31) * 11 for s in range(seqs)]
    c, q, off, table = make(6, lens, rows, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5, longest - 200, 70)
    check(bsq, c, q, off, lens, table, D ** -0.5, 100, 4)
    check(bsq, c, q, off, lens, table, D ** -0.5, 0, 0, trees(7, rows))


@pytest.mark.parametrize("D,n,heads,hq", [(64, 100, 2, 4), (64, 40, 2, 4), (256, 100, 2, 4)])
def test_few_columns_of_many_pages(bsq, D, n, heads, hq):  # noqa: F811
    """The form of many rows, its pages in runs of several workgroups."""
    rows, lens = [n, 3], [9990, 70]
    c, q, off, table = make(8, lens, rows, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5, 0, 0, trees(9, rows))
    check(bsq, c, q, off, lens, table, D ** -0.5, 9700, 70)


@pytest.mark.parametrize("window", [1 << 31, (1 << 31) + 64, 1 << 40, (1 << 63) - 1])
@pytest.mark.parametrize("D,seqs,n,heads,hq", [
    (128, 64, 8, 8, 32), (128, 64, 5, 8, 32), (128, 16, 48, 8, 32), (64, 65, 9, 4, 16),   # blocks of 32 columns
    (256, 30, 9, 8, 32), (128, 2, 9, 2, 8), (64, 2, 1, 2, 8), (128, 2, 100, 2, 8)])
def test_windows_longer_than_any_sequence(bsq, D, seqs, n, heads, hq, window):  # noqa: F811
    """A window past 2^31 - 1 is none: every token is seen, the sinks among them, and the call is
    kv_cache_attention's, bit for bit."""
    rows, lens = [n] * seqs, [n + 7 * (s * 13 % 17) for s in range(seqs)]
    c, q, off, table = make(2, lens, rows, heads, hq, D)
    d = dev_cache(bsq, c)
    want = bsq.kv_cache_attention(dev_rows(q), d, i32(off), i32(lens), i32(table), n, max(lens), scale=0.1,
                                  return_lse=True)
    out, lse = torch.full_like(want[0], 5.0), torch.full_like(want[1], 5.0)
    call(bsq, c, q, off, lens, table, 0.1, window, 4, dev=d, out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("rows", [[1, 1], [9, 3], [100, 2]])
@pytest.mark.parametrize("tree", [False, True])
def test_tables_that_end_before_the_sequence(bsq, rows, tree):  # noqa: F811
    """Tokens past the table's pages are not seen; the sinks are, also where the whole window is past
    them."""
    lens = [700, 300]
    c, q, off, table = make(4, lens, rows, 2, 4, 64)
    masks = trees(2, rows) if tree else None
    for width in (1, 2, 4, 8):
        cut = [r[:width] for r in table]
        for window, sinks in ((90, 70), (90, 500), (400, 3), (90, 0)):
            check(bsq, c, q, off, lens, cut, 0.125, window, sinks, masks)


def test_rows_past_max_q_and_unowned_rows_are_left(bsq):  # noqa: F811
    rows, lens = [5, 9], [50, 70]
    c, q, off, table = make(1, lens, rows, 1, 2, 64)
    q = np.concatenate([q, q[:3]])
    masks = trees(1, rows) + [set()] * 3
    out = torch.full((17, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((17, 2), 5.0, device="cuda")
    call(bsq, c, q, off, lens, table, 0.1, masks=masks, max_q=6, words=1, out=out, lse=lse)
    want, _ = call(bsq, c, q, off, lens, table, 0.1, masks=masks)
    torch.cuda.synchronize()
    assert torch.equal(out[:11], want[:11]) and bool((out[11:] == 5).all()) and bool((lse[11:] == 5).all())


def test_refusals_of_the_binding(bsq):  # noqa: F811
    rows, lens = [3], [50]
    c, q, off, table = make(1, lens, rows, 1, 2, 64)
    d, qd = dev_cache(bsq, c), dev_rows(q)
    m = torch.ones((3, 1), dtype=torch.int64, device="cuda")

    def go(**kw):
        a = dict(masks=m, max_q=3, sinks=0, window=0)
        a.update(kw)
        return bsq.kv_cache_attention_masked(qd, d, i32(off), i32(lens), i32(table), a.pop("max_q"), 50, **a)
    go()
    go(masks=m.view(torch.uint64))
    for err, kw in [(TypeError, dict(masks=m.int())), (TypeError, dict(masks=m[:, 0])),
                    (TypeError, dict(masks=m.cpu())), (TypeError, dict(masks=m.repeat(1, 2)[:, ::2])),
                    (bsq.BsqError, dict(masks=m[:2])), (bsq.BsqError, dict(max_q=65)),
                    (bsq.BsqError, dict(masks=m[:, :0])), (bsq.BsqError, dict(sinks=-1)),
                    (bsq.BsqError, dict(sinks=1 << 31)), (bsq.BsqError, dict(window=-1))]:
        with pytest.raises(err):
            go(**kw)
