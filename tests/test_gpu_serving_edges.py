"""Edges of the serving operators: pages without a number in their scale beside far smaller ones,
numbers at the ends of their range, rows past the host-side bounds,
more pages asked for than there are numbers."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_serving_kv import (attend, bsq, check, deal, dev_cache, dev_rows, i32,  # noqa: F401
                                 make, random_cache, same_cache)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention


@pytest.mark.parametrize("D,heads", [(64, 1), (128, 2), (256, 1)])
@pytest.mark.parametrize("vs", [7, 27, 60])
@pytest.mark.parametrize("rows,L,window", [(2, 664, 600), (130, 330, 200)])
def test_nan_page_that_a_row_does_not_see(bsq, D, heads, vs, rows, L, window):  # noqa: F811
    """The first page has the NaN scale and the window of the later rows starts past it; V's
    other scales are 2^-120 to 2^-67: those rows keep every bit of V.  664 tokens: the wave that
    meets the NaN page has another page after it."""
    c, q, off, table = make(D + vs, [L], [rows], heads, 2 * heads, D)
    c.vs[:] = vs
    c.vs[table[0][0]] = 255
    out = check(bsq, c, q, off, [L], table, D ** -0.5, window)
    assert np.isnan(out).any() and np.isfinite(out).any()


@pytest.mark.parametrize("rows", [10, 80])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1])
def test_windows_longer_than_any_sequence(bsq, rows, window):  # noqa: F811
    """As no window, also where a sequence has rows before its first token."""
    lens = [rows - 7, 300, 3]
    c, q, off, table = make(rows, [rows, 300, rows], [rows] * 3, 2, 4, 64)
    got = attend(bsq, c, q, off, lens, table, 0.1, window)
    want = attend(bsq, c, q, off, lens, table, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(want[1][7:rows]).all()


# ------------------------------------------------------------------ experts


@pytest.mark.parametrize("T", [1, 3, 20])
def test_hidden_values_past_the_bf16_range(bsq, T):  # noqa: F811
    """A gated value between the largest BF16 number and the largest fp32 one stays that number,
    and one past fp32 is infinite, not NaN."""
    from test_gpu_serving_moe import Layer, check as close

    E, H, I = 2, 128, 128
    L = Layer(0, E, H, I, "mxfp8")
    for name, n, k in (("w13", 2 * I, H), ("w2", H, I)):
        codes, scales = L.host[name][:2]
        codes[:] = 0
        scales[:] = 127
    one = int(R.to_e4m3(1.0))
    codes, scales = L.host["w13"][:2]
    # W1 row: 2^64 x0; W3 row: 2^64 (x0 + x1)
    for e in range(E):
        codes[e * 2 * I:e * 2 * I + 2 * I, 0] = one
        codes[e * 2 * I + I:e * 2 * I + 2 * I, 1] = one
    scales[:] = 127 + 64
    codes, scales = L.host["w2"][:2]
    codes[:] = one
    scales[:] = 127 - 100
    x = np.zeros((T, H))
    x[:, 0] = 1.0
    x[:, 1] = -2.0 ** -11                                    # h = 2^128 - 2^117, BF16 ends at 2^128 - 2^120
    ids, w = np.zeros((T, 1), np.int32), np.full((T, 1), 0.5, np.float32)

    def run():
        return bsq.moe_few_tokens(dev_rows(x), "mxfp8", *L.dev(), E, 1, topk_ids=i32(ids),
                                  topk_weights=torch.from_numpy(w).cuda())[0]
    y = run()
    torch.cuda.synchronize()
    close(y, *L.reference(x, ids, w))
    assert abs(float(y[0, 0]) / (2.0 ** 34 * (1 - 2.0 ** -11)) - 1) <= 2.0 ** -8
    x[:, 1] = 1.0                                            # h = 2^129
    y = run()
    torch.cuda.synchronize()
    assert torch.all(y == np.inf)


# ------------------------------------------------------------------ host-side bounds


@pytest.mark.parametrize("most", [1, 2, 5, 6, 40, 64, 70])
def test_append_stops_at_its_bound(bsq, most):  # noqa: F811
    """Rows of a sequence past max_new are not written and have no part in a scale."""
    rng = np.random.default_rng(most)
    heads, D, olds, news = 2, 64, [0, 3, 62, 130, 64], [1, 9, 7, 200, 64]
    lens = [a + b for a, b in zip(olds, news)]
    pages, width = sum(R.pages_of(n) for n in lens) + 2, max(R.pages_of(n) for n in lens)
    c = random_cache(rng, pages, heads, D)
    table = deal(rng, lens, pages, width)
    off = np.concatenate([[0], np.cumsum(news)])
    x = R.bf16(rng.standard_normal((off[-1], heads, D)) * 2.0 ** np.arange(off[-1] // 9 + 1).repeat(9)
               [:off[-1], None, None] * 2.0 ** -20)
    d = dev_cache(bsq, c)
    bsq.kv_cache_append(d, dev_rows(x), dev_rows(-x), i32(off), i32(lens), i32(table), most)
    for s, n in enumerate(news):
        m = min(n, most)
        rows = slice(off[s], off[s] + m)
        R.append(c, x[rows], -x[rows], [0, m], [olds[s] + m], [table[s]])
    torch.cuda.synchronize()
    same_cache(d, c)


@pytest.mark.parametrize("D,hq,heads", [(64, 4, 2), (128, 4, 2), (256, 2, 1)])
@pytest.mark.parametrize("most,lens", [(1, [300, 70, 9]), (3, [300, 70, 9]), (2, [3000, 200, 9]),
                                       (70, [400, 150, 9]), (100, [400, 150, 9]), (90, [4000, 150, 9]), (100, [200, 150, 9]), (3, [140, 70, 9])])
def test_attention_stops_at_its_bound(bsq, D, hq, heads, most, lens):  # noqa: F811
    """Rows of a sequence past max_q keep what out and lse held, and the others their places."""
    rows = [130, 40, 5]
    c, q, off, table = make(D + most, lens, rows, heads, hq, D)
    out = torch.full((off[-1], hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((off[-1], hq), 5.0, device="cuda")
    attend(bsq, c, q, off, lens, table, 0.1, max_q=most, out=out, lse=lse)
    torch.cuda.synchronize()
    want, wlse, bo, bl, _ = R.attention(c, q, off, lens, table, 0.1)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for s, n in enumerate(rows):
        done, left = slice(off[s], off[s] + min(n, most)), slice(off[s] + min(n, most), off[s + 1])
        assert np.all(np.abs(out[done] - want[done]) <= bo[done])
        assert np.all(np.abs(lse[done] - wlse[done]) <= bl[done])
        assert np.all(out[left] == 7) and np.all(lse[left] == 5), s


# ------------------------------------------------------------------ pages


@pytest.mark.parametrize("n,width", [(70, 2 ** 25 - 1), (1030, 2 ** 21)])
def test_needs_past_32_bits(bsq, n, width):  # noqa: F811
    """Requests whose needs add up to more than 2^31 pages: those that were served before the pages
    ended have them, the others fail and change neither lengths nor counts."""
    pages = 40
    table = torch.empty((n, width), dtype=torch.int32, device="cuda")      # 9 GB, hardly touched
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    add = [64 * width if width < 2 ** 25 else 2 ** 31 - 64] * n
    add[0], add[1], add[-1] = 130, 1, 64
    status = bsq.kv_pages_reserve(table, lens, refs, i32(np.arange(n)), i32(add))
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0] + [1] * (n - 2)
    assert lens.tolist() == [130, 1] + [0] * (n - 2)
    assert refs.tolist() == [1] * 4 + [0] * (pages - 4)
    assert table[0, :3].tolist() == [0, 1, 2] and table[1, 0].item() == 3


@pytest.mark.parametrize("kept", [64, 70, 128, 129, 150])
def test_tokens_taken_back(bsq, kept):  # noqa: F811
    """A sequence is shortened as the header says: the pages given up are given out again, and
    what is appended then is what a sequence holds that never had the other tokens."""
    rng = np.random.default_rng(kept)
    L, D, more = 150, 64, 90
    x = R.bf16(rng.standard_normal((L, 1, D)))
    y = R.bf16(rng.standard_normal((more, 1, D)))
    y[0] = 7.9                                               # no smaller scale than x's
    d, c = bsq.kv_cache(6, 1, D), R.Cache(6, 1, D)
    table, lens = torch.full((2, 6), -1, dtype=torch.int32, device="cuda"), i32([0, 0])
    refs = i32([0] * 6)

    def reserve(slot, n):
        assert bsq.kv_pages_reserve(table, lens, refs, i32([slot]), i32([n])).tolist() == [0]
    reserve(0, L)
    bsq.kv_cache_append(d, dev_rows(x), dev_rows(x), i32([0, L, L]), lens, table, L)
    up = table[0, -(-kept // 64):-(-L // 64)].long()
    refs[up] -= 1
    lens[0] = kept
    reserve(1, 64)                                           # a page given up, where there is one
    reserve(0, more)
    bsq.kv_cache_append(d, dev_rows(y), dev_rows(y), i32([0, more, more]), lens, table, more)
    torch.cuda.synchronize()
    rows = [table[0].tolist()]
    R.append(c, x[:kept], x[:kept], [0, kept], [kept], rows)
    R.append(c, y, y, [0, more], [kept + more], rows)
    assert lens.tolist() == [kept + more, 64]
    assert refs.tolist() == [1] * (-(-(kept + more) // 64) + 1) + [0] * (5 - -(-(kept + more) // 64))
    got = [t.cpu().numpy() for t in d]
    for p in range(-(-(kept + more) // 64)):
        page, n = rows[0][p], min(64, kept + more - 64 * p)
        assert np.array_equal(got[0][page, 0, :, :n], c.k[page, 0, :, :n])
        assert np.array_equal(got[1][page, 0][:, R.v_place(np.arange(n))], c.v[page, 0][:, R.v_place(np.arange(n))])
        assert got[2][page, 0] == c.ks[page, 0] and got[3][page, 0] == c.vs[page, 0]
