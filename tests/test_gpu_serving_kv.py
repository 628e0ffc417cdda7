"""The 8-bit cache's append and attention on the GPU against the 64-bit reference: bytes for
the append, the summed rounding bounds of serving_ref for the attention."""
import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_amd as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device="cuda")


def dev_cache(bsq, c):
    return bsq.KvCache(*(torch.from_numpy(a.copy()).cuda() for a in c.arrays()))


def dev_rows(x):
    return torch.tensor(x).to(torch.bfloat16).cuda()


def same_cache(dev, ref):
    for name, d, r in zip(("k", "v", "k scales", "v scales"), dev, ref.arrays()):
        assert np.array_equal(d.cpu().numpy(), r), name


def random_cache(rng, pages, heads, D, scale_spread=3):
    """Every byte set: codes without NaN, scales around 2^-7."""
    c = R.Cache(pages, heads, D)
    for a in (c.k, c.v):
        a[:] = R.to_e4m3(rng.standard_normal(a.shape) * 60)
    for a in (c.ks, c.vs):
        a[:] = rng.integers(119, 119 + scale_spread, a.shape)
    return c


def deal(rng, lens, pages, width):
    order = list(rng.permutation(pages))
    return [[int(order.pop()) if k < R.pages_of(n) else int(rng.integers(-9, pages + 9))
             for k in range(width)] for n in lens]


# ------------------------------------------------------------------ append


@pytest.mark.parametrize("D,heads", [(64, 1), (64, 5), (128, 2), (256, 3)])
@pytest.mark.parametrize("olds,news", [
    ([0, 63, 64, 65], [1, 1, 1, 1]), ([0, 1, 62, 127], [5, 5, 5, 5]), ([10, 0, 3, 60], [0, 2, 4, 3]),
    ([0, 0, 7, 130], [64, 128, 200, 63]), ([33, 0, 64, 1], [31, 6, 7, 300])])
def test_append_bytes(bsq, D, heads, olds, news):
    rng = np.random.default_rng(D + heads + sum(olds) + 7 * sum(news))
    lens = [a + b for a, b in zip(olds, news)]
    pages, width = sum(R.pages_of(n) for n in lens) + 4, max(R.pages_of(n) for n in lens) + 1
    c = R.Cache(pages, heads, D, fill=0xFF)          # what no one wrote may be anything
    table = deal(rng, lens, pages, width)
    off0 = np.concatenate([[0], np.cumsum(olds)])
    off1 = np.concatenate([[0], np.cumsum(news)])
    spread = np.exp2(rng.integers(-6, 7, (off0[-1], 1, 1)))
    k0, v0 = (R.bf16(rng.standard_normal((off0[-1], heads, D)) * spread) for _ in range(2))
    # the second call's tokens are larger in some heads: those pages' old codes move
    grow = np.exp2(rng.integers(-8, 9, (1, heads, 1)))
    k1, v1 = (R.bf16(rng.standard_normal((off1[-1], heads, D)) * grow) for _ in range(2))
    d = dev_cache(bsq, c)
    for k, v, off, ln in ((k0, v0, off0, olds), (k1, v1, off1, lens)):
        n = int(max(np.diff(off), default=0))
        kv = torch.stack([dev_rows(k), dev_rows(v)], 1)          # slices of one projection
        bsq.kv_cache_append(d, kv[:, 0], kv[:, 1], i32(off), i32(ln), i32(table), n)
        R.append(c, k, v, off, ln, table)
        torch.cuda.synchronize()
        same_cache(d, c)


def test_append_special_values(bsq):
    """NaN and Inf poison their (page, head) alone, now and for tokens to come; zeros,
    subnormals and the largest numbers keep the rule's bytes; signs of zero stay."""
    rng = np.random.default_rng(5)
    heads, D = 6, 64
    x = rng.standard_normal((70, heads, D))
    x[:, 1] = 0.0
    x[::2, 1] = -0.0
    x[:, 2] *= 2.0 ** -130
    x[:, 3] *= 2.0 ** 126
    x[3, 4, 5] = np.nan
    x[66, 5, 0] = np.inf
    x[10:12, 0] = [[448 * 2.0 ** 3] * D, [1.0] * D]
    x = R.bf16(x)
    c = R.Cache(3, heads, D)
    table = [[2, 0]]
    d = dev_cache(bsq, c)
    for lo, hi in ((0, 68), (68, 70)):
        bsq.kv_cache_append(d, dev_rows(x[lo:hi]), dev_rows(x[lo:hi]), i32([0, hi - lo]), i32([hi]),
                            i32(table), hi - lo)
        R.append(c, x[lo:hi], x[lo:hi], [0, hi - lo], [hi], table)
    torch.cuda.synchronize()
    assert c.ks[2, 4] == 255 and c.ks[0, 4] != 255 and c.ks[0, 5] == 255 and c.ks[2, 1] == 0
    same_cache(d, c)


def test_append_skips_what_it_cannot_place(bsq):
    """Pages outside the cache or the table, more rows than tokens, offsets that run backwards
    or past the rows: skipped, the rest written."""
    rng = np.random.default_rng(6)
    heads, D = 2, 128
    x = R.bf16(rng.standard_normal((90, heads, D)))
    c = random_cache(rng, 6, heads, D)
    table = [[-1, 2], [5, 77], [0, 1], [3, 4]]
    offsets, lens = [0, 70, 80, 90, 90], [70, 66, 4, 30]
    d = dev_cache(bsq, c)
    bsq.kv_cache_append(d, dev_rows(x), dev_rows(x), i32(offsets), i32(lens), i32(table), 70)
    R.append(c, x, x, offsets, lens, table)
    torch.cuda.synchronize()
    same_cache(d, c)
    # offsets past the rows and backwards
    bsq.kv_cache_append(d, dev_rows(x), dev_rows(x), i32([0, 91, 80, 70, 70]), i32([91, 66, 9, 9]),
                        i32(table), 70)
    torch.cuda.synchronize()
    same_cache(d, c)


# ------------------------------------------------------------------ attention


def attend(bsq, c, q, offsets, lens, table, scale, window=0, max_kv=None, dev=None, max_q=None,
           **kw):
    n = max_q or int(np.max(np.diff(np.asarray(offsets)), initial=0))
    return bsq.kv_cache_attention(dev_rows(q), dev or dev_cache(bsq, c), i32(offsets), i32(lens),
                                  i32(table), n, int(max(lens)) if max_kv is None else max_kv,
                                  scale=scale, window=window, return_lse=True, **kw)


def check(bsq, c, q, offsets, lens, table, scale, window=0, **kw):
    out, lse = attend(bsq, c, q, offsets, lens, table, scale, window, **kw)
    torch.cuda.synchronize()
    want, wlse, bo, bl, owned = R.attention(c, q, offsets, lens, table, scale, window)
    out, lse = out.double().cpu().numpy()[owned], lse.double().cpu().numpy()[owned]
    want, wlse, bo, bl = want[owned], wlse[owned], bo[owned], bl[owned]
    assert np.array_equal(np.isnan(out), np.isnan(want))
    assert np.array_equal(np.isnan(lse), np.isnan(wlse))
    fine = np.isfinite(wlse)
    assert np.array_equal(lse[~fine & ~np.isnan(wlse)], wlse[~fine & ~np.isnan(wlse)])
    ok = ~np.isnan(want)
    worst = np.max((np.abs(out - want) / np.maximum(bo, 1e-300))[ok & (bo > 0)], initial=0)
    assert np.all(np.abs(out - want)[ok] <= bo[ok]), worst
    assert np.all(np.abs(lse - wlse)[fine] <= bl[fine])
    return out


def make(seed, lens, rows, heads, hq, D, extra_pages=3):
    rng = np.random.default_rng(seed)
    pages, width = sum(R.pages_of(n) for n in lens) + extra_pages, max(R.pages_of(n) for n in lens) + 2
    c = random_cache(rng, pages, heads, D)
    # whatever lies past a sequence's end, NaN codes too
    table = deal(rng, lens, pages, width)
    for s, n in enumerate(lens):
        if n % 64:
            page = table[s][n // 64]
            t = np.arange(n % 64, 64)
            c.k[page][:, :, t] = 0x7F
            c.v[page][:, :, R.v_place(t)] = 0xFF
    offsets = np.concatenate([[0], np.cumsum(rows)])
    return c, R.bf16(rng.standard_normal((offsets[-1], hq, D))), offsets, table


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,hq", [(1, 1), (2, 8), (3, 3), (2, 14), (1, 17)])
def test_single_tokens(bsq, D, heads, hq):
    lens = [1, 63, 64, 65, 300]
    c, q, off, table = make(D + hq, lens, [1] * 5, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [[2, 7, 3], [16, 1, 5]])
def test_a_few_rows(bsq, D, rows):
    """Up to 64 (row, head) columns a head: several blocks of 16."""
    lens = [2, 200, 129]
    lens = [max(a, b) for a, b in zip(lens, rows)]
    c, q, off, table = make(D + rows[0], lens, rows, 2, 8, D)
    check(bsq, c, q, off, lens, table, D ** -0.5)


@pytest.mark.parametrize("D,hq,heads", [(64, 4, 4), (128, 6, 2), (256, 2, 1), (128, 7, 1)])
@pytest.mark.parametrize("window", [0, 1, 63, 64, 65, 150])
def test_many_rows(bsq, D, hq, heads, window):
    rows, lens = [130, 0, 1, 77], [130, 64, 1, 333]
    c, q, off, table = make(D + hq, lens, rows, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5, window)


@pytest.mark.parametrize("window", [1, 2, 64, 100, 5000])
@pytest.mark.parametrize("D", [64, 128])
def test_window_of_single_tokens(bsq, D, window):
    """Pages before the window need not be in the table any more."""
    lens = [700, 64, 65, 5]
    c, q, off, table = make(window, lens, [1, 1, 2, 1], 2, 4, D)
    for p in range((700 - window) // 64 if window < 700 else 0):
        table[0][p] = -1
    check(bsq, c, q, off, lens, table, D ** -0.5, window)


@pytest.mark.parametrize("rows", [1, 100])
def test_rows_that_see_nothing(bsq, rows):
    """No tokens, more rows than tokens, no page that the cache has: zeros and -inf."""
    D, lens = 128, [0, 3, 70, 64]
    n = [rows, rows + 3, rows, 0]
    c, q, off, table = make(rows, [64, 64, 128, 64], n, 2, 4, D)
    table[2] = [-1, c.ks.shape[0]] + table[2][2:]
    out = check(bsq, c, q, off, lens, table, D ** -0.5)
    assert np.all(out[:rows] == 0)


@pytest.mark.parametrize("rows,kv", [(1, 3000), (2, 9000), (3, 20001)])
def test_split_over_the_tokens(bsq, rows, kv):
    D, lens = 64, [kv, 40, 2600]
    c, q, off, table = make(kv, lens, [rows] * 3, 1, 2, D)
    check(bsq, c, q, off, lens, table, D ** -0.5)
    # a bound on the lengths that is too low, or far too high, changes the split alone
    check(bsq, c, q, off, lens, table, D ** -0.5, max_kv=2700)
    check(bsq, c, q, off, lens, table, D ** -0.5, max_kv=70000)
    check(bsq, c, q, off, lens, table, D ** -0.5, max_kv=1)
    check(bsq, c, q, off, lens, table, D ** -0.5, window=2777)


@pytest.mark.parametrize("hq,heads", [(2, 2), (7, 1), (6, 2)])
@pytest.mark.parametrize("window", [0, 100])
def test_many_rows_in_wide_workgroups(bsq, hq, heads, window):
    """head_dim 128 takes 256 columns a workgroup where a call may have 512 of them: so does a
    loose bound on the rows.  NaN scales there as well."""
    rows, lens = [300, 1, 0, 257], [300, 200, 70, 501]
    c, q, off, table = make(hq, lens, rows, heads, hq, 128)
    check(bsq, c, q, off, lens, table, 128 ** -0.5, window, max_q=512 * 256 // heads)
    c.ks[table[0][4], 0] = 255
    c.vs[table[3][7], heads - 1] = 255
    check(bsq, c, q, off, lens, table, 128 ** -0.5, window, max_q=512 * 256 // heads)


def test_more_than_64_splits(bsq):
    D, lens = 64, [75000, 64 * 16 * 65 + 1]
    c, q, off, table = make(5, lens, [1, 2], 1, 2, D)
    check(bsq, c, q, off, lens, table, D ** -0.5)


@pytest.mark.parametrize("D,hq,heads", [(64, 4, 2), (128, 2, 1), (256, 6, 1)])
@pytest.mark.parametrize("rows", [70, 300])
def test_many_rows_split_over_the_tokens(bsq, D, hq, heads, rows):
    """Too few rows for every CU: their pages are split too.  Up to and over 1024 pairs of a
    row and a head, which are joined by four waves and by one."""
    lens, n = [2500, 40, 1030], [rows, 3, rows - 5]
    c, q, off, table = make(D + rows, lens, n, heads, hq, D)
    check(bsq, c, q, off, lens, table, D ** -0.5)
    check(bsq, c, q, off, lens, table, D ** -0.5, max_kv=600)
    check(bsq, c, q, off, lens, table, D ** -0.5, max_kv=20000)
    check(bsq, c, q, off, lens, table, D ** -0.5, window=1111)


@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0, 1e-30])
def test_scales_of_the_scores(bsq, rows, scale):
    lens = [200, 90]
    c, q, off, table = make(3, lens, [rows, 90 if rows > 1 else 1], 2, 4, 128)
    check(bsq, c, q, off, lens, table, scale)


@pytest.mark.parametrize("rows", [1, 90])
def test_page_scales_far_apart(bsq, rows):
    """V scales from 2^-120 to 2^60 in one sequence, K scales over 2^30: the sums hold in
    units that follow them."""
    rng = np.random.default_rng(9)
    lens = [64 * 8 - 5, 64 * 3]
    c, q, off, table = make(4, lens, [rows, rows], 1, 2, 128)
    c.vs[:] = rng.integers(7, 188, c.vs.shape)
    c.ks[:] = rng.integers(90, 121, c.ks.shape)
    check(bsq, c, q, off, lens, table, 128 ** -0.5)
    # every page of a sequence but one empty of magnitude
    c.vs[:] = 0
    c.vs[table[0][3]] = 127
    check(bsq, c, q, off, lens, table, 128 ** -0.5)


@pytest.mark.parametrize("rows", [1, 100])
def test_one_token_takes_all_the_weight(bsq, rows):
    """Scores hundreds apart, the largest first, last or in between."""
    lens = [300, 300, 300]
    c, q, off, table = make(11, lens, [rows] * 3, 1, 1, 64)
    for s, t in enumerate((0, 150, 299)):
        page, u = table[s][t // 64], t % 64
        c.ks[page] = 125
        c.set_codes("k", page, 0, u, R.to_e4m3(np.full(64, 400.0)))
    q = R.bf16(np.abs(q) * 3)
    check(bsq, c, q, off, lens, table, 0.125)


@pytest.mark.parametrize("rows", [1, 100])
def test_nan_scales_reach_the_rows_that_see_them(bsq, rows):
    """A NaN scale of K or V makes NaN of the rows that see its page, and of none before it or
    with a window past it; rows of other heads and sequences stay."""
    lens = [300, 200, 210]
    c, q, off, table = make(12, lens, [rows] * 3, 2, 4, 128)
    c.ks[table[0][4], 0] = 255                        # tokens 256 .. 299
    c.vs[table[1][0], 1] = 255
    check(bsq, c, q, off, lens, table, 0.1)
    check(bsq, c, q, off, lens, table, 0.1, window=30)


def test_strides_output_and_streams(bsq):
    """K and V pages in one allocation, a padded table, q and out as slices, lse given, another
    stream; rows that no sequence owns and columns beside out stay as they were."""
    lens, rows = [150, 9, 500], [1, 2, 1]
    c, q, off, table = make(21, lens, rows, 2, 4, 64)
    P = c.ks.shape[0]
    flat = 2 * 64 * 64
    both = torch.full((P, 2 * flat + 64), 0xFF, dtype=torch.uint8, device="cuda")
    k = both[:, :flat].unflatten(1, (2, 4, 64, 16))
    v = both[:, flat + 32:2 * flat + 32].unflatten(1, (2, 64, 64))
    sc = torch.full((P, 7), 0xFF, dtype=torch.uint8, device="cuda")
    d = bsq.KvCache(k, v, sc[:, 1:3], sc[:, 4:6])
    for x, a in zip(d, c.arrays()):
        x.copy_(torch.from_numpy(a))
    M = len(table[0])
    wide = torch.full((3, M + 5), -3, dtype=torch.int32, device="cuda")
    wide[:, :M] = i32(table)
    qkv = torch.full((5, 9, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qkv[:4, 2:6] = dev_rows(q)
    big = torch.full((6, 10, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 4), 5.0, device="cuda")
    want, _, bo, _, _ = R.attention(c, q, off, lens, table, 0.2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bsq.kv_cache_attention(qkv[:, 2:6], d, i32(off), i32(lens), wide[:, :M], 2, 500, scale=0.2,
                           out=big[:5, 3:7], lse=lse, stream=side)
    with torch.cuda.stream(side):
        again = bsq.kv_cache_attention(qkv[:, 2:6], d, i32(off), i32(lens), wide[:, :M], 2, 500, scale=0.2)
    torch.cuda.synchronize()
    got = big[:4, 3:7].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= bo) and torch.equal(again[:4], big[:4, 3:7])
    assert torch.all(big[4:] == 3) and torch.all(big[:, :3] == 3) and torch.all(big[:, 7:] == 3)
    assert torch.all(lse[4] == 5) and torch.all(torch.isfinite(lse))


def test_same_bits_again(bsq):
    """The order of every sum is fixed."""
    for rows, kv in ((1, 9000), (1, 300), (150, 700)):
        lens = [kv, kv // 2]
        c, q, off, table = make(kv, lens, [rows] * 2, 2, 8, 128)
        d = dev_cache(bsq, c)
        a = attend(bsq, c, q, off, lens, table, 0.1, dev=d)
        for _ in range(3):
            b = attend(bsq, c, q, off, lens, table, 0.1, dev=d)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("rows", [1, 40])
def test_offsets_past_32_bits(bsq, rows):
    """Pages whose codes lie past 4 GiB: append there, attend, copy away and attend again."""
    heads, D = 8, 128
    P = (1 << 32) // (heads * D * 64) + 20
    d = bsq.kv_cache(P, heads, D)
    rng = np.random.default_rng(2)
    L = 130
    x, y, q = (R.bf16(rng.standard_normal((n, h, D))) for n, h in ((L, heads), (L, heads), (rows, heads)))
    table = [[P - 1, P - 3, P - 2]]
    bsq.kv_cache_append(d, dev_rows(x), dev_rows(y), i32([0, L]), i32([L]), i32(table), L)
    small, near = R.Cache(3, heads, D), [[2, 0, 1]]
    R.append(small, x, y, [0, L], [L], near)
    out = attend(bsq, None, q, [0, rows], [L], table, 0.09, dev=d)[0]
    bsq.kv_pages_copy(d, i32([P - 1, P - 3, P - 2]), i32([2, 0, 1]))
    moved = attend(bsq, None, q, [0, rows], [L], near, 0.09, dev=d)[0]
    torch.cuda.synchronize()
    want, _, bo, _, _ = R.attention(small, q, [0, rows], [L], near, 0.09)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bo)
    assert torch.equal(out, moved)
    t = np.arange(64)
    assert np.array_equal(d.k_codes[2].cpu().numpy(), small.k[2])
    assert np.array_equal(d.v_codes[0].cpu().numpy()[:, :, R.v_place(t)], small.v[0][:, :, R.v_place(t)])


def test_refusals_on_the_gpu(bsq):
    d = bsq.kv_cache(3, 2, 64)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    off, lens, table = i32([0, 1, 2]), i32([3, 4]), i32([[0, 1], [2, 1]])
    with pytest.raises(TypeError):
        bsq.kv_cache_attention(q.float(), d, off, lens, table, 1, 4)
    with pytest.raises(TypeError):
        bsq.kv_cache_attention(q.transpose(0, 1), d, off, lens, table, 1, 4)
    with pytest.raises(TypeError):
        bsq.kv_cache_attention(q, d, off, lens, table.t(), 1, 4)
    with pytest.raises(bsq.BsqError):
        bsq.kv_cache_attention(q[:, :3], d, off, lens, table, 1, 4)
    with pytest.raises(bsq.BsqError):
        bsq.kv_cache_attention(q, d, off[:2], lens, table, 1, 4)
    with pytest.raises(bsq.BsqError):
        bsq.kv_cache_attention(q, d, off, lens, table, 1, 4, window=-1)
    with pytest.raises(bsq.BsqError):
        bsq.kv_cache_attention(q, d, off, lens, table, 1, 4, out=q[:1])
    with pytest.raises(bsq.BsqError):
        bsq.kv_cache_attention(q, d._replace(v_codes=d.v_codes[:2]), off, lens, table, 1, 4)
    with pytest.raises(bsq.BsqError):
        bsq.kv_cache_append(d, q, q, off, lens, table, 1)        # four heads for a cache of two
    with pytest.raises(bsq.BsqError):
        bsq.kv_cache_attention(q.repeat(1, 1, 1), d, off, lens, table, 1, 100000,
                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
