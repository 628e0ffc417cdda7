"""Log probabilities, entropy and likeliest tokens on the GPU: ids exactly, values within the
reference's bounds."""
import numpy as np
import pytest
import torch

import decoder_ref as R
from test_gpu_serving_kv import bsq, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def check(bsq, x, tokens, top, **kw):  # noqa: F811
    got = bsq.token_logprobs(x, i32(tokens), top=top, **kw)
    torch.cuda.synchronize()
    t = np.asarray(tokens)
    lp, H, ids, best, bo, be, bb = R.logprobs(x.double().cpu().numpy(), t if t.ndim == 2 else t[:, None], top)
    assert np.array_equal(got.top_ids.cpu().numpy(), ids)
    for g, w, b in ((got.logprobs, lp.reshape(t.shape), bo.reshape(t.shape)), (got.entropy, H, be),
                    (got.top_logprobs, best, bb)):
        g = g.double().cpu().numpy()
        assert g.shape == w.shape and np.array_equal(np.isfinite(g), np.isfinite(w))
        ok = np.isfinite(w)
        assert np.array_equal(g[~ok], w[~ok])
        assert np.all(np.abs(g - w)[ok] <= b[ok]), np.max((np.abs(g - w)[ok] / b[ok]))
    return got


def random(rows, vocab, dtype, seed=0, scale=2.5):
    rng = np.random.default_rng(rows + vocab + seed)
    return torch.tensor(rng.standard_normal((rows, vocab)) * scale, device="cuda").to(dtype), \
        rng.integers(0, vocab, (rows, 3))


VOCABS = [1, 2, 7, 63, 64, 100, 2040, 2041, 2048, 2049, 8184, 8185, 8192, 8193, 16385, 50257, 100003]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("top", [0, 1, 5, 64])
def test_sizes(bsq, vocab, top, dtype):  # noqa: F811
    x, t = random(3, vocab, dtype)
    check(bsq, x, t, min(top, vocab))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 130000), (600, 300), (513, 9001), (40, 131072), (2, 524280),
                                        (900, 20011), (300, 50021)])
def test_rows(bsq, rows, vocab, dtype):  # noqa: F811
    """Short and long slices, of one chunk and of several, with a join and without; rows of odd
    lengths, which begin anywhere in 16 bytes."""
    x, t = random(rows, vocab, dtype)
    check(bsq, x, t, 20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("start", [0, 1, 3, 5, 7])
@pytest.mark.parametrize("vocab", [333, 4100])
def test_rows_of_a_larger_tensor(bsq, dtype, start, vocab):  # noqa: F811
    """Rows that begin anywhere in 16 bytes; numbers beside them that would win."""
    x, t = random(5, vocab, dtype)
    big = torch.full((5, vocab + 21), 1e4, device="cuda", dtype=dtype)
    view = big[:, start:start + vocab]
    view.copy_(x)
    a, b = check(bsq, view, t, 9), bsq.token_logprobs(x, i32(t), top=9)
    torch.cuda.synchronize()
    assert torch.equal(a.top_ids, b.top_ids)


@pytest.mark.parametrize("vocab", [70, 5000, 40000])
@pytest.mark.parametrize("rows", [2, 600])
def test_equal_logits(bsq, rows, vocab):  # noqa: F811
    """All equal, and a few values only: more elements tie than are ranked at once."""
    x = torch.zeros((rows, vocab), device="cuda")
    x[1] = torch.tensor(np.random.default_rng(1).integers(-2, 3, vocab), device="cuda").float()
    x[0, ::2] = -0.0
    t = np.random.default_rng(2).integers(0, vocab, (rows, 1))
    check(bsq, x[:2], t[:2], 40)
    if rows > 2:
        got = bsq.token_logprobs(x, i32(t), top=3)
        torch.cuda.synchronize()
        assert got.top_ids[2:].tolist() == [[0, 1, 2]] * (rows - 2)
        assert torch.allclose(got.entropy[2:], torch.tensor(np.log(vocab), dtype=torch.float32, device="cuda"), rtol=1e-5)


@pytest.mark.parametrize("order", ["ascending", "descending"])
@pytest.mark.parametrize("vocab", [3001, 33000])
def test_sorted_logits(bsq, vocab, order):  # noqa: F811
    x = torch.linspace(-9, 9, vocab, device="cuda")
    if order == "descending":
        x = x.flip(0)
    check(bsq, x[None].repeat(2, 1), [[0, vocab - 1]] * 2, 64)


@pytest.mark.parametrize("vocab", [90, 20000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_special_logits(bsq, vocab, dtype):  # noqa: F811
    inf, nan = float("inf"), float("nan")
    x, t = random(12, vocab, dtype)
    x[0] = -inf
    x[1] = nan
    x[2, 5:] = -inf
    x[3, ::2] = nan
    x[4, [3, vocab - 1]] = inf
    x[5, 7] = inf
    x[6] *= 300
    x[7] = -inf
    x[7, vocab // 2] = -3e38
    x[8, 0] = 3e38
    x[9] = x[9] - 1e4
    x[10, 1:] = -inf
    if dtype == torch.bfloat16:      # NaNs of every kind
        x[11].view(torch.int16)[::3] = 0x7F81
        x[11].view(torch.int16)[1::3] = -1
    t[:, 0] = 3
    t[:, 1] = [-1, vocab, 2 ** 31 - 1, -2 ** 31, 0, 7, 1, vocab // 2, 0, 0, 0, 0]
    check(bsq, x, t, 6)
    check(bsq, x, t, 60)


def test_one_token_a_row_and_none(bsq):  # noqa: F811
    x, t = random(7, 3000, torch.float32)
    a = check(bsq, x, t[:, 0], 4)
    assert a.logprobs.shape == (7,)
    b = bsq.token_logprobs(x, top=4)
    c = bsq.token_logprobs(x, i32(t[:, :0]))
    torch.cuda.synchronize()
    assert b.logprobs is None and torch.equal(b.top_ids, a.top_ids) and torch.equal(b.entropy, a.entropy)
    assert c.logprobs.shape == (7, 0) and c.top_ids.shape == (7, 0) and torch.equal(c.entropy, a.entropy)
    d = bsq.token_logprobs(x[:0], i32(t[:0]), top=2)
    assert d.logprobs.shape == (0, 3) and d.top_ids.shape == (0, 2) and d.entropy.shape == (0,)


def test_many_tokens_a_row(bsq):  # noqa: F811
    x, _ = random(3, 700, torch.bfloat16)
    check(bsq, x, np.tile(np.arange(-3, 720), (3, 1)), 2)


def test_equal_inputs_give_equal_bits(bsq):  # noqa: F811
    x, t = random(9, 60000, torch.float32)
    want = bsq.token_logprobs(x, i32(t), top=33)
    for _ in range(3):
        got = bsq.token_logprobs(x, i32(t), top=33)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_row_past_32_bits(bsq):  # noqa: F811
    """Rows whose offsets pass 2^32 bytes and 2^31 elements."""
    x, t = random(2, 5000, torch.bfloat16)
    big = torch.zeros(2 ** 31 + 20000, dtype=torch.bfloat16, device="cuda")
    view = big.as_strided((2, 5000), (2 ** 31 + 9001, 1))
    view.copy_(x)
    a, b = bsq.token_logprobs(view, i32(t), top=5), bsq.token_logprobs(x, i32(t), top=5)
    torch.cuda.synchronize()
    assert torch.equal(a.top_ids, b.top_ids) and torch.allclose(a.logprobs, b.logprobs, rtol=1e-5)


def test_refusals_of_the_binding(bsq):  # noqa: F811
    x = torch.zeros((4, 50), device="cuda")
    t = i32([0, 1, 2, 3])
    ws = torch.empty(4, dtype=torch.uint8, device="cuda")
    for err, kw in [(TypeError, dict(logits=x.half())), (TypeError, dict(logits=x.cpu())),
                    (TypeError, dict(logits=x[0])), (TypeError, dict(logits=x.t())),
                    (TypeError, dict(tokens=t.long())), (TypeError, dict(tokens=t.cpu())),
                    (TypeError, dict(top="a")), (bsq.BsqError, dict(tokens=t[:3])),
                    (bsq.BsqError, dict(top=-1)), (bsq.BsqError, dict(top=51)),
                    (bsq.BsqError, dict(logits=x.repeat(1, 3), top=65)),
                    (bsq.BsqError, dict(logits=x[:, :0])),
                    (bsq.BsqError, dict(logits=torch.zeros((4, 9000), device="cuda"), workspace=ws)),
                    (bsq.BsqError, dict(logits=torch.zeros((1, 1 << 19), device="cuda"), tokens=t[:1]))]:
        args = dict(logits=x, tokens=t)
        args.update(kw)
        with pytest.raises(err):
            bsq.token_logprobs(**args)


@pytest.mark.parametrize("vocab,rows", [(300, 2), (40000, 2), (40000, 700)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_vocabularies(bsq, vocab, rows, dtype):  # noqa: F811
    """Most of the vocabulary masked, by -inf, by the type's lowest number or by a large one: fewer
    tokens left than are asked for, one, none; the left ones early, late and in between."""
    x, t = random(rows, vocab, dtype)
    low = torch.finfo(dtype).min
    keep = [[0, 1, 2], [vocab - 1], [5, vocab // 2, vocab - 3], [], list(range(100, 130)),
            list(range(0, vocab, 97))]
    cases = [(m, k) for m in (-float("inf"), low, -1e9, -2e4) for k in keep]
    y = torch.empty((len(cases), vocab), device="cuda", dtype=dtype)
    for i, (m, k) in enumerate(cases):
        y[i] = m
        if k:
            y[i, k] = x[0, k]
    if rows > 2:                     # long slices, several chunks each
        y = y.repeat(rows // len(cases) + 1, 1)
    t = np.tile([[0, 1, vocab - 1]], (y.shape[0], 1))
    got = bsq.token_logprobs(y, i32(t), top=20)
    want = check(bsq, y[:len(cases)], t[:len(cases)], 20)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for r in range(0, y.shape[0], len(cases)):
            part = g[r:r + len(cases)]
            assert torch.equal(part, g[:len(part)])
        assert torch.allclose(g[:len(cases)].float(), w.float(), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("shift", [1e3, -1e3, 1.5e4, -1.5e4, 1.7e4, -1.7e4, 1e6, -1e6, 1e37])
def test_shifted_logits(bsq, shift):  # noqa: F811
    """What is added to all logits is not lost."""
    x, t = random(3, 30000, torch.float32)
    check(bsq, x + shift, t, 12)


@pytest.mark.parametrize("vocab", [20000, 130000])
def test_ties_of_many_in_long_slices(bsq, vocab):  # noqa: F811
    """More equal numbers than are ranked at once, beside larger ones, in slices of several chunks."""
    x = torch.zeros((2100, vocab), device="cuda", dtype=torch.bfloat16)
    rng = np.random.default_rng(3)
    for r in range(4):
        at = rng.choice(vocab, 3 + 5 * r, replace=False)
        x[r, torch.tensor(at, device="cuda")] = torch.tensor(rng.integers(1, 4, len(at)), device="cuda").to(x.dtype)
    x[4] = torch.linspace(-3, 3, vocab, device="cuda").to(x.dtype)
    t = rng.integers(0, vocab, (2100, 1))
    got = bsq.token_logprobs(x, i32(t), top=16)
    torch.cuda.synchronize()
    _, _, ids, best, _, _, bb = R.logprobs(x[:5].double().cpu().numpy(), t[:5], 16)
    assert np.array_equal(got.top_ids[:5].cpu().numpy(), ids)
    assert np.all(np.abs(got.top_logprobs[:5].double().cpu().numpy() - best) <= bb)
    assert bool((got.top_ids[5:] == torch.arange(16, device="cuda")).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(2048, 100003), (600, 131072)])
def test_many_rows_of_many_chunks(bsq, rows, vocab, dtype):  # noqa: F811
    """Slices of 7 and of 25 chunks: hundreds of terms a thread, random ones, rising ones, whose sums
    are rescaled at every chunk, and equal ones.

    Bounds, U = 2^-24.  A term is off by 4 (|d| + 2) U of it, d = z - max (its exponent's rounding,
    the hardware's exponential, and the same again where slices meet).  A thread adds 16 terms for each
    of up to C = (vocab + 7) / 4096 chunks, all of one sign: 16 C U of the sum.  A rescale costs 3 U and
    the rounding of its exponent, at most C + 2 times (the threads' and the slices' meeting among them):
    3 (C + 2) U, and U for each unit of e that the largest rises, at most the row's range.  Six and three
    sums over the threads and six over slices: 15 U.  All of that holds for the sum of s and for that of
    s d.  The base-2 logarithm is off by 2 U of it and U; a product and a difference follow."""
    U = 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn((rows, vocab), generator=g, device="cuda") * 2.5).to(dtype)
    x[1] = torch.linspace(-9, 9, vocab, device="cuda").to(dtype)
    x[2] = torch.linspace(-60, 20, vocab, device="cuda").to(dtype)
    x[3] = -7.25
    some = [0, 1, 2, 3, rows // 2, rows - 1]
    t = torch.randint(0, vocab, (rows, 4), generator=g, device="cuda", dtype=torch.int32)
    got = bsq.token_logprobs(x, t, top=20)
    torch.cuda.synchronize()
    z, t = x[some].double().cpu().numpy(), t[some].cpu().numpy()
    lp, H, ids, best, *_ = R.logprobs(z, t, 20)
    assert np.array_equal(got.top_ids[some].cpu().numpy(), ids)
    C = (vocab + 7 + 4095) // 4096
    for r in range(len(some)):
        d = z[r] - z[r].max()
        p = np.exp(d)
        log_l = np.log(p.sum())
        p /= p.sum()
        sums = (16 * C + 3 * (C + 2) + 15 - d.min()) * U
        off = (p * (np.abs(d) + 2)).sum() * 4 * U + sums
        off_log = off * (1 + 2.0 ** -10) + 6 * U * log_l + 2 * U
        for a, want, at in ((got.logprobs, lp, t[r]), (got.top_logprobs, best, ids[r])):
            bound = off_log + (np.abs(d[at]) + np.abs(want[r])) * 2 * U
            assert np.all(np.abs(a[some[r]].double().cpu().numpy() - want[r]) <= bound), r
        bound = off_log + (p * np.abs(d)).sum() * (off + sums + 8 * U) + \
            (p * np.abs(d) * (np.abs(d) + 2)).sum() * 4 * U + 4 * U * (H[r] + log_l)
        assert abs(got.entropy[some[r]].item() - H[r]) <= bound, r
