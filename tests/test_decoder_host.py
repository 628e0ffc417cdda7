"""Checks of bsq_decoder.h's entry points that need no GPU: exports, refusals (every one returns
before any HIP call; the pointers are never dereferenced) and the references of the GPU tests."""
import ctypes

import numpy as np
import pytest

import decoder_ref as R
from test_abi_host import declared_functions
from test_serving_host import FAKE, INVALID, OK, UNSUPPORTED
from conftest import ROOT

HEADER = ROOT + "/include/bsq_decoder.h"


@pytest.fixture(scope="module")
def lib():
    import fp8_quantization_amd as bsq

    return bsq.serving_lib()


def test_library_exports_its_header(lib):
    for name in declared_functions(HEADER):
        assert getattr(lib, name).argtypes is not None, name
    assert "qk_norm_rope" in declared_functions(HEADER)


# ------------------------------------------------------------------ norm and rotation


def rope(lib, dtype=0, q=FAKE, ldq=512, hq=4, k=FAKE, ldk=256, hkv=2, v=FAKE, ldv=256, D=128, rows=3,
         qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE, f=FAKE, rot=128, pairs=0, qo=FAKE, ldqo=512, ko=FAKE,
         ldko=256, vo=FAKE, ldvo=256):
    return lib.qk_norm_rope(dtype, q, ldq, hq, k, ldk, hkv, v, ldv, D, rows, qw, kw, eps, pos, f, rot,
                            pairs, qo, ldqo, ko, ldko, vo, ldvo, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(D=0), UNSUPPORTED),
    (dict(D=100), UNSUPPORTED), (dict(D=264), UNSUPPORTED), (dict(rot=136), UNSUPPORTED),
    (dict(rot=24), UNSUPPORTED), (dict(rot=-16), UNSUPPORTED), (dict(hq=0), INVALID),
    (dict(hq=65536), INVALID), (dict(hkv=0), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=1 << 31), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(v=None), INVALID), (dict(vo=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(ldq=504), INVALID), (dict(ldq=516), INVALID),
    (dict(qo=None), INVALID), (dict(ko=FAKE + 2), INVALID), (dict(ldvo=248), INVALID),
    (dict(pos=None), INVALID), (dict(f=None), INVALID), (dict(f=FAKE + 4), INVALID),
    (dict(qw=FAKE + 2), INVALID), (dict(rows=1 << 27), INVALID)])
def test_rope_refusals(lib, kw, status):
    assert rope(lib, **kw) == status
    assert lib.bsq_serving_last_error()


def test_rope_nothing_to_do(lib):
    assert rope(lib, rows=0, q=None, k=None, v=None, qo=None, ko=None, vo=None) == OK
    assert lib.bsq_serving_last_error() == b""


def test_reference_rotation_keeps_lengths_and_differences():
    """A pair's length stays, and scores depend on the difference of positions alone."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 2, 32))
    f = 100.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        a, _ = R.norm_rope(x, None, 0.0, np.array([5, 6, 7, 8]), f, inter)
        b, _ = R.norm_rope(x, None, 0.0, np.array([105, 106, 107, 108]), f, inter)
        assert np.allclose((a * a).sum(-1), (x * x).sum(-1))
        assert np.allclose((a[0] * a[3]).sum(-1), (b[0] * b[3]).sum(-1))
        assert not np.allclose(a, b) and np.array_equal(a[..., 16:], x[..., 16:])
    n, bound = R.norm_rope(x, np.ones(32), 0.0, np.zeros(4, int), f, False)
    assert np.allclose((n * n).mean(-1), 1) and np.all(bound < 0.02)


# ------------------------------------------------------------------ attention under masks


def masked(lib, sinks=0, masks=FAKE, words=1, max_q=1, window=0, ws=FAKE, ws_bytes=1 << 30, max_kv=20000,
           **kw):
    from test_serving_host import cache

    return lib.kv_cache_attention_masked(
        ctypes.byref(kw.get("c") or cache()), FAKE, 512, 4, FAKE, FAKE, FAKE, 400, 400, kw.get("seqs", 2), 8,
        max_q, max_kv, 0.1, window, sinks, masks, words, FAKE, 512, None, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(sinks=-1), dict(sinks=1 << 31), dict(words=0), dict(words=-1), dict(words=1 << 31),
    dict(max_q=65), dict(words=2, max_q=129), dict(masks=FAKE + 4), dict(window=-1), dict(ws=None),
    dict(ws=FAKE + 8), dict(ws_bytes=16)])
def test_masked_refusals(lib, kw):
    assert masked(lib, **kw) == INVALID
    assert lib.bsq_serving_last_error()


def test_masked_nothing_to_do(lib):
    assert masked(lib, seqs=0) == OK and masked(lib, max_q=0, words=0) == OK


def test_masked_workspace(lib):
    """Without sinks that of kv_cache_attention; sinks lengthen a window's pages."""
    w, m = lib.kv_cache_attention_workspace, lib.kv_cache_attention_masked_workspace
    for a in ((2, 128, 4, 2, 8, 1, 100000), (8, 64, 32, 3, 60, 20, 5000), (1, 256, 8, 9, 9, 1, 70000)):
        for window in (0, 100, 4000):
            assert m(*a, window, 0, 0) == w(*a, window)
    assert m(2, 128, 4, 2, 8, 1, 100000, 300, 100, 0) == 0
    assert m(2, 128, 4, 2, 8, 1, 100000, 300, 50000, 0) > 0
    assert m(2, 128, 4, 2, 8, 1, 100000, 300, -1, 0) == m(2, 128, 4, 2, 8, 1, 100000, 300, 1, -1) == -1
    assert lib.bsq_serving_last_error()
    # trees: blocks of columns fill the chip, or their pages are split
    assert m(8, 128, 32, 16, 700, 48, 6000, 0, 0, 1) == 0
    assert m(8, 128, 32, 1, 25, 25, 20000, 0, 0, 1) > 0 and m(8, 128, 32, 1, 25, 25, 2000, 0, 0, 1) == 0
    assert m(8, 128, 32, 1, 100, 100, 9000, 0, 0, 2) == 0 and m(8, 128, 32, 1, 100, 100, 10000, 0, 0, 2) > 0


def test_masked_workspace_of_masks_that_the_call_refuses(lib):
    """Words that do not hold max_q bits, or are too many."""
    m = lib.kv_cache_attention_masked_workspace
    for max_q, words in ((65, 1), (129, 2), (20000, 300), (1, 1 << 31), (1, 1 << 62)):
        assert masked(lib, max_q=max_q, words=words) == INVALID
        assert m(2, 128, 4, 2, 8, max_q, 20000, 0, 0, words) == -1 and lib.bsq_serving_last_error()
    for max_q, words in ((64, 1), (65, 2), (128, 2), (0, 1)):
        assert m(2, 128, 4, 2, 8, max_q, 20000, 0, 0, words) >= 0


@pytest.mark.parametrize("sizes", [(8, 128, 32, 1, 25, 25, 20000), (8, 128, 32, 1, 100, 100, 10000),
                                   (2, 64, 8, 2, 60, 30, 9000), (8, 256, 32, 1, 40, 40, 30000)])
def test_masked_workspace_of_windows_longer_than_any_sequence(lib, sizes):
    """A window past 2^31 - 1 is none, beside sinks too."""
    m = lib.kv_cache_attention_masked_workspace
    for window in (1 << 31, 1 << 40, (1 << 63) - 1):
        for words in (0, 2):
            assert m(*sizes, window, 4, words) == m(*sizes, 0, 4, words)


def test_reference_masks():
    """The reference's masks by hand: 5 rows after 4 tokens."""
    def see(*a):
        return np.nonzero(R.seen_tokens(*a))[0].tolist()
    assert see(9, 5, 2, 0, 0, None) == [0, 1, 2, 3, 4, 5, 6]
    assert see(9, 5, 2, 3, 0, None) == [4, 5, 6] and see(9, 5, 2, 3, 2, None) == [0, 1, 4, 5, 6]
    assert see(9, 5, 4, 0, 0, {0, 3}) == [0, 1, 2, 3, 4, 7]
    assert see(9, 5, 4, 3, 0, {0, 3}) == [3, 4, 7] and see(9, 5, 4, 3, 1, {0, 3}) == [0, 3, 4, 7]
    assert see(9, 5, 4, 1, 0, {0, 3}) == [4, 7] and see(9, 5, 4, 0, 0, set()) == [0, 1, 2, 3]
    assert see(2, 5, 4, 0, 0, {0, 3, 4}) == [0, 1] and see(2, 5, 1, 0, 0, None) == []
    assert R.words([{0, 64, 63}, set()], 2).tolist() == [[1 - (1 << 63), 1], [0, 0]]


def test_reference_attention_is_the_causal_one():
    import serving_ref as S

    rng = np.random.default_rng(1)
    c = S.Cache(3, 1, 64)
    k = S.bf16(rng.standard_normal((130, 1, 64)))
    S.append(c, k, k, [0, 130], [130], [[2, 0, 1]])
    q = S.bf16(rng.standard_normal((4, 2, 64)))
    chain = [set(range(i + 1)) for i in range(4)]
    for window in (0, 60):
        want = S.attention(c, q, [0, 4], [130], [[2, 0, 1]], 0.125, window)
        for masks in (None, chain):
            got = R.attention(c, q, [0, 4], [130], [[2, 0, 1]], 0.125, window, 0, masks)
            assert all(np.allclose(a, b, rtol=1e-12, atol=0) for a, b in zip(got, want))
    tree = R.attention(c, q, [0, 4], [130], [[2, 0, 1]], 0.125, 0, 0, [{0}, {1}, {0, 2}, {1, 3}])
    causal = S.attention(c, q, [0, 4], [130], [[2, 0, 1]], 0.125)
    off = np.abs(tree[0] - causal[0]) > causal[2]
    assert off[1:].any((1, 2)).all() and not off[0].any()    # the bounds tell one token less


# ------------------------------------------------------------------ routing


def route(lib, dtype=1, z=FAKE, ldl=64, T=5, E=64, k=6, score=0, bias=FAKE, groups=8, keep=3, top=2,
          renorm=1, factor=1.0, ids=FAKE, w=FAKE):
    return lib.moe_route(dtype, z, ldl, T, E, k, score, bias, groups, keep, top, renorm, factor, ids, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(score=2), UNSUPPORTED), (dict(score=-1), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(E=0), INVALID),
    (dict(E=1025, groups=1, ldl=2000), INVALID), (dict(groups=0), INVALID), (dict(groups=7), INVALID),
    (dict(E=65, ldl=65, groups=65), INVALID), (dict(keep=0), INVALID), (dict(keep=9), INVALID),
    (dict(top=0), INVALID), (dict(top=3), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID),
    (dict(k=9, keep=1), INVALID), (dict(factor=float("inf")), INVALID), (dict(z=None), INVALID),
    (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(ldl=63), INVALID),
    (dict(z=FAKE + 2), INVALID), (dict(dtype=0, z=FAKE + 1), INVALID), (dict(bias=FAKE + 2), INVALID),
    (dict(T=1 << 27), INVALID)])
def test_route_refusals(lib, kw, status):
    assert route(lib, **kw) == status
    assert lib.bsq_serving_last_error()


def test_route_nothing_to_do(lib):
    assert route(lib, T=0, z=None, ids=None, w=None) == OK


def group(lib, ids=FAKE, T=3000, k=8, E=64, pad=128, ro=FAKE, so=FAKE, ri=FAKE, er=FAKE, ws=FAKE, n=1 << 20):
    return lib.moe_group_rows(ids, T, k, E, pad, ro, so, ri, er, ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(k=0), dict(T=1 << 28, k=8), dict(T=1 << 40, k=1 << 40), dict(E=0), dict(E=1025),
    dict(pad=0), dict(pad=65537), dict(ids=None), dict(ro=None), dict(so=None), dict(ri=None),
    dict(ws=None), dict(ws=FAKE + 8), dict(n=100), dict(ids=FAKE + 2), dict(er=FAKE + 1)])
def test_group_refusals(lib, kw):
    assert group(lib, **kw) == INVALID
    assert lib.bsq_serving_last_error()


def test_group_workspace(lib):
    w = lib.moe_group_rows_workspace
    assert w(0, 1, 8) == 0 and w(64, 8, 256) == 0
    assert w(16384, 8, 256) > 4 * 16384 * 8 and w(16384, 8, 256) % (256 * 4) == 0
    assert w((1 << 31) - 1, 1, 1024) > 0
    assert w(-1, 1, 8) == -1 and w(1, 0, 8) == -1 and w(1, 1, 0) == -1 and lib.bsq_serving_last_error()


def test_reference_route_by_hand():
    z = np.log([[1.0, 2, 3, 4, 5, 6, 7, 8]])
    ids, w, _ = R.route(z, 2, "softmax", groups=4, keep=2, top=2, renormalize=False)
    assert ids.tolist() == [[7, 6]] and np.allclose(w, [[8 / 36, 7 / 36]])
    bias = np.array([0, 0, 1.0, 0, 0, 0, 0, 0])
    ids, w, _ = R.route(z, 2, "softmax", bias=bias, groups=4, keep=2, factor=2.0)
    assert ids.tolist() == [[2, 7]] and np.allclose(w, [[2 * 3 / 11, 2 * 8 / 11]])
    ids, w, _ = R.route(z, 2, "sigmoid")
    assert ids.tolist() == [[7, 6]] and np.allclose(w[0, 0] / w[0, 1], (8 / 9) / (7 / 8))
    ids, w, _ = R.route(np.array([[-np.inf, np.nan, -np.inf, -900.0, -901.0]]), 3, "sigmoid")
    assert ids.tolist() == [[3, 4, 0]] and np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e), 0]])
    ids, w, _ = R.route(np.array([[1.0, np.inf, np.inf, 0.0]]), 3, "softmax")
    assert ids.tolist() == [[1, 2, 0]] and w.tolist() == [[0.5, 0.5, 0.0]]


def test_reference_rows_by_hand():
    rows, scales, index, entry = R.group_rows(np.array([[2, 0], [0, 0], [-1, 3]]), 3, 4)
    assert rows.tolist() == [0, 3, 3, 4] and scales.tolist() == [0, 4, 4, 8]
    assert index.tolist() == [0, 1, 1, 0, -1, -1] and entry.tolist() == [[3, 0], [1, 2], [-1, -1]]


# ------------------------------------------------------------------ log probabilities


def logprobs(lib, dtype=1, z=FAKE, ldl=50000, R=4, V=50000, tokens=FAKE, n=2, top=3, lp=FAKE, H=FAKE,
             ids=FAKE, best=FAKE, ws=FAKE, size=1 << 20):
    return lib.token_logprobs(dtype, z, ldl, R, V, tokens, n, top, lp, H, ids, best, ws, size, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), UNSUPPORTED), (dict(V=(1 << 19) - 7, ldl=1 << 19), UNSUPPORTED), (dict(V=0), INVALID),
    (dict(R=-1), INVALID), (dict(R=1 << 31), INVALID), (dict(top=-1), INVALID), (dict(top=65), INVALID),
    (dict(V=2, top=3), INVALID), (dict(n=-1), INVALID), (dict(n=1 << 31), INVALID), (dict(z=None), INVALID),
    (dict(tokens=None), INVALID), (dict(lp=None), INVALID), (dict(ids=None), INVALID),
    (dict(best=None), INVALID), (dict(ldl=49999), INVALID), (dict(z=FAKE + 2), INVALID),
    (dict(dtype=0, z=FAKE + 1), INVALID), (dict(tokens=FAKE + 2), INVALID), (dict(ws=None), INVALID),
    (dict(ws=FAKE + 8), INVALID), (dict(size=100), INVALID), (dict(R=1 << 24), INVALID)])
def test_logprobs_refusals(lib, kw, status):
    assert logprobs(lib, **kw) == status
    assert lib.bsq_serving_last_error()


def test_logprobs_tokens_of_a_row_at_most(lib):
    """So many that a thread's index, 256 past the last, still is a number of 32 bits."""
    assert logprobs(lib, R=0, n=1 << 30) == OK
    for n in ((1 << 30) + 1, (1 << 31) - 1, 1 << 31):
        assert logprobs(lib, R=0, n=n) == logprobs(lib, n=n) == INVALID


def test_logprobs_nothing_to_do_and_workspace(lib):
    assert logprobs(lib, R=0, z=None, tokens=None) == OK
    w = lib.token_logprobs_workspace
    assert w(5, 2000, 4) == 0 and w(3000, 8000, 4) == 0 and w(2048, 128000, 20) == 0
    assert w(1, 128000, 5) == 63 * (5 * 8 + 12) and w(512, 128000, 20) == 512 * 4 * (20 * 8 + 12)
    assert w(1, 0, 0) == -1 and w(1, 5, 6) == -1 and w(1, 1 << 19, 1) == -1 and lib.bsq_serving_last_error()


def test_reference_logprobs_by_hand():
    z = np.log(np.array([[1.0, 3, 3, 1]]))
    lp, H, ids, best, *bounds = R.logprobs(z, np.array([[0, 2, 4, -1]]), 3)
    assert np.allclose(lp[0, :2], np.log([1 / 8, 3 / 8])) and lp[0, 2] == lp[0, 3] == -np.inf
    assert ids.tolist() == [[1, 2, 0]] and np.allclose(H, -2 * (np.log(1 / 8) / 8 + np.log(3 / 8) * 3 / 8))
    assert all(np.all(b < 1e-5) for b in bounds)
    lp, H, ids, best, *_ = R.logprobs(np.array([[np.nan, np.inf, 0, np.inf]]), np.array([[1, 2]]), 4)
    assert np.allclose(lp, [[-np.log(2), -np.inf]]) and np.allclose(H, np.log(2)) and ids.tolist() == [[1, 3, 2, 0]]
    lp, H, ids, _, *_ = R.logprobs(np.full((1, 3), -np.inf), np.array([[1]]), 2)
    assert lp[0, 0] == -np.inf and H[0] == 0 and ids.tolist() == [[0, 1]]
