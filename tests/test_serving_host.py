"""Checks of libbsq_serving that need no GPU: its exports, its refusals (every one returns
before any HIP call; the pointers are never dereferenced), workspace sizes, the Python
binding's refusals, and the 64-bit reference that the GPU tests compare with."""
import ctypes
import os

import numpy as np
import pytest
import torch

import serving_ref as R
from test_abi_host import declared_functions

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bsq_serving.h")
LIB = os.path.join(ROOT, "fp8_quantization_amd", "libbsq_serving.so")
OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 0x10000


class Cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("scale_stride", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


def cache(**kw):
    d = dict(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, num_pages=10,
             page_stride=2 * 128 * 64, scale_stride=2, num_heads=2, head_dim=128)
    d.update(kw)
    return Cache(**d)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from fp8_quantization_amd import build

        build.build()
    lib = ctypes.CDLL(LIB)
    i64, i32, p, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
    lib.kv_cache_append.argtypes = [p, p, i64, p, i64, p, p, p, i64, i64, i64, i64, i64, p]
    lib.kv_cache_attention.argtypes = [p, p, i64, i64, p, p, p, i64, i64, i64, i64, i64, i64, f32, i64,
                                       p, i64, p, p, i64, p]
    lib.kv_cache_attention_workspace.argtypes = [i64] * 8
    lib.kv_cache_attention_workspace.restype = i64
    lib.kv_pages_copy.argtypes = [p, p, p, i64, p]
    lib.kv_pages_reserve.argtypes = [p, i64, i64, i64, p, p, i64, p, p, i64, p, p]
    lib.kv_pages_fork.argtypes = [p, p, i64, i64, i64, p, p, p, p, i64, p, p]
    lib.kv_pages_free.argtypes = [p, i64, i64, i64, p, p, i64, p, i64, p]
    lib.kv_pages_compact.argtypes = [p, p, i64, i64, i64, p, p, p, i64, p, p, p, i64, p]
    lib.kv_pages_compact_workspace.argtypes = [i64]
    lib.kv_pages_compact_workspace.restype = i64
    lib.moe_few_tokens.argtypes = [i32, p, i64, i64, i64, i64, i64, i64, p, p, p, p, p, i32, p, p, p,
                                   i64, p, i64, p]
    lib.moe_few_tokens_workspace.argtypes = [i64] * 4
    lib.moe_few_tokens_workspace.restype = i64
    lib.bsq_serving_last_error.restype = ctypes.c_char_p
    return lib


def test_library_exports_its_header(lib):
    names = declared_functions(HEADER)
    assert names == sorted([
        "kv_cache_append", "kv_cache_attention", "kv_cache_attention_workspace", "kv_pages_copy",
        "kv_pages_reserve", "kv_pages_fork", "kv_pages_free", "kv_pages_compact",
        "kv_pages_compact_workspace", "moe_few_tokens", "moe_few_tokens_workspace",
        "bsq_serving_last_error"])
    for n in names:
        assert hasattr(lib, n), n


def append(lib, c=None, k=FAKE, ldk=256, v=FAKE, ldv=256, offsets=FAKE, lens=FAKE, table=FAKE, ldt=4,
           max_pages=4, seqs=2, rows=8, max_new=4):
    return lib.kv_cache_append(ctypes.byref(c or cache()), k, ldk, v, ldv, offsets, lens, table, ldt,
                               max_pages, seqs, rows, max_new, None)


BAD_CACHES = [(dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED),
              (dict(num_heads=0), INVALID), (dict(num_heads=70000), INVALID),
              (dict(num_pages=-1), INVALID), (dict(num_pages=1 << 31), INVALID),
              (dict(page_stride=2 * 128 * 64 - 16), INVALID), (dict(page_stride=2 * 128 * 64 + 8), INVALID),
              (dict(scale_stride=1), INVALID), (dict(k_codes=None), INVALID),
              (dict(v_scales=None), INVALID), (dict(v_codes=FAKE + 8), INVALID)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_cache_is_refused(lib, kw, status):
    assert append(lib, cache(**kw)) == status
    assert lib.bsq_serving_last_error()
    assert lib.kv_pages_copy(ctypes.byref(cache(**kw)), FAKE, FAKE, 1, None) == status


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k=FAKE + 2), dict(ldk=255), dict(ldk=252), dict(ldv=260),
    dict(offsets=None), dict(lens=None), dict(table=None), dict(ldt=3), dict(max_pages=-1),
    dict(seqs=-1), dict(rows=-1), dict(max_new=-1), dict(rows=1 << 31),
    dict(seqs=1 << 30, max_new=1 << 20, max_pages=1 << 20, ldt=1 << 20)])
def test_append_refusals(lib, kw):
    assert append(lib, **kw) == INVALID
    assert lib.bsq_serving_last_error()


@pytest.mark.parametrize("kw", [dict(seqs=0), dict(rows=0), dict(max_new=0), dict(max_pages=0),
                                dict(c=cache(num_pages=0))])
def test_append_nothing_to_do(lib, kw):
    assert append(lib, **kw) == OK
    assert lib.bsq_serving_last_error() == b""


def attend(lib, c=None, q=FAKE, ldq=512, hq=4, offsets=FAKE, lens=FAKE, table=FAKE, ldt=400,
           max_pages=400, seqs=2, rows=8, max_q=1, max_kv=20000, scale=0.1, window=0, out=FAKE,
           ldo=512, lse=None, ws=FAKE, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = 1 << 30
    return lib.kv_cache_attention(ctypes.byref(c or cache()), q, ldq, hq, offsets, lens, table, ldt,
                                  max_pages, seqs, rows, max_q, max_kv, scale, window, out, ldo, lse,
                                  ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(q=FAKE + 4), dict(ldq=511), dict(ldq=508), dict(ldo=504),
    dict(hq=3), dict(hq=0), dict(hq=65536 * 2), dict(max_q=-1), dict(max_kv=-1), dict(window=-1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=None), dict(ws=FAKE + 8),
    dict(ws_bytes=16), dict(offsets=None), dict(ldt=399), dict(rows=-5),
    dict(max_q=1 << 30, hq=16), dict(seqs=1 << 30, max_q=1 << 20)])
def test_attention_refusals(lib, kw):
    assert attend(lib, **kw) == INVALID
    assert lib.bsq_serving_last_error()


@pytest.mark.parametrize("kw", [dict(seqs=0), dict(rows=0), dict(max_q=0)])
def test_attention_nothing_to_do(lib, kw):
    assert attend(lib, **kw) == OK


def test_attention_workspace(lib):
    w = lib.kv_cache_attention_workspace
    assert w(2, 128, 4, 2, 8, 1, 500, 0) == 0                   # one run of pages
    big = w(2, 128, 4, 2, 8, 1, 100000, 0)
    assert big > 0 and big % (8 * 4 * 130 * 4) == 0             # splits * rows * heads * (D + 2) floats
    assert w(2, 128, 4, 2, 8, 1, 100000, 300) == 0              # a window leaves little to split
    assert w(2, 128, 4, 200, 40000, 200, 100000, 0) == 0        # rows enough without splitting
    assert w(2, 128, 4, 1, 100, 100, 100000, 0) > 0             # many rows, but not for every CU
    assert w(0, 128, 4, 2, 8, 1, 500, 0) == -1
    assert w(2, 100, 4, 2, 8, 1, 500, 0) == -1
    assert w(2, 128, 4, 2, -1, 1, 500, 0) == -1
    assert lib.bsq_serving_last_error()


def test_page_refusals(lib):
    c = ctypes.byref(cache())
    assert lib.kv_pages_copy(c, None, FAKE, 1, None) == INVALID
    assert lib.kv_pages_copy(c, FAKE, FAKE, -1, None) == INVALID
    assert lib.kv_pages_copy(c, FAKE, FAKE, 1 << 31, None) == INVALID
    assert lib.kv_pages_copy(c, None, None, 0, None) == OK

    def reserve(table=FAKE, ldt=4, M=4, S=2, lens=FAKE, refs=FAKE, pages=10, slots=FAKE, add=FAKE, n=1,
                status=FAKE):
        return lib.kv_pages_reserve(table, ldt, M, S, lens, refs, pages, slots, add, n, status, None)
    for kw in (dict(table=None), dict(ldt=3), dict(M=-1), dict(S=-1), dict(lens=None), dict(refs=None),
               dict(pages=-1), dict(slots=None), dict(add=None), dict(n=-1), dict(status=None)):
        assert reserve(**kw) == INVALID, kw
    assert reserve(n=0, slots=None, add=None, status=None) == OK

    def fork(table=FAKE, ldt=4, M=4, S=2, lens=FAKE, refs=FAKE, pa=FAKE, ch=FAKE, n=1, status=FAKE):
        return lib.kv_pages_fork(c, table, ldt, M, S, lens, refs, pa, ch, n, status, None)
    for kw in (dict(table=None), dict(ldt=3), dict(lens=None), dict(refs=None), dict(pa=None),
               dict(ch=None), dict(n=-1), dict(status=None)):
        assert fork(**kw) == INVALID, kw
    assert fork(n=0, pa=None, ch=None, status=None) == OK

    def free(table=FAKE, ldt=4, M=4, S=2, lens=FAKE, refs=FAKE, pages=10, slots=FAKE, n=1):
        return lib.kv_pages_free(table, ldt, M, S, lens, refs, pages, slots, n, None)
    for kw in (dict(table=None), dict(ldt=3), dict(lens=None), dict(refs=None), dict(slots=None),
               dict(n=-1)):
        assert free(**kw) == INVALID, kw
    assert free(n=0, slots=None) == OK

    need = lib.kv_pages_compact_workspace(10)
    assert need >= 4 * (4 + 10 + 10) and lib.kv_pages_compact_workspace(-1) == -1

    def compact(table=FAKE, ldt=4, M=4, S=2, lens=FAKE, refs=FAKE, out=FAKE + 4096, ldo=4,
                refs_out=FAKE, live=FAKE, ws=FAKE, n=need):
        return lib.kv_pages_compact(c, table, ldt, M, S, lens, refs, out, ldo, refs_out, live, ws, n,
                                    None)
    for kw in (dict(table=None), dict(out=None), dict(ldo=3), dict(refs=None), dict(refs_out=None),
               dict(live=None), dict(ws=None), dict(ws=FAKE + 4), dict(n=need - 1),
               dict(out=FAKE, ldo=8)):
        assert compact(**kw) == INVALID, kw


def moe(lib, fmt=0, x=FAKE, ldx=256, T=2, H=256, I=128, E=8, k=2, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE,
        logits=FAKE, ids=FAKE, weights=FAKE, y=FAKE, ldy=256, ws=FAKE, n=1 << 20):
    return lib.moe_few_tokens(fmt, x, ldx, T, H, I, E, k, w13, s13, w2, s2, logits, 1, ids, weights, y,
                              ldy, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), UNSUPPORTED), (dict(fmt=7), UNSUPPORTED), (dict(T=65), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(H=200), INVALID), (dict(I=64), INVALID), (dict(I=0), INVALID),
    (dict(H=1 << 18, ldx=1 << 18, ldy=1 << 18), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID),
    (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(k=17, E=20), INVALID), (dict(x=None), INVALID),
    (dict(x=FAKE + 2), INVALID), (dict(ldx=250), INVALID), (dict(y=None), INVALID),
    (dict(ldy=260), INVALID), (dict(w13=None), INVALID), (dict(w13=FAKE + 8), INVALID),
    (dict(s13=FAKE + 2), INVALID), (dict(s2=None), INVALID), (dict(ids=None), INVALID),
    (dict(weights=None), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 8), INVALID),
    (dict(n=100), INVALID)])
def test_moe_refusals(lib, kw, status):
    assert moe(lib, **kw) == status
    assert lib.bsq_serving_last_error()


def test_moe_nothing_to_do_and_workspace(lib):
    assert moe(lib, T=0) == OK and moe(lib, H=0, ldx=0, ldy=0) == OK
    w = lib.moe_few_tokens_workspace
    assert w(2, 256, 128, 2) == 2 * 2 * 128 * 4                  # h alone
    assert w(32, 256, 128, 2) == 32 * 2 * (128 + 256) * 4        # and the entries' parts
    assert w(65, 256, 128, 2) == -1 and w(2, 256, 100, 2) == -1 and w(2, 256, 128, 0) == -1


def test_binding_refuses_cpu_tensors_and_bad_caches():
    import fp8_quantization_amd as bsq

    c = bsq.kv_cache(4, 2, 64, device="cpu")
    assert [tuple(t.shape) for t in c] == [(4, 2, 4, 64, 16), (4, 2, 64, 64), (4, 2), (4, 2)]
    i = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    table = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(TypeError, match="GPU"):
        bsq.kv_cache_append(c, x, x, i, i[:2], table, 1)
    with pytest.raises(TypeError, match="GPU"):
        bsq.kv_cache_attention(x, c, i, i[:2], table, 1, 10)
    with pytest.raises(TypeError, match="KvCache"):
        bsq.kv_pages_copy([1, 2], i, i)
    with pytest.raises(TypeError):
        bsq.kv_pages_free(table, i[:2], i, i)
    with pytest.raises(TypeError, match="GPU"):
        bsq.moe_few_tokens(x[0], "mxfp4", i, i, i, i, 4, 2, router_logits=i)
    for bad in (dict(head_dim=80), dict(num_heads=0), dict(num_pages=-1)):
        with pytest.raises(bsq.BsqError):
            bsq.kv_cache(**{**dict(num_pages=1, num_heads=1, head_dim=64, device="cpu"), **bad})


# ------------------------------------------------------------------ the reference itself


def test_reference_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(R.E4M3, codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    x = np.random.default_rng(3).standard_normal(4000) * np.exp2(np.random.default_rng(4).uniform(-14, 10, 4000))
    x = np.concatenate([x, R.E4M3[:127], (R.E4M3[:126] + R.E4M3[1:127]) / 2, [-0.0, 1e9, -1e9]])
    want = torch.tensor(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.to_e4m3(x), want)


def test_reference_place_is_a_permutation():
    p = R.v_place(np.arange(64))
    assert sorted(p) == list(range(64)) and p[1] == 1 and p[4] == 16 and p[16] == 4


def test_reference_append_in_two_calls_keeps_values_within_a_step():
    """A page filled by two calls, the second with larger values: the old codes are re-encoded
    on the grown scale, within half a step of that scale."""
    rng = np.random.default_rng(0)
    x = R.bf16(rng.standard_normal((40, 1, 64)))
    x[30:] *= 64
    c = R.Cache(1, 1, 64)
    R.append(c, x[:30], x[:30], [0, 30], [30], [[0]])
    first = c.values("k", 0, 0, 30)
    most = 448 * 2.0 ** (int(c.ks[0, 0]) - 127)                  # the rule's scale saturates above it
    held = np.clip(x[:30, 0], -most, most)
    assert np.all(np.abs(first - held) <= np.maximum(np.abs(held) * 2.0 ** -4,
                                                     2.0 ** (int(c.ks[0, 0]) - 127 - 10)))
    R.append(c, x[30:], x[30:], [0, 10], [40], [[0]])
    got = c.values("v", 0, 0, 40)
    step = 2.0 ** (int(c.vs[0, 0]) - 127 - 10)                   # half the smallest step
    assert np.all(np.abs(got[:30] - first) <= np.maximum(np.abs(first) * 2.0 ** -4, step))


def test_reference_attention_catches_a_shifted_mask():
    """The bounds are tight enough to tell a mask that is off by one token."""
    rng = np.random.default_rng(1)
    c = R.Cache(3, 1, 64)
    k = R.bf16(rng.standard_normal((130, 1, 64)))
    R.append(c, k, R.bf16(rng.standard_normal((130, 1, 64))), [0, 130], [130], [[2, 0, 1]])
    q = R.bf16(rng.standard_normal((1, 1, 64)))
    out, lse, bo, bl, _ = R.attention(c, q, [0, 1], [130], [[2, 0, 1]], 0.125)
    off, lse2, _, _, _ = R.attention(c, q, [0, 1], [129], [[2, 0, 1]], 0.125)
    assert np.any(np.abs(out - off) > bo) and np.all(np.abs(lse - lse2) > bl)


def test_reference_pool():
    p = R.Pool([[0, 1, 9], [2, 9, 9], [9, 9, 9]], [100, 64, 0], [1, 1, 1, 0, 0])
    assert p.fork([0, 1], [2, 2 + 5]) == [0, 2]
    assert p.lens[2] == 100 and p.table[2][:2] == [0, 3] and p.refs == [2, 1, 1, 1, 0]
    assert p.reserve([1, 0], [65, 1]) == [1, 0]                  # two pages are not left, none is needed
    p.free([0])
    assert p.refs == [1, 0, 1, 1, 0]
    assert p.compact() == 3 and p.refs == [1, 1, 1, 0, 0] and p.table[2][:2] == [0, 1]
