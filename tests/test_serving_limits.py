"""Sizes past what one launch holds (2^32 - 1 threads) are refused by the library's own checks,
before any HIP call.  No GPU needed; the pointers are never dereferenced."""
import ctypes

from test_abi_host import declared_functions
from test_serving_host import FAKE, HEADER, INVALID, append, cache, lib  # noqa: F401


def test_append_of_too_many_pages(lib):  # noqa: F811
    # 2^24 pages by 256 threads; 2^26 sequences of a token by 64
    assert append(lib, seqs=1 << 18, max_new=64 * 63 + 2, max_pages=70, ldt=70) == INVALID
    assert b"too large" in lib.bsq_serving_last_error()
    assert append(lib, seqs=1 << 26, max_new=1) == INVALID


def test_attention_of_too_many_sequences(lib):  # noqa: F811
    w = lib.kv_cache_attention_workspace
    assert w(8, 128, 32, 1 << 20, 1 << 20, 1, 500, 0) == 0           # 2^23 workgroups of 256
    assert w(8, 128, 32, 1 << 21, 1 << 21, 1, 500, 0) == -1          # 2^24
    assert b"too large" in lib.bsq_serving_last_error()
    assert w(8, 128, 32, 1 << 18, 1 << 25, 128, 500, 0) == 0         # 512 columns: 2^22 of 512
    assert w(8, 128, 32, 1 << 19, 1 << 26, 128, 500, 0) == -1        # 2^23
    assert w(8, 256, 32, 1 << 17, 1 << 24, 64, 500, 0) == 0          # 256 columns: 2^21 of 512
    assert w(8, 256, 32, 1 << 19, 1 << 24, 64, 500, 0) == -1         # 2^23


def test_pages_of_too_many_requests(lib):  # noqa: F811
    c = ctypes.byref(cache())                                        # two workgroups a page, one for its table
    assert lib.kv_pages_copy(c, FAKE, FAKE, 1 << 23, None) == INVALID
    assert b"too large" in lib.bsq_serving_last_error()
    assert lib.kv_pages_fork(c, FAKE, 4, 4, 2, FAKE, FAKE, FAKE, FAKE, 1 << 23, FAKE, None) == INVALID
    assert lib.kv_pages_free(FAKE, 4, 4, 2, FAKE, FAKE, 10, FAKE, 1 << 24, None) == INVALID


def test_raw_library_takes_plain_numbers():
    """serving_lib() has its signatures: 64-bit sizes go through as they are."""
    import fp8_quantization_amd as bsq

    raw = bsq.serving_lib()
    assert raw.kv_cache_attention_workspace(8, 64, 8, 70, 70, 1, 6400, 0) > 0
    assert raw.kv_cache_attention_workspace(1, 256, 32, 1, 1 << 20, 64, 100000, 0) > 1 << 32
    assert raw.kv_pages_compact_workspace(1 << 30) > 1 << 32
    assert raw.kv_pages_compact_workspace(-1) == -1
    assert raw.moe_few_tokens_workspace(64, 1 << 17, 1 << 17, 16) == 64 * 16 * 4 << 18
    assert raw.bsq_serving_last_error() == b""
    for name in declared_functions(HEADER):
        assert getattr(raw, name).argtypes is not None, name
