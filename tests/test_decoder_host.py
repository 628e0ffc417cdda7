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
