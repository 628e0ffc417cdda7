"""The package without the serving operators' libraries: the quantizers are there, and a serving
name says what is missing when it is used.  Each case is a copy of the package in an interpreter
of its own.  CPU only."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

PACKAGE = os.path.join(ROOT, "fp8_quantization_amd")
LIBS = ("libbsq_serving.so", "_serving.so")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not all(os.path.exists(os.path.join(PACKAGE, n)) for n in ("libbsq.so",) + LIBS):
        import __graft_entry__

        __graft_entry__.build()


def python(where, code):
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    return subprocess.run([sys.executable, "-c", code], cwd=where, env=env, capture_output=True,
                          text=True, timeout=300)


def copy(tmp_path, without):
    shutil.copytree(PACKAGE, tmp_path / "fp8_quantization_amd",
                    ignore=lambda d, names: [n for n in names if n in without or n == "__pycache__"])
    return tmp_path


USE = """
import fp8_quantization_amd as bsq
assert bsq.version() and bsq.quantize_block_scaled and bsq.BLOCK_SIZE[bsq.MXFP4] == 32
assert "kv_cache" in dir(bsq) and "serving" in dir(bsq)
for name in ("kv_cache_attention", "moe_few_tokens", "KvCache", "serving"):
    try:
        getattr(bsq, name)
    except ImportError as e:
        print(e)
    else:
        raise SystemExit(name + " is there")
try:
    bsq.kv_cash
except AttributeError:
    print("no such name")
"""


@pytest.mark.parametrize("without", [LIBS[:1], LIBS[1:], LIBS])
def test_quantizers_without_the_serving_libraries(tmp_path, without):
    res = python(copy(tmp_path, without), USE)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "serving" in res.stdout and "no such name" in res.stdout


def test_quantizers_beside_an_extension_of_another_build(tmp_path):
    """An extension that cannot be loaded stops the serving names alone."""
    (copy(tmp_path, LIBS[1:]) / "fp8_quantization_amd" / "_serving.so").write_bytes(b"of another build")
    res = python(tmp_path, USE)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "_serving.so" in res.stdout


def test_serving_names_load_their_libraries_on_first_use():
    res = python(ROOT, """
import fp8_quantization_amd as bsq
def loaded():
    return "libbsq_serving.so" in open("/proc/self/maps").read()
assert not loaded()
from fp8_quantization_amd import KvCache, kv_cache
assert loaded() and bsq.kv_cache is kv_cache and bsq.KV_PAGE == 64 and bsq.serving.KvCache is KvCache
c = bsq.kv_cache(1, 1, 64, device="cpu")
try:
    bsq.kv_cache(1, 1, 65)
except bsq.BsqError as e:
    assert e.status == 2
else:
    raise SystemExit("not refused")
""")
    assert res.returncode == 0, res.stdout + res.stderr
