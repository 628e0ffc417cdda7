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


# ------------------------------------------------------------------ building


@pytest.fixture()
def build(monkeypatch):
    """The build script, its compiler calls recorded instead of run: (module, library names)."""
    import importlib.util

    spec = importlib.util.spec_from_file_location("bsq_build_of_a_test", os.path.join(PACKAGE, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    calls = []
    monkeypatch.setattr(mod, "_compile", lambda lib, cmd, tmp, verbose: calls.append((os.path.basename(lib), cmd)))
    return mod, calls


C_LIBS = ["libbsq.so", "libbsq_serving.so", "libbsq_ceiling.so"]


def test_extension_is_built_last_and_with_hipccs_compiler(build):
    mod, calls = build
    assert os.path.basename(mod.build()) == "libbsq.so"
    assert [n for n, _ in calls] == C_LIBS + ["_serving.so"]
    assert all(cmd[0] == mod.HIPCC for _, cmd in calls)


@pytest.mark.parametrize("what", ["torch", "headers"])
def test_c_libraries_are_built_without_torch(build, what, monkeypatch, tmp_path, capsys):
    """No torch, or one without headers: the C libraries, a note, and no extension left over from
    another build."""
    mod, calls = build
    if what == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        import torch

        monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
    monkeypatch.setattr(mod, "SERVING_EXT", str(tmp_path / "_serving.so"))
    (tmp_path / "_serving.so").write_bytes(b"of another build")
    mod.build()
    assert [n for n, _ in calls] == C_LIBS
    assert not (tmp_path / "_serving.so").exists()
    assert "_serving.so" in capsys.readouterr().err
