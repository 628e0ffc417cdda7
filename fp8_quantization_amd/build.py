"""Build ``libbsq.so``, ``libbsq_serving.so`` and ``libbsq_ceiling.so`` in-tree with hipcc for gfx950.

Flags that matter for bit-exact results:
  -ffp-contract=off                          no fused multiply-adds are formed
  -fhip-fp32-correctly-rounded-divide-sqrt   IEEE division (the NVFP4 scale)
  -fno-gpu-flush-denormals-to-zero           fp32 subnormals are kept
and, for this GPU pool, packed fp32 instructions are disabled
(-Xclang -target-feature -Xclang -packed-fp32-ops; the host pass warns that
it does not know the feature, which is harmless).
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbsq.so")
SOURCES = [os.path.join(CSRC, "bsq_api.cpp"), os.path.join(CSRC, "bsq_kernels.hip"),
           os.path.join(CSRC, "bsq_consume.hip")]
# the same-byte-mix streaming kernel the bench compares the quantizers with
CEILING_LIB = os.path.join(HERE, "libbsq_ceiling.so")
CEILING_SOURCES = [os.path.join(CSRC, "bsq_ceiling.hip")]
# the serving operators
SERVING_LIB = os.path.join(HERE, "libbsq_serving.so")
SERVING_SOURCES = [os.path.join(CSRC, f) for f in ("bsq_serving_api.cpp", "bsq_kv.hip",
                                                   "bsq_pages.hip", "bsq_moe.hip",
                                                   "bsq_rope.hip", "bsq_route.hip",
                                                   "bsq_logprobs.hip")]
# their Python binding, a CPython extension over torch's C++ tensors
SERVING_EXT = os.path.join(HERE, "_serving.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
]


def build(verbose: bool = False, extra=()) -> str:
    """Build libbsq.so, libbsq_serving.so, libbsq_ceiling.so and, where torch is, the extension
    over the second; returns the path of the first."""
    _build_one(LIB, SOURCES, verbose, extra)
    _build_one(SERVING_LIB, SERVING_SOURCES, verbose, extra)
    _build_one(CEILING_LIB, CEILING_SOURCES, verbose, extra)
    _build_ext(verbose)
    return LIB


def _build_one(lib, sources, verbose, extra):
    tmp = lib + ".tmp"
    _compile(lib, [HIPCC, *FLAGS, *extra, *sources, "-o", tmp], tmp, verbose)


def _build_ext(verbose):
    """_serving.so: host C++ only, beside the library it links.  It needs torch and the headers of
    torch and Python; users of the C ABI do not, so without them it is left out."""
    import sysconfig

    try:
        import torch

        base = os.path.dirname(os.path.abspath(torch.__file__))
    except ImportError:
        return _no_ext("torch")
    include, python = os.path.join(base, "include"), sysconfig.get_paths()["include"]
    for header in (os.path.join(include, "torch", "csrc", "Exceptions.h"),
                   os.path.join(python, "Python.h")):
        if not os.path.exists(header):
            return _no_ext(header)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    tmp = SERVING_EXT + ".tmp"
    _compile(SERVING_EXT, [
        HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
        "-Wno-unknown-pragmas", "-Wno-unused-command-line-argument",
        "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-I" + os.path.join(ROOT, "include"), "-I" + include,
        "-I" + os.path.join(include, "torch", "csrc", "api", "include"),
        "-I" + python, "-I" + os.path.join(rocm, "include"),
        os.path.join(CSRC, "bsq_serving_py.cpp"), "-o", tmp, "-L" + HERE, "-l:libbsq_serving.so",
        "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_hip", "-lc10",
        "-lc10_hip", "-Wl,-rpath,$ORIGIN"], tmp, verbose)


def _no_ext(missing):
    """No extension rather than one of another build."""
    sys.stderr.write(f"_serving.so (Python binding of libbsq_serving.so) not built: no {missing}\n")
    if os.path.exists(SERVING_EXT):
        os.remove(SERVING_EXT)


def _compile(lib, cmd, tmp, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed building {os.path.basename(lib)}")
    noise = [ln for ln in (res.stdout + res.stderr).splitlines()
             if ln.strip() and "packed-fp32-ops" not in ln]
    if verbose and noise:
        print("\n".join(noise))
    os.replace(tmp, lib)


if __name__ == "__main__":
    build(verbose=True)
