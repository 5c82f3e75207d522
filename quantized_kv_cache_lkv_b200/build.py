"""Build liblkv.so (the CUDA library behind include/lkv.h) in-tree for sm_100a,
and the CPython module _native.so that calls it with torch tensors.

Each .cu file under csrc/ is compiled to an object under _build/ (in
parallel), then all are linked into quantized_kv_cache_lkv_b200/liblkv.so
with the CUDA runtime linked statically.  nvcc cross-compiles, so this works
on a machine without a GPU.  csrc/binding.cpp is compiled by g++ against the
headers of Python and torch, after the library, which needs neither: where there
is no torch, the library is all there is (run this file itself then; the package
imports torch).
"""
import concurrent.futures as cf
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "liblkv.so")
NATIVE = os.path.join(PKG, "_native.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]
# Translation units whose results must be bit-exact with the oracle (codes,
# (scale, zero), tiers and positions): no multiply-add contraction, so a
# plain a * b + c there can never turn into one fused operation.  The
# decode's deliberate fused operations live in other files.
NO_FMAD = ("quantize.cu", "tier.cu", "rope_append.cu")


def extra_flags(src):
    return ["--fmad=false"] if os.path.basename(src) in NO_FMAD else []


def nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return (sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) +
            [os.path.join(ROOT, "include", "lkv.h")])


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags(src), "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{p.stdout}\n{p.stderr}")
    return obj, p.stderr


def _native_key():
    """What the module is built against, as the text that it carries; None without torch."""
    try:
        version = importlib.metadata.version("torch")  # without importing it
    except importlib.metadata.PackageNotFoundError:  # a source tree on the path, or none
        try:
            import torch
        except ImportError:
            return None
        version = torch.__version__
    return f"lkv _native for torch {version}, {sysconfig.get_config_var('SOABI')}"


def _native_is_current(key):
    if not os.path.exists(NATIVE):
        return False
    newest = max(os.path.getmtime(f) for f in (os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "lkv.h"),
                                               os.path.abspath(__file__)))
    if os.path.getmtime(NATIVE) < newest:
        return False
    with open(NATIVE, "rb") as f:
        return key.encode() + b"\0" in f.read()


def build_native(force: bool = False) -> str:
    """_native.so: the torch libraries it needs are already loaded when it is imported."""
    key = _native_key()
    if key is None:
        raise ImportError("_native.so needs torch")
    if not force and _native_is_current(key):
        return NATIVE
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = NATIVE + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DLKV_NATIVE_KEY="{key}"',
           *("-I" + d for d in inc), os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L" + os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, NATIVE)
    return NATIVE


def build_library(force: bool = False, verbose: bool = False) -> str:
    srcs = _sources()
    newest = max(os.path.getmtime(f) for f in srcs + _headers() + [os.path.abspath(__file__)])
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """liblkv.so, then _native.so where there is a torch to build it against."""
    path = build_library(force, verbose)
    try:
        build_native(force)
    except ImportError as e:
        warnings.warn(f"{path} is built; {e}")
    return path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
