"""Build liblkv.so (the CUDA library behind include/lkv.h) in-tree for sm_100a,
and the CPython module _native.so that calls it with torch tensors.

Each .cu file under csrc/ is compiled to an object under _build/ (in
parallel), then all are linked into quantized_kv_cache_lkv_b200/liblkv.so
with the CUDA runtime linked statically.  nvcc cross-compiles, so this works
on a machine without a GPU.  csrc/binding.cpp is compiled by g++ against the
headers of Python and torch.
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

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


def build_native(force: bool = False) -> str:
    """_native.so: the torch libraries it needs are already loaded when it is imported."""
    src = os.path.join(CSRC, "binding.cpp")
    newest = max(os.path.getmtime(f) for f in (src, os.path.join(ROOT, "include", "lkv.h"), os.path.abspath(__file__)))
    if not force and os.path.exists(NATIVE) and os.path.getmtime(NATIVE) >= newest:
        return NATIVE
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = NATIVE + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + d for d in inc), src, "-o", tmp,
           "-L" + os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, NATIVE)
    return NATIVE


def build(force: bool = False, verbose: bool = False) -> str:
    build_native(force)
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


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
