"""What is built when: the C library needs no torch, and the native module is built
again for another torch or Python."""
import importlib
import os
import subprocess
import sys

import pytest

from quantized_kv_cache_lkv_b200 import build, lkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_TORCH = """
import importlib.metadata, os, sys, warnings
sys.path.insert(0, {root!r})
version = importlib.metadata.version
def none(name):
    if name == "torch":
        raise importlib.metadata.PackageNotFoundError(name)
    return version(name)
importlib.metadata.version = none
sys.modules["torch"] = None  # import torch raises ImportError
spec = importlib.util.spec_from_file_location("build", {path!r})
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)
build.BUILD, build.LIB, build.NATIVE = (os.path.join({tmp!r}, n) for n in ("o", "liblkv.so", "_native.so"))
build._sources = lambda: [os.path.join(build.CSRC, "multi.cu")]
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    assert build.build() == build.LIB
assert os.path.exists(build.LIB) and not os.path.exists(build.NATIVE)
assert any("torch" in str(w.message) for w in said)
"""


def test_library_without_torch(tmp_path):
    code = "import importlib.util" + WITHOUT_TORCH.format(root=ROOT, path=build.__file__, tmp=str(tmp_path))
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr


def test_library_comes_before_the_module(monkeypatch):
    """A module that cannot be built leaves the library built, and says so."""
    done = []
    monkeypatch.setattr(build, "build_library", lambda force, verbose: done.append("library") or build.LIB)

    def fails(force):
        done.append("module")
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(build, "build_native", fails)
    with pytest.raises(RuntimeError, match="g"):
        build.build()
    assert done == ["library", "module"]


def test_module_is_built_again_for_another_torch(monkeypatch):
    build.build()
    assert build._native_is_current(build._native_key())
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.1" if name == "torch" else version(name))
    assert not build._native_is_current(build._native_key())
    built = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: built.append(cmd) or subprocess.CompletedProcess(cmd, 1, "", "stop here"))
    with pytest.raises(RuntimeError, match="stop here"):
        build.build_native()
    assert len(built) == 1 and any("torch 0.1" in word for word in built[0])


def test_torch_without_a_distribution(monkeypatch):
    """A source tree of torch on the path has no entry among the installed packages."""
    def none(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(importlib.metadata, "version", none)
    import torch
    assert f"torch {torch.__version__}," in build._native_key()


@pytest.mark.parametrize("error,says", [(ImportError("undefined symbol: _ZN2at"), "does not load .*undefined symbol"),
                                        (ModuleNotFoundError("No module named '_native'"), "is missing")])
def test_what_is_said_of_a_module_that_does_not_load(monkeypatch, error, says):
    real = importlib.import_module

    def load(name, package=None):
        if name == "._native":
            raise error
        return real(name, package)

    monkeypatch.setattr(lkv, "_nat", None)
    monkeypatch.setattr(importlib, "import_module", load)
    with pytest.raises(RuntimeError, match=says):
        lkv.native()
