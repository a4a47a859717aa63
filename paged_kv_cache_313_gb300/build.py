"""Build libpa.so in-tree with nvcc for sm_103a (GB300), and _pa_bind.so, the
compiled part of the Python binding, with g++.

Each translation unit compiles in parallel to an object file, then nvcc links
the library.  The CUDA runtime is linked statically, so the library needs only
the driver at load time; _pa_bind.so links to it and to PyTorch's libraries.
Usage: ``python -m
paged_kv_cache_313_gb300.build [--force]``.
"""
from __future__ import annotations

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
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libpa.so")
BIND = os.path.join(BUILD, "_pa_bind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa.so")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "pa.h")]


def _older(target, deps) -> bool:
    """Whether target is missing or older than one of deps."""
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in deps)


def _bind_made_for() -> str:
    """The Python and the PyTorch that a binding built now is for (PyTorch's version file holds its commit too)."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return "\n".join([sys.version, sysconfig.get_config_var("SOABI") or "", _torch_dir(), f.read()])


def _bind_stale() -> bool:
    """Whether the binding is missing, older than its sources, or made for another Python or PyTorch."""
    if _older(BIND, [os.path.join(CSRC, "bind.cpp"), os.path.join(INCLUDE, "pa.h")]):
        return True
    try:
        with open(BIND + ".for") as f:
            return f.read() != _bind_made_for()
    except OSError:
        return True


def _torch_dir() -> str | None:
    """Where PyTorch is installed (found without importing it), or None."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _compile_bind() -> str:
    obj = os.path.join(BUILD, "bind.o")
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-isystem",
           sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{r.stderr}")
    return obj


def _link_bind(obj: str) -> None:
    libs = os.path.join(_torch_dir(), "lib")
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-l:libpa.so", "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking the Python binding failed:\n{r.stderr}")
    if os.path.exists(BIND + ".for"):
        os.remove(BIND + ".for")
    os.replace(tmp, BIND)
    with open(BIND + ".for", "w") as f:
        f.write(_bind_made_for())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every .cu under csrc/ and link _build/libpa.so, and build _build/_pa_bind.so from bind.cpp, each where it is
    stale; returns the library's path.  The library does not need PyTorch, and is linked before the binding is looked at;
    the binding is left out where there is no PyTorch."""
    library = force or _older(LIB, _deps())
    binding = _torch_dir() is not None and (force or _bind_stale())
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        bind = ex.submit(_compile_bind) if binding else None
        if library:
            _build_library(verbose, extra_flags)
        if binding:
            _link_bind(bind.result())
    return LIB


def _build_library(verbose: bool, extra_flags) -> None:
    cc = nvcc()
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-Xlinker", "--no-undefined"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
