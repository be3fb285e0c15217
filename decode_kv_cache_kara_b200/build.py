"""In-tree build of libkara.so (nvcc, sm_100a) and of its Python marshalling next to this file.

``python -m decode_kv_cache_kara_b200.build`` compiles every ``csrc/*.cu`` into one shared
library with a C ABI (``include/kara.h``), and ``csrc/native.cpp`` (host code: the argument
marshalling of the per-layer calls) into the extension module ``_native``. The library needs the
CUDA toolkit alone, the module the headers of Python and torch too: the library is linked
whether or not the module compiles, and the module's file name carries the torch and the Python
that it was built for. ``ensure_built()`` rebuilds what is older than its sources or missing.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkara.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkara")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def native_path() -> str:
    """The marshalling module for the running Python and torch: both fix its binary interface."""
    import torch
    return os.path.join(PKG, f"_native.torch-{torch.__version__}"
                             f"{sysconfig.get_config_var('EXT_SUFFIX')}")


def _older(target: str, deps: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps)


def _stale() -> bool:
    """Whether the library is missing or older than its sources."""
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _native_stale() -> bool:
    """The same of the marshalling module, for the running Python and torch."""
    return _older(native_path(), [os.path.join(CSRC, "native.cpp")] +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _native_command(out: str) -> list:
    import torch
    t = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        raise RuntimeError("g++ not found: a C++ compiler is required to build the binding")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    headers = [os.path.join(t, "include"), os.path.join(t, "include/torch/csrc/api/include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = [cxx, "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE]
    for h in headers:
        cmd += ["-isystem", h]
    return cmd + [os.path.join(CSRC, "native.cpp"), "-o", out, "-L" + os.path.join(t, "lib"),
                  "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-ldl"]


def build_native(verbose: bool = False) -> str:
    """Compile the marshalling module. Returns its path; RuntimeError if it does not compile."""
    try:
        path = native_path()
        cmd = _native_command(path + ".tmp")
    except ImportError as e:
        raise RuntimeError(f"the binding needs torch: {e}") from e
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding failed to compile:\n{res.stdout}\n{res.stderr}")
    os.replace(path + ".tmp", path)
    return path


def build_library(verbose: bool = False, extra_flags=None) -> str:
    """Compile every CUDA source to an object, then link libkara.so. Returns its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + ARCH + ["-I", INCLUDE, "-I", CSRC] + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, "-c", src, "-o", obj] + flags
        res = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, cmd, res

    # one nvcc process per source, in parallel
    from concurrent.futures import ThreadPoolExecutor
    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as pool:
        results = list(pool.map(compile_one, srcs))
    objs = []
    for src, obj, cmd, res in results:
        if verbose:
            print(" ".join(cmd), flush=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and res.stderr.strip():
            print(res.stderr, flush=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [cc, "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC", "-cudart", "static"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build(verbose: bool = False, extra_flags=None) -> str:
    """The library, then the marshalling module; a module that does not compile raises when the
    library is in place. Returns the library's path."""
    build_library(verbose, extra_flags)
    build_native(verbose)
    return LIB


def ensure_built(verbose: bool = False) -> str:
    """Builds what is missing or out of date. Without the marshalling module the library still
    serves its C ABI: that it does not compile is a warning here."""
    if _stale():
        build_library(verbose)
    try:
        if _native_stale():
            build_native(verbose)
    except (RuntimeError, ImportError) as e:
        warnings.warn(f"the calls around the paged cache will not load: {e}")
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
