"""In-tree build of libkara.so (nvcc, sm_100a) and of its Python marshalling next to this file.

``python -m decode_kv_cache_kara_b200.build`` compiles every ``csrc/*.cu`` into one shared
library with a C ABI (``include/kara.h``), and ``csrc/native.cpp`` (host code: the argument
marshalling of the per-layer calls) into the extension module ``_native``; ``ensure_built()``
rebuilds only when a source or the header is newer than either.
"""

from __future__ import annotations

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
LIB = os.path.join(PKG, "libkara.so")
NATIVE = os.path.join(PKG, "_native.so")
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


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(NATIVE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    deps = sources() + [os.path.join(CSRC, "native.cpp")] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


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


def build(verbose: bool = False, extra_flags=None) -> str:
    """Compile every source to an object, then link libkara.so. Returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + ARCH + ["-I", INCLUDE, "-I", CSRC] + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, "-c", src, "-o", obj] + flags
        res = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, cmd, res

    # one compiler process per source, in parallel
    from concurrent.futures import ThreadPoolExecutor
    srcs = sources()
    cmd = _native_command(NATIVE + ".tmp")
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as pool:
        native = pool.submit(subprocess.run, cmd, capture_output=True, text=True)
        results = list(pool.map(compile_one, srcs))
        res = native.result()
    if verbose:
        print(" ".join(cmd), flush=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding failed to compile:\n{res.stdout}\n{res.stderr}")
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
    os.replace(NATIVE + ".tmp", NATIVE)
    return LIB


def ensure_built(verbose: bool = False) -> str:
    if _stale():
        build(verbose=verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
