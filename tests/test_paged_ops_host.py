"""Host side of the operators around the paged cache (CPU)."""

import ctypes
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

from decode_kv_cache_kara_b200 import build as B
from decode_kv_cache_kara_b200 import kara as K

SIZES = """
import ctypes
from decode_kv_cache_kara_b200 import kara as K
for hkv, d, width, batch in ((0, 128, 64, 3), (-1, 128, 64, 3), (2, 0, 64, 3), (2, -64, 64, 3),
                             (2, 128, 64, 0), (2, 128, 64, -2), (2, 128, 0, 3), (2, 128, -5, 3)):
    p = K._Pool(256, 256, 0, 0, batch, width, 64, 16, hkv, d)
    for op in (K.OP_SPARSE, K.OP_PREFIX)[:2 if width > 0 else 1]:
        size = K.lib().kara_workspace_bytes(op, ctypes.byref(p), 0, 0, 4, 8)
        assert size == 0, (op, hkv, d, width, batch, size)
"""


def test_workspace_sizes_of_impossible_pools_are_zero(lib_path):
    """In a process of its own: a division by the number of KV heads would end it."""
    run = subprocess.run([sys.executable, "-c", SIZES], cwd=B.ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]


def test_sparse_workspace_ends_with_the_table(lib_path):
    """num_pages beyond the table means every page; the lists of such a call are no longer than the
    table is wide."""
    p = K._Pool(256, 256, 0, 0, 128, 1024, 64, 16, 4, 128)

    def size(pages):
        return K.lib().kara_workspace_bytes(K.OP_SPARSE, ctypes.byref(p), 0, 0, 28, pages)

    assert size(1023) < size(1024) == size(1025) == size(2 ** 31 - 1)


LINE = r"""
#include <cstdio>
#include "paged_plan.cuh"
int main() {
  const long long totals[] = {1, 5, 147, 148, 70000, 2147483647LL, 2147483648LL, 2163212288LL,
                              4294967296LL, 5000000011LL, 30000000000LL};
  for (long long total : totals)
    for (int parts : {1, 2, 44, 148, 160}) {
      if (parts > total) continue;
      for (int r = 0; r < parts; ++r) {
        const long long first = kara::part_start(r, parts, total);
        const long long end = kara::part_start(r + 1, parts, total);
        if (first >= end || kara::part_of(first, parts, total) != r ||
            kara::part_of(end - 1, parts, total) != r) {
          std::printf("%lld units, %d parts, part %d: [%lld, %lld)\n", total, parts, r, first, end);
          return 1;
        }
      }
    }
  return 0;
}
"""


def test_parts_of_a_work_line_past_32_bits(tmp_path):
    """Where a part starts and which part holds a unit agree, for lines of more units than 32 bits
    hold (many groups behind a long prefix; too much work to run)."""
    src, exe = tmp_path / "line.cu", tmp_path / "line"
    src.write_text(LINE)
    run = subprocess.run([B.nvcc(), "-std=c++17", "-I", B.CSRC, "-I", B.INCLUDE, str(src), "-o",
                          str(exe)] + B.ARCH, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


@pytest.fixture
def small_build(monkeypatch, tmp_path):
    """A build of one small source in a folder of its own, with a binding that does not compile."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int kara_one() { return 1; }\n')
    monkeypatch.setattr(B, "sources", lambda: [str(src)])
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(B, "_native_command", lambda out: [sys.executable, "-c", "raise SystemExit(3)"])
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    return tmp_path


def test_library_is_linked_where_the_binding_does_not_compile(small_build):
    with pytest.raises(RuntimeError, match="binding"):
        B.build()
    assert ctypes.CDLL(B.LIB).kara_one() == 1


def test_ensure_built_warns_without_the_binding(small_build):
    with pytest.warns(UserWarning, match="binding failed"):
        assert B.ensure_built() == B.LIB
    assert ctypes.CDLL(B.LIB).kara_one() == 1


def test_binding_is_named_for_its_python_and_torch(monkeypatch):
    name = os.path.basename(B.native_path())
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert B.native_path() != name and B._native_stale()


def test_missing_or_broken_binding_is_a_library_error(lib_path, monkeypatch, tmp_path):
    monkeypatch.setattr(K, "_NATIVE", None)
    path = tmp_path / "_native.so"
    monkeypatch.setattr(B, "native_path", lambda: str(path))
    with pytest.raises(K.KaraLibraryError, match="missing"):
        K._native()
    path.write_bytes(b"not a module")
    with pytest.raises(K.KaraLibraryError, match="cannot load"):
        K._native()
