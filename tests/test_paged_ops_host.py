"""Host side of the operators around the paged cache (CPU)."""

import ctypes
import subprocess
import sys

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
