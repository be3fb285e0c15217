"""GPU parity of the operators around the paged cache at the edges of their contracts: pages that
the table does not hold, scores and values that are not finite, malformed inputs one at a time.

Tolerances are those of test_parity_paged_ops.py; page numbers, bounds, cache bytes and status
codes are exact.
"""

import math

import numpy as np
import pytest
import torch

from decode_kv_cache_kara_b200 import kara as K
from oracle import paged_ops as op
from tests import helpers as H
from tests.test_parity_paged_ops import (PAGE, Cache, append_inputs, attention_close, bf16, i32,
                                         inv_freq, prefix_cache, rotation_close)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- sparse attention

def select_without(c, q, bounds, pages, bad):
    """The selection of sequence 0 when the pages `bad` have no score."""
    n = -(-int(c.lengths[0]) // PAGE)
    blocks = np.where(np.isin(np.arange(n), bad), 0, c.table[0, :n])
    s = op.page_scores(H.f64(q[0]), H.f64(bounds), blocks)
    s[:, bad] = -np.inf
    return np.stack([op.select_pages(s[g], pages, 1, 2) for g in range(c.hkv)])


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("bad", [[10], [3, 4, 20, 21, 22], list(range(1, 40))])
def test_a_competing_page_without_a_block_goes_last(bad, hq):
    """All scores are below 0; a page whose block id is out of range is chosen only where nothing
    else is left, and adds nothing to the output."""
    pages = 12
    c = Cache(91, [16 * 44 - 3], 2, 64)
    c.k = -c.k.abs()
    c.kd = c.k.cuda()
    q = bf16(c.gen, 1, hq, 64).abs()
    bounds = c.bounds()
    for i, p in enumerate(bad):
        c.table[0, p] = (c.num_blocks + 5, -1, 2 ** 31 - 1)[i % 3]
    sel = torch.empty((1, 2, pages), dtype=torch.int32, device="cuda")
    status = K.new_status()
    out = K.paged_sparse_attn(q.cuda(), c.kd, c.vd, bounds.cuda(), c.make_pool(), pages, sel=sel,
                              status=status)
    assert K.read_status(status) == K.ERR_BAD_BLOCK
    want = select_without(c, q, bounds, pages, bad)
    assert np.array_equal(H.i32(sel)[0], want)
    read = np.where(np.isin(want, bad), -1, want)[None]
    ref, mag = op.sparse_attention(H.f64(q), H.f64(c.k), H.f64(c.v), read, c.table, c.lengths,
                                   0.125, PAGE)
    attention_close(out, ref, mag)


@pytest.mark.parametrize("hq", [2, 14, 16])
def test_selection_where_fp32_scores_are_not_numbers(hq):
    """Pages of one repeated key whose products with queries of mixed sign overflow: in fp32 their
    scores are inf - inf, in 64 bits they are numbers and belong to the largest."""
    hkv, d, pages = 2, 128, 20
    c = Cache(92, [700, 300], hkv, d)
    c.k[:] = c.k[:, :1]
    c.k[::3] *= 2.0 ** 100
    c.kd = c.k.cuda()
    q = bf16(c.gen, 2, hq, d) * 2.0 ** 40
    bounds = c.bounds()
    sel = torch.empty((2, hkv, pages - 5), dtype=torch.int32, device="cuda")
    K.paged_sparse_attn(q.cuda(), c.kd, c.vd, bounds.cuda(), c.pool, pages - 5, sel=sel)
    for b, n in enumerate(c.lengths):
        s = op.page_scores(H.f64(q[b]), H.f64(bounds), c.table[b, :-(-int(n) // PAGE)])
        for g in range(hkv):
            assert np.array_equal(H.i32(sel[b, g]), op.select_pages(s[g], pages - 5, 1, 2))


# -------------------------------------------------------------------- values that are not finite

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pages", [1, 3, 11, 15])
def test_infinity_in_the_last_shared_page(pages, d):
    """A prefix that ends inside a key tile, with infinite values in its last page: infinite
    outputs in those channels, not NaN, and the other channels keep their values."""
    c, ptr = prefix_cache(93, [5], [pages], 2, d)
    q = bf16(c.gen, 5, 8, d)
    last = int(c.table[0, pages - 1])
    c.vd[last, 3, 0, 7] = float("inf")
    c.vd[last, 15, 1, 20] = float("-inf")
    status = K.new_status()
    out = K.paged_prefix_attn(q.cuda(), c.kd, c.vd, c.pool, i32(ptr), i32([pages]), status=status)
    assert K.read_status(status) == 0
    assert (out[:, :4, 7] == float("inf")).all() and (out[:, 4:, 20] == float("-inf")).all()
    ref, mag = op.dense_attention(H.f64(q), H.f64(c.k), H.f64(c.v), c.table, c.lengths,
                                  1 / math.sqrt(d), PAGE)
    fine = np.ones(ref.shape, bool)
    fine[:, :4, 7] = fine[:, 4:, 20] = False
    attention_close(out.cpu()[torch.from_numpy(fine)], ref[fine], mag[fine])


@pytest.mark.parametrize("rows", [3, 40])
def test_nan_queries_and_lone_nan_keys_reach_the_output(rows):
    """A NaN query's outputs are NaN, and so are those of a row whose only own key is NaN; the
    others keep their values. `rows` takes both forms of the join."""
    hq = 64
    c, ptr = prefix_cache(94, [rows], [6], 8, 64, least=2)
    c.lengths[0] = 6 * PAGE + 1                      # row 0: one key of its own
    c.pool = c.make_pool()
    q = bf16(c.gen, rows, hq, 64).cuda()
    good = K.paged_prefix_attn(q, c.kd, c.vd, c.pool, i32(ptr), i32([6]))
    bounds = c.bounds().cuda()
    good_sparse = K.paged_sparse_attn(q, c.kd, c.vd, bounds, c.pool, 4)
    c.kd[int(c.table[0, 6]), 0, 5] = float("nan")    # KV head 5
    q[1, 9] = float("nan")
    bad = torch.zeros((rows, hq), dtype=torch.bool, device="cuda")
    bad[0, 40:48] = True
    bad[1, 9] = True
    out = K.paged_prefix_attn(q, c.kd, c.vd, c.pool, i32(ptr), i32([6]))
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], good[~bad])
    out = K.paged_sparse_attn(q, c.kd, c.vd, bounds, c.pool, 4)
    assert torch.isnan(out[bad]).all()
    bad[1, 8:16] = True                              # NaN takes part in the group's selection
    assert torch.equal(out[~bad], good_sparse[~bad])


def test_a_context_of_one_nan_key():
    c = Cache(95, [1, 0, 5], 2, 128)
    c.kd[int(c.table[0, 0]), 0] = float("nan")
    q = bf16(c.gen, 3, 4, 128).cuda()
    for out in (K.paged_sparse_attn(q, c.kd, c.vd, c.bounds().cuda(), c.pool, 4),
                K.paged_prefix_attn(q, c.kd, c.vd, c.pool, i32([0, 1, 2, 3]), i32([0, 0, 0]))):
        assert torch.isnan(out[0]).all() and (out[1] == 0).all() and torch.isfinite(out[2]).all()


@pytest.mark.parametrize("pages", [9, 10, 2 ** 31 - 1])
def test_more_pages_than_the_table_has(pages):
    """num_pages at and beyond the table's width (9): attention over every slot, with the fixed
    pages outnumbering the table too."""
    c = Cache(96, [120, 3, 0, 77], 2, 64)
    assert c.table.shape[1] == 9
    q = bf16(c.gen, 4, 6, 64)
    status = K.new_status()
    for sink, recent in ((1, 2), (min(pages - 1, 2 ** 30), 1)):
        out = K.paged_sparse_attn(q.cuda(), c.kd, c.vd, c.bounds().cuda(), c.pool, pages, sink,
                                  recent, status=status)
        assert K.read_status(status) == 0
        ref, mag = op.dense_attention(H.f64(q), H.f64(c.k), H.f64(c.v), c.table, c.lengths, 0.125,
                                      PAGE)
        attention_close(out, ref, mag)
