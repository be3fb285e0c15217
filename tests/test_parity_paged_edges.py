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
                                         inv_freq, prefix_cache, rotation_close,
                                         sparse_reference)

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


# ------------------------------------------------------------------- malformed inputs, one by one

@pytest.mark.parametrize("cu", [[0, 4, 2, 9], [0, 4, 12, 9], [-1, 4, 6, 9], [0, 4, 6, 10],
                                [3, 3, 9, 1], [2 ** 31 - 1, 2, 2, 9]])
def test_append_skips_the_sequences_of_bad_token_counts(cu):
    """A healthy cache: sequences whose range of tokens descends or leaves [0, tokens] are skipped
    and reported, the others are appended; rows of no sequence stay as they were."""
    tokens, hq, hkv, d = 9, 6, 2, 64
    ctx = np.array([5, 20, 33])
    c = Cache(97, [n + 16 for n in ctx], hkv, d)
    c.lengths = ctx
    pool = c.make_pool()
    (q, k, v), dev = append_inputs(c, hq, tokens, True)
    pos = np.arange(tokens) * 7
    q_out = torch.full((tokens, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((tokens, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
    status = K.new_status()
    K.paged_rope_append(*dev, c.kd, c.vd, pool, inv_freq(d).cuda(), i32(pos), cu_tokens=i32(cu),
                        q_out=q_out, k_out=k_out, status=status)
    assert K.read_status(status) == K.ERR_INVALID_ARG
    good = [b for b in range(3) if 0 <= cu[b] <= cu[b + 1] <= tokens]
    assert 0 < len(good) < 3
    at = np.concatenate([np.zeros((0, 3))] +
                        [[(t, b, ctx[b] + i) for i, t in enumerate(range(cu[b], cu[b + 1]))]
                         for b in good if cu[b] < cu[b + 1]]).astype(np.int64)
    rows = np.unique(at[:, 0])
    rest = np.setdiff1d(np.arange(tokens), rows)
    rotation_close(q_out[rows], q[rows], pos[rows], inv_freq(d), False)
    rotation_close(k_out[rows], k[rows], pos[rows], inv_freq(d), False)
    assert (q_out[rest] == 5).all() and (k_out[rest] == 5).all()
    kref, vref = H.bits(c.k), H.bits(c.v)
    blk, row = c.table[at[:, 1], at[:, 2] // PAGE], at[:, 2] % PAGE
    kref[blk, row] = H.bits(k_out)[at[:, 0]]
    vref[blk, row] = H.bits(v)[at[:, 0]]
    assert np.array_equal(H.bits(c.kd), kref) and np.array_equal(H.bits(c.vd), vref)


@pytest.mark.parametrize("fault", ["past_table", "negative", "bad_block"])
def test_bounds_and_sparse_report_one_fault(fault):
    """One fault in one sequence of a healthy cache: its own code, and the other sequences' results
    are right."""
    c = Cache(98, [300, 75, 16, 0], 2, 64)
    c.table = np.where(c.table < 0, c.table[1, 0], c.table)    # every entry names a block
    q = bf16(c.gen, 4, 6, 64).cuda()
    bounds = c.bounds()
    _, ref, mag = sparse_reference(c, H.f64(q), H.f64(bounds), c.lengths, 6, 1, 2)
    whole = K.paged_page_bounds(c.kd, c.make_pool())
    if fault == "bad_block":
        c.table[0, 11] = c.num_blocks
    else:
        c.lengths[0] = -1 if fault == "negative" else PAGE * c.table.shape[1] + 1
    code = K.ERR_BAD_BLOCK if fault == "bad_block" else K.ERR_INVALID_ARG
    pool = c.make_pool()
    status = K.new_status()
    out = K.paged_sparse_attn(q, c.kd, c.vd, bounds.cuda(), pool, 6, status=status)
    assert K.read_status(status) == code
    assert torch.isfinite(out).all()
    attention_close(out[1:], ref[1:], mag[1:])
    status = K.new_status()
    got = K.paged_page_bounds(c.kd, pool, status=status)
    assert K.read_status(status) == code
    # the pages of the other sequences, and those of the first that are still named by its table
    old = c.pool.block_table[0].cpu().numpy()
    lost = old[11:12] if fault == "bad_block" else old[:300 // PAGE]
    kept = np.setdiff1d(np.arange(c.num_blocks), lost)
    assert torch.equal(got[kept], whole[kept]) and (got[lost] == 0).all()


@pytest.mark.parametrize("fault", ["descends", "past_batch", "below_zero", "pages_negative",
                                   "pages_past_table", "row_outside", "shorter_than_prefix"])
def test_prefix_reports_one_fault(fault):
    """One bad group or row among healthy ones: ERR_INVALID_ARG, and the healthy groups' rows are
    right."""
    c, _ = prefix_cache(99, [3, 3, 4], [5, 9, 2], 2, 64, least=1)
    q = bf16(c.gen, 10, 4, 64).cuda()
    ptr, pages, rows = [0, 3, 6, 10], [5, 9, 2], list(range(10))
    want = K.paged_prefix_attn(q, c.kd, c.vd, c.pool, i32(ptr), i32(pages))
    good = list(range(3))
    if fault == "descends":
        ptr = [0, 3, 6, 5]                          # the last group
        good = list(range(6))
    elif fault == "past_batch":
        ptr, good = [0, 3, 6, 11], list(range(6))
    elif fault == "below_zero":
        ptr, good = [-2, 3, 6, 10], list(range(3, 10))
    elif fault == "pages_negative":
        pages, good = [5, -3, 2], [0, 1, 2, 6, 7, 8, 9]
    elif fault == "pages_past_table":
        pages, good = [5, c.table.shape[1] + 1, 2], [0, 1, 2, 6, 7, 8, 9]
    elif fault == "row_outside":
        rows[4], good = 10, [0, 1, 2, 3, 5, 6, 7, 8, 9]
    else:
        c.lengths[4], good = 9 * PAGE - 1, [0, 1, 2, 3, 5, 6, 7, 8, 9]
    status = K.new_status()
    out = torch.full((10, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    K.paged_prefix_attn(q, c.kd, c.vd, c.make_pool(), i32(ptr), i32(pages), group_rows=i32(rows),
                        out=out, status=status)
    assert K.read_status(status) == K.ERR_INVALID_ARG
    ref, mag = op.dense_attention(H.f64(q), H.f64(c.k), H.f64(c.v), c.table,
                                  np.where(np.isin(np.arange(10), good), c.lengths, 0), 0.125, PAGE)
    attention_close(out[good], ref[good], mag[good])
    attention_close(want[good], ref[good], mag[good])


def test_prefix_pages_of_empty_groups_do_not_matter():
    """A plan of a fixed number of groups: behind and between those in use lie empty ones with any
    prefix_pages."""
    c, _ = prefix_cache(100, [3, 4], [5, 2], 2, 64)
    q = bf16(c.gen, 7, 4, 64)
    status = K.new_status()
    out = K.paged_prefix_attn(q.cuda(), c.kd, c.vd, c.pool, i32([0, 0, 3, 3, 7, 7, 7]),
                              i32([-7, 5, 2 ** 31 - 1, 2, c.table.shape[1] + 1, -2 ** 31]),
                              status=status)
    assert K.read_status(status) == 0
    ref, mag = op.dense_attention(H.f64(q), H.f64(c.k), H.f64(c.v), c.table, c.lengths, 0.125, PAGE)
    attention_close(out, ref, mag)
