"""GPU parity of the operators around the paged cache (paged_rope_append, paged_page_bounds,
paged_sparse_attn, paged_prefix_attn) against the fp64 oracle, and their run in a decode loop.

Tolerances. Rotation: the fp32 sine and cosine of the reduced angle and two fp32 products are
off by at most 2^-20 of |x| + |y| together, and the result is rounded to bf16 once (2^-8 of the
value). Attention: the weights are rounded to bf16 before their product with V (2^-8 of each
weight), the fp32 logits and exponentials are off by less than 2^-12 of a weight, and the output
is rounded once (2^-8): |out - ref| <= 2^-8 |ref| + (2^-8 + 2^-12)(1 + 2^-8) sum w |v|. Bounds,
values and page numbers are exact.
"""

import math

import numpy as np
import pytest
import torch

from decode_kv_cache_kara_b200 import kara as K
from oracle import paged_ops as op
from tests import helpers as H

pytestmark = pytest.mark.gpu
PAGE = 16


def bf16(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(torch.bfloat16)


class Cache:
    """A small paged cache on the host and on the device; lengths[b] slots hold tokens, `room`
    more slots have blocks."""

    def __init__(self, seed, lengths, hkv, d, room=0, spare=3, scale=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.gen, self.hkv, self.d = gen, hkv, d
        pages = [(n + room + PAGE - 1) // PAGE for n in lengths]
        self.num_blocks = sum(pages) + spare
        perm = torch.randperm(self.num_blocks, generator=gen).tolist()
        width = max(max(pages), 1) + 1
        self.table = np.full((len(lengths), width), -1, dtype=np.int64)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.lengths = np.array(lengths, dtype=np.int64)
        self.k = bf16(gen, self.num_blocks, PAGE, hkv, d, scale=scale)
        self.v = bf16(gen, self.num_blocks, PAGE, hkv, d)
        self.kd, self.vd = self.k.cuda(), self.v.cuda()
        self.pool = self.make_pool()

    def make_pool(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return K.PagedPool(torch.tensor(self.table, **i32), torch.tensor(self.lengths, **i32),
                           torch.zeros(self.num_blocks, **i32), torch.zeros(1, **i32),
                           self.num_blocks, self.hkv, self.d)

    def bounds(self):
        """Bounds of every page (complete or not: only complete ones may matter)."""
        return torch.stack([self.k.amin(1), self.k.amax(1)], 2)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def attention_close(out, ref, mag):
    got = H.f64(out)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * (1 + 2.0 ** -8) * mag
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / np.maximum(bound, 1e-30)).max()))


# ------------------------------------------------------------------------------ rotary append

def inv_freq(rd, base=10000.0):
    return torch.tensor(base ** (-np.arange(0, rd, 2) / rd), dtype=torch.float32)


APPEND = {
    # name: (ctx, new, hq, hkv, d, rd, interleaved, packed)
    "decode_g7": ([0, 15, 16, 300, 31], None, 28, 4, 128, 128, False, True),
    "decode_d64": ([5, 47], None, 8, 8, 64, 64, True, False),
    "one": ([1000], None, 32, 8, 128, 128, False, True),
    "ragged": ([0, 3, 16, 250, 7, 31], [40, 0, 16, 1, 17, 130], 14, 2, 128, 128, False, True),
    "partial_rotary": ([9, 0], [23, 50], 6, 3, 128, 32, False, True),
    "interleaved": ([9, 1], [23, 33], 5, 1, 64, 16, True, True),
    "many": (list(range(300)), [1 + i % 3 for i in range(300)], 2, 1, 64, 64, False, False),
    "g1_wide": ([2], [37], 24, 24, 128, 96, True, True),
}


def append_inputs(c, hq, tokens, packed, seed=7):
    gen = torch.Generator().manual_seed(seed)
    x = bf16(gen, tokens, hq + 2 * c.hkv, c.d)
    xd = x.cuda()
    parts = [slice(0, hq), slice(hq, hq + c.hkv), slice(hq + c.hkv, hq + 2 * c.hkv)]
    host = [x[:, p] for p in parts]
    dev = [xd[:, p] if packed else xd[:, p].contiguous() for p in parts]
    return host, dev


def rotation_close(got, x, pos, freq, interleaved):
    ref = op.rotate(H.f64(x), pos, H.f64(freq), interleaved)
    size = op.rotate(np.abs(H.f64(x)), np.zeros_like(pos), H.f64(freq), interleaved)
    half = len(freq)
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    both = size[..., first] + size[..., second]
    mag = np.zeros_like(ref)
    mag[..., first] = mag[..., second] = both
    err = np.abs(H.f64(got) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * (1 + 2.0 ** -8) * mag).all(), err.max()


@pytest.mark.parametrize("name", list(APPEND))
def test_append_matches_oracle(name):
    ctx, new, hq, hkv, d, rd, interleaved, packed = APPEND[name]
    counts = new or [1] * len(ctx)
    c = Cache(11, [n + m for n, m in zip(ctx, counts)], hkv, d)
    c.lengths = np.array(ctx)
    pool = c.make_pool()
    total = sum(counts)
    pad = 0 if new is None else 3                   # rows behind the last sequence
    (q, k, v), dev = append_inputs(c, hq, total + pad, packed)
    rng = np.random.default_rng(5)
    pos = rng.integers(0, 3000, total + pad)
    pos[0] = 2_000_000_011                          # a far position
    freq = inv_freq(rd)
    cu = np.concatenate([[0], np.cumsum(counts)])
    bounds = torch.full((c.num_blocks, hkv, 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.full((total + pad, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((total + pad, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
    status = K.new_status()
    K.paged_rope_append(*dev, c.kd, c.vd, pool, freq.cuda(), i32(pos),
                        cu_tokens=None if new is None else i32(cu), interleaved=interleaved,
                        bounds=bounds, q_out=q_out, k_out=k_out, status=status)
    assert K.read_status(status) == 0
    rotation_close(q_out[:total], q[:total], pos[:total], freq, interleaved)
    rotation_close(k_out[:total], k[:total], pos[:total], freq, interleaved)
    assert (q_out[total:] == 5).all() and (k_out[total:] == 5).all()
    # the cache: k_out and v bit for bit in the tokens' slots, every other slot as it was
    kref, vref = H.bits(c.k), H.bits(c.v)
    at = op.append_slots(c.lengths, cu)
    blk, row = c.table[at[:, 1], at[:, 2] // PAGE], at[:, 2] % PAGE
    kref[blk, row] = H.bits(k_out)[at[:, 0]]
    vref[blk, row] = H.bits(v)[at[:, 0]]
    assert np.array_equal(H.bits(c.kd), kref) and np.array_equal(H.bits(c.vd), vref)
    # bounds of the pages that became complete, of the cache as it is now
    want = op.page_bounds(H.f64(c.kd), c.table, c.lengths + counts, c.lengths,
                          np.full(bounds.shape, 7.0), PAGE)
    assert np.array_equal(H.f64(bounds), want)


def test_append_in_place_and_ring():
    """q_out = q, k_out = k; a ring shorter than the call's tokens keeps the last ones."""
    ctx, counts, hq, hkv, d, w = [5, 40], [9, 21], 6, 2, 64, 8
    c = Cache(3, [n + m for n, m in zip(ctx, counts)], hkv, d)
    c.lengths = np.array(ctx)
    pool = c.make_pool()
    (q, k, _), dev = append_inputs(c, hq, sum(counts), False)
    pos, freq = np.arange(sum(counts)) * 3, inv_freq(d)
    ring = torch.zeros((2, 2 * w, hq, d), dtype=torch.bfloat16, device="cuda")
    status = K.new_status()
    K.paged_rope_append(*dev, c.kd, c.vd, pool, freq.cuda(), i32(pos),
                        cu_tokens=i32([0, 9, 30]), q_ring=ring, window=w, q_out=dev[0],
                        k_out=dev[1], status=status)
    assert K.read_status(status) == 0
    rotation_close(dev[0], q, pos, freq, False)
    rotation_close(dev[1], k, pos, freq, False)
    for b, (n, m, t0) in enumerate(((5, 9, 0), (40, 21, 9))):
        for i in range(m - w, m):
            for r in ((n + i) % w, (n + i) % w + w):
                assert torch.equal(ring[b, r], dev[0][t0 + i])


def test_append_reports_bad_slots_and_writes_nothing_there():
    c = Cache(4, [20, 16, 5], 2, 64)
    c.table[2, 0] = c.num_blocks                     # a bad block id
    c.lengths = np.array([19, 16 * c.table.shape[1], 3])   # sequence 1: past the table
    pool = c.make_pool()
    (q, _, _), dev = append_inputs(c, 4, 3, True)
    for row, code in ((1, K.ERR_INVALID_ARG), (2, K.ERR_BAD_BLOCK)):
        cu = [0, 0, 1, 1] if row == 1 else [0, 0, 0, 1]
        status = K.new_status()
        before = c.kd.clone()
        out = K.paged_rope_append(*dev, c.kd, c.vd, pool, inv_freq(64).cuda(), i32([4, 4, 4]),
                                  cu_tokens=i32(cu), status=status)
        assert K.read_status(status) == code
        assert torch.equal(c.kd, before)
        rotation_close(out[:1], q[:1], np.array([4]), inv_freq(64), False)
    for cu in ([0, 2, 1, 3], [0, 1, 2, 4], [-1, 1, 2, 3]):
        status = K.new_status()
        K.paged_rope_append(*dev, c.kd, c.vd, pool, inv_freq(64).cuda(), i32([4, 4, 4]),
                            cu_tokens=i32(cu), status=status)
        assert K.read_status(status) in (K.ERR_INVALID_ARG, K.ERR_BAD_BLOCK)


# -------------------------------------------------------------------------------- page bounds

@pytest.mark.parametrize("hkv,d", [(1, 64), (4, 128), (3, 64), (24, 128)])
@pytest.mark.parametrize("tail", [None, 0, 1, 40])
def test_page_bounds_match_oracle(hkv, d, tail):
    lengths = [0, 1, 15, 16, 17, 200, 333, 31]
    c = Cache(21, lengths, hkv, d, room=1)
    start = torch.full((c.num_blocks, hkv, 2, d), 9.0, dtype=torch.bfloat16, device="cuda")
    first = None if tail is None else [max(0, n - tail) - (n == 1) * 5 for n in lengths]
    status = K.new_status()
    got = K.paged_page_bounds(c.kd, c.pool, bounds=start,
                              from_slot=None if first is None else i32(first), new_slots=1,
                              status=status)
    assert K.read_status(status) == 0
    want = op.page_bounds(H.f64(c.k), c.table, c.lengths + 1, first,
                          np.full(start.shape, 9.0), PAGE)
    assert np.array_equal(H.f64(got), want)


def test_page_bounds_many_rows_and_errors():
    lengths = [(i * 37) % 90 for i in range(600)]
    c = Cache(22, lengths, 2, 64)
    got = K.paged_page_bounds(c.kd, c.pool)
    want = op.page_bounds(H.f64(c.k), c.table, c.lengths, None, np.zeros(got.shape), PAGE)
    assert np.array_equal(H.f64(got), want)
    c.table[2, 0] = -7
    c.lengths[4] = 16 * c.table.shape[1] + 1
    status = K.new_status()
    got = K.paged_page_bounds(c.kd, c.make_pool(), status=status)
    assert K.read_status(status) in (K.ERR_BAD_BLOCK, K.ERR_INVALID_ARG)
    c.lengths[4] = 0
    want = op.page_bounds(H.f64(c.k), np.where(c.table == -7, 0, c.table), c.lengths, None,
                          np.zeros(got.shape), PAGE)
    fine = np.ones(len(want), bool)
    fine[0] = False                                  # the oracle's stand-in for the bad block
    assert np.array_equal(H.f64(got)[fine], want[fine])


# --------------------------------------------------------------------------- sparse attention

SPARSE = {
    # name: (lengths, hq, hkv, d, pages, sink, recent)
    "g7": ([700, 0, 1, 16, 17, 128, 129, 300, 1023], 28, 4, 128, 8, 1, 2),
    "g1_d64": ([333, 64, 80, 81], 3, 3, 64, 5, 0, 1),
    "g8_long": ([9000, 5000], 16, 2, 128, 40, 2, 3),
    "only_fixed": ([400, 90], 4, 2, 64, 4, 1, 3),
    "one_page": ([400, 5], 4, 2, 64, 1, 0, 1),
    "all": ([400, 5], 10, 2, 128, 100, 1, 1),
    "g5_odd": ([2500], 5, 1, 64, 33, 0, 4),
}


def sparse_reference(c, q, bounds, lengths, pages, sink, recent):
    hkv = c.hkv
    sel = np.full((len(lengths), hkv, pages), -1, dtype=np.int64)
    for b, n in enumerate(lengths):
        np_ = -(-int(n) // PAGE)
        s = op.page_scores(q[b], bounds, c.table[b, :np_])
        for g in range(hkv):
            sel[b, g] = op.select_pages(s[g], pages, sink, recent)
    out, mag = op.sparse_attention(q, H.f64(c.kd), H.f64(c.vd), sel, c.table, lengths,
                                   1 / math.sqrt(c.d), PAGE)
    return sel, out, mag


@pytest.mark.parametrize("new_slots", [0, 1])
@pytest.mark.parametrize("name", list(SPARSE))
def test_sparse_matches_oracle(name, new_slots):
    lengths, hq, hkv, d, pages, sink, recent = SPARSE[name]
    c = Cache(31, lengths, hkv, d, room=1, scale=1.5)
    q = bf16(c.gen, len(lengths), hq, d, scale=1.5)
    bounds = c.bounds()
    sel = torch.full((len(lengths), hkv, pages), 77, dtype=torch.int32, device="cuda")
    status = K.new_status()
    out = K.paged_sparse_attn(q.cuda(), c.kd, c.vd, bounds.cuda(), c.pool, pages,
                              sink_pages=sink, recent_pages=recent, new_slots=new_slots, sel=sel,
                              status=status)
    assert K.read_status(status) == 0
    ref_sel, ref, mag = sparse_reference(c, H.f64(q), H.f64(bounds), c.lengths + new_slots, pages,
                                         sink, recent)
    assert np.array_equal(H.i32(sel), ref_sel)
    attention_close(out, ref, mag)
    again = K.paged_sparse_attn(q.cuda(), c.kd, c.vd, bounds.cuda(), c.pool, pages,
                                sink_pages=sink, recent_pages=recent, new_slots=new_slots)
    assert torch.equal(out, again)                   # without sel, and deterministic


@pytest.mark.parametrize("kind", ["zero_query", "equal_pages", "near_ties", "huge", "vast", "tiny",
                                  "two_values"])
def test_sparse_selection_at_the_border(kind):
    """Scores that fp32 cannot tell apart, or that are equal: the selection is still that of the
    exact scores, ties to the lower page."""
    hq, hkv, d, pages = 6, 2, 128, 20
    c = Cache(41, [3100, 700], hkv, d)
    q = bf16(c.gen, 2, hq, d)
    if kind == "zero_query":
        q.zero_()
    elif kind == "equal_pages":
        c.k[:] = c.k[0:1]
    elif kind == "near_ties":                        # pages differ in one small channel only
        c.k[:] = c.k[0:1]
        c.k[..., 5] = (torch.rand(c.num_blocks, 1, 1, generator=c.gen) * 2.0 ** -12).to(
            torch.bfloat16)
    elif kind == "huge":                             # fp32 sums overflow for some pages
        c.k[::3] *= 2.0 ** 100
        q *= 2.0 ** 24
    elif kind == "vast":                             # so do products
        c.k[::3] *= 2.0 ** 100
        q *= 2.0 ** 100
    elif kind == "tiny":                             # fp32 products vanish
        c.k *= 2.0 ** -90
        q *= 2.0 ** -60
    else:
        c.k[:] = torch.where(torch.rand(c.num_blocks, 1, 1, 1, generator=c.gen) < 0.5, 1.0, -1.0)
        q = q.abs()
    c.kd = c.k.cuda()
    bounds = c.bounds()
    sel = torch.empty((2, hkv, pages), dtype=torch.int32, device="cuda")
    K.paged_sparse_attn(q.cuda(), c.kd, c.vd, bounds.cuda(), c.pool, pages, sel=sel)
    for b, n in enumerate(c.lengths):
        s = op.page_scores(H.f64(q[b]), H.f64(bounds), c.table[b, :-(-int(n) // PAGE)])
        for g in range(hkv):
            assert np.array_equal(H.i32(sel[b, g]), op.select_pages(s[g], pages, 1, 2))


def test_sparse_skips_what_the_table_does_not_hold():
    c = Cache(42, [500, 500], 2, 64, scale=2.0)
    q = bf16(c.gen, 2, 4, 64)
    c.table[1, 0] = c.num_blocks + 5                 # the sink page of sequence 1
    status = K.new_status()
    out = K.paged_sparse_attn(q.cuda(), c.kd, c.vd, c.bounds().cuda(), c.make_pool(), 6,
                              status=status)
    assert K.read_status(status) == K.ERR_BAD_BLOCK
    assert torch.isfinite(out).all()
    c.lengths[0] = 16 * c.table.shape[1] + 1
    status = K.new_status()
    K.paged_sparse_attn(q.cuda(), c.kd, c.vd, c.bounds().cuda(),
                        Cache.make_pool(c), 6, status=status)
    assert K.read_status(status) in (K.ERR_INVALID_ARG, K.ERR_BAD_BLOCK)


def test_sparse_ignores_what_lies_behind_the_last_slot():
    c = Cache(43, [37, 250], 2, 128)
    q = bf16(c.gen, 2, 8, 128).cuda()
    bounds = c.bounds().cuda()
    out = K.paged_sparse_attn(q, c.kd, c.vd, bounds, c.pool, 5)
    for b, n in enumerate(c.lengths):
        blk = int(c.table[b, n // PAGE])
        c.kd[blk, n % PAGE:] = float("nan")
        c.vd[blk, n % PAGE:] = float("inf")
    assert torch.equal(K.paged_sparse_attn(q, c.kd, c.vd, bounds, c.pool, 5), out)


# --------------------------------------------------------------------- shared-prefix attention

PREFIX = {
    # name: (rows per group, prefix pages per group, hq, hkv, d)
    "samples": ([8], [9], 28, 4, 128),
    "ragged_groups": ([1, 3, 0, 17, 2, 1], [4, 8, 2, 21, 0, 0], 16, 2, 128),
    "two_tiles": ([19], [40], 8, 1, 64),             # 152 query rows: both teams
    "many_rows": ([70, 2], [33, 130], 8, 1, 128),    # 560 query rows: three items
    "g1_d64": ([5, 4], [3, 17], 3, 3, 64),
    "one_page": ([2, 2], [1, 1], 14, 2, 128),
    "g3": ([130], [9], 6, 2, 64),
    "hkv8": ([6, 9], [16, 64], 32, 8, 128),
}


def prefix_cache(seed, rows, pages, hkv, d, scale=1.0, least=0):
    """Rows of a group share their first pages; 0 to 90 slots of their own behind them."""
    rng = np.random.default_rng(seed)
    group = [j for j, r in enumerate(rows) for _ in range(r)]
    own = rng.integers(least, 91, len(group))
    own[0] = max(0, least)
    c = Cache(seed, [pages[j] * PAGE + int(n) for j, n in zip(group, own)], hkv, d, room=1,
              scale=scale)
    first = {}
    for i, j in enumerate(group):
        first.setdefault(j, i)
        c.table[i, :pages[j]] = c.table[first[j], :pages[j]]
    c.pool = c.make_pool()
    return c, np.concatenate([[0], np.cumsum(rows)])


def check_prefix(c, q, ptr, pages, new_slots=0, scale=None, **kw):
    status = K.new_status()
    out = K.paged_prefix_attn(q.cuda(), c.kd, c.vd, c.pool, i32(ptr), i32(pages),
                              new_slots=new_slots, scale=scale, status=status, **kw)
    assert K.read_status(status) == 0
    ref, mag = op.dense_attention(H.f64(q), H.f64(c.kd), H.f64(c.vd), c.table,
                                  c.lengths + new_slots,
                                  1 / math.sqrt(c.d) if scale is None else scale, PAGE)
    attention_close(out, ref, mag)
    return out


@pytest.mark.parametrize("new_slots", [0, 1])
@pytest.mark.parametrize("name", list(PREFIX))
def test_prefix_matches_oracle(name, new_slots):
    rows, pages, hq, hkv, d = PREFIX[name]
    c, ptr = prefix_cache(51, rows, pages, hkv, d)
    q = bf16(c.gen, len(c.lengths), hq, d)
    out = check_prefix(c, q, ptr, pages, new_slots)
    assert torch.equal(out, check_prefix(c, q, ptr, pages, new_slots))
    # the same as rows on their own, up to the rounding of both
    if new_slots == 0:
        own = H.f64(K.paged_decode_attn(q.cuda(), c.kd, c.vd, c.pool))
        assert np.abs(H.f64(out) - own).max() <= 2.0 ** -5 * max(1.0, np.abs(own).max())


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0])
def test_prefix_peaked_rows(scale):
    """Strong logits that grow along the prefix: the exponent base moves again and again."""
    c, ptr = prefix_cache(52, [5, 3], [40, 24], 2, 128)
    grow = torch.linspace(0.2, 3.0, 40)
    for j, i in ((0, 0), (1, 5)):
        for p in range((40, 24)[j]):
            c.k[int(c.table[i, p])] *= float(grow[p])
    c.kd = c.k.cuda()
    check_prefix(c, bf16(c.gen, 8, 8, 128, scale=2.0), ptr, [40, 24], scale=scale)


@pytest.mark.parametrize("pages", [1, 11, 20])
def test_prefix_without_logits(pages):
    """scale = 0: the plain mean of the values, with a prefix that ends inside a key tile."""
    c, ptr = prefix_cache(56, [5], [pages], 2, 128)
    check_prefix(c, bf16(c.gen, 5, 8, 128, scale=2.0), ptr, [pages], scale=0.0)


def test_prefix_with_rows_in_any_order():
    """group_rows: members anywhere in the batch; rows in no group keep their output; a row
    listed twice is computed."""
    c, _ = prefix_cache(53, [4, 3], [11, 6], 2, 64)
    n = len(c.lengths)
    perm = np.array([6, 1, 3, 0, 5, 2, 4])
    c.table, c.lengths = c.table[perm], c.lengths[perm]
    c.pool = c.make_pool()
    place = np.argsort(perm)                         # where the old rows went
    listed = np.concatenate([place[:4], place[4:6], place[4:5]])
    q = bf16(c.gen, n, 6, 64)
    out = torch.full((n, 6, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    status = K.new_status()
    K.paged_prefix_attn(q.cuda(), c.kd, c.vd, c.pool, i32([0, 4, 7]), i32([11, 6]),
                        group_rows=i32(listed), out=out, status=status)
    assert K.read_status(status) == 0
    ref, mag = op.dense_attention(H.f64(q), H.f64(c.k), H.f64(c.v), c.table, c.lengths, 0.125,
                                  PAGE)
    done = np.unique(listed)
    attention_close(out[done], ref[done], mag[done])
    rest = [i for i in range(n) if i not in done]
    assert rest and (out[rest] == 3).all()
    assert torch.equal(K.paged_prefix_attn(q.cuda(), c.kd, c.vd, c.pool, i32([0]), i32([]),
                                           out=out.clone()), out)


def test_prefix_reports_bad_groups():
    c, ptr = prefix_cache(54, [3, 3], [5, 5], 2, 64, least=1)
    q = bf16(c.gen, 6, 4, 64).cuda()
    bad_row = list(range(6))
    bad_row[4] = 6
    for bad in (dict(ptr=[0, 4, 3]), dict(ptr=[0, 3, 7]), dict(ptr=[-1, 3, 6]),
                dict(pages=[5, -1]), dict(pages=[5, c.table.shape[1] + 1]),
                dict(pages=[5, c.table.shape[1]]), dict(rows=bad_row)):
        status = K.new_status()
        K.paged_prefix_attn(q, c.kd, c.vd, c.pool, i32(bad.get("ptr", ptr)),
                            i32(bad.get("pages", [5, 5])),
                            group_rows=i32(bad["rows"]) if "rows" in bad else None, status=status)
        assert K.read_status(status) in (K.ERR_INVALID_ARG, K.ERR_BAD_BLOCK), bad
    c.table[0, 2] = -1
    status = K.new_status()
    K.paged_prefix_attn(q, c.kd, c.vd, c.make_pool(), i32(ptr), i32([5, 5]), status=status)
    assert K.read_status(status) == K.ERR_BAD_BLOCK


# ------------------------------------------------------------------------------------ together

def test_decode_loop_with_the_operators():
    """A prompt enters the cache of four samples that share its whole pages, then steps run:
    blocks, rotary append with bounds and ring, shared-prefix and block-sparse attention of the
    new token, lengths; in the middle a window compression with its bounds refreshed."""
    batch, hq, hkv, d, w, keep, steps = 4, 14, 2, 128, 32, 8, 45
    prompt = 16 * 6
    gen = torch.Generator().manual_seed(61)
    num_blocks, width = 120, 20
    dev = dict(device="cuda")
    table = np.full((batch, width), -1, dtype=np.int64)
    table[:, :6] = np.arange(6)
    pool = K.PagedPool(i32(table), i32([0] * batch), i32(np.arange(num_blocks - 1, -1, -1)),
                       i32([num_blocks - 6]), num_blocks, hkv, d)
    kd = torch.zeros((num_blocks, PAGE, hkv, d), dtype=torch.bfloat16, **dev)
    vd = torch.zeros_like(kd)
    bounds = torch.zeros((num_blocks, hkv, 2, d), dtype=torch.bfloat16, **dev)
    ring = torch.zeros((batch, 2 * w, hq, d), dtype=torch.bfloat16, **dev)
    tail, due, count = i32([0] * batch), i32([0] * batch), i32([0])
    status, freq = K.new_status(), inv_freq(d)
    x = bf16(gen, prompt, hq + 2 * hkv, d)
    xd = x.cuda()
    # the prompt once, through the first row
    K.paged_rope_append(xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:], kd, vd, pool,
                        freq.cuda(), i32(np.arange(prompt)),
                        cu_tokens=i32([0] + [prompt] * batch), bounds=bounds, status=status)
    pool.ctx_len.fill_(prompt)
    position = np.full(batch, prompt)
    compressed = 0
    for step in range(steps):
        K.kara_step_begin(pool, status)
        x = bf16(gen, batch, hq + 2 * hkv, d).cuda()
        q = K.paged_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], kd, vd, pool,
                                freq.cuda(), i32(position), bounds=bounds, q_ring=ring, window=w,
                                status=status)
        shared = K.paged_prefix_attn(q, kd, vd, pool, i32([0, batch]), i32([6]), new_slots=1,
                                     status=status)
        sel = torch.empty((batch, hkv, 5), dtype=torch.int32, **dev)
        sparse = K.paged_sparse_attn(q, kd, vd, bounds, pool, 5, new_slots=1, sel=sel,
                                     status=status)
        lengths = H.i32(pool.ctx_len) + 1
        tab = H.i32(pool.block_table)
        ref, mag = op.dense_attention(H.f64(q), H.f64(kd), H.f64(vd), tab, lengths,
                                      1 / math.sqrt(d), PAGE)
        attention_close(shared, ref, mag)
        want = op.page_bounds(H.f64(kd), tab, lengths, None, H.f64(bounds), PAGE)
        assert np.array_equal(H.f64(bounds), want)   # up to date at every step
        for b in range(batch):
            s = op.page_scores(H.f64(q[b]), want, tab[b, :-(-int(lengths[b]) // PAGE)])
            for g in range(hkv):
                assert np.array_equal(H.i32(sel[b, g]), op.select_pages(s[g], 5, 1, 2))
        ref, mag = op.sparse_attention(H.f64(q), H.f64(kd), H.f64(vd), H.i32(sel), tab, lengths,
                                       1 / math.sqrt(d), PAGE)
        attention_close(sparse, ref, mag)
        K.kara_step_end(pool, tail, w, step % 10 == 9, due, count)
        position += 1
        n_due = int(count.item()) if step % 10 == 9 else 0
        if n_due:
            ids = due[:n_due].contiguous()
            scores = K.kara_score_ring(ring, kd, pool, w, ids, n_due, status=status)
            kept = K.kara_select_chunks(scores, keep, 0.5, 8, 1)
            start = (pool.ctx_len - w).clone()
            K.kara_compact([kd], [vd], pool, w, kept[None], seq_ids=ids, status=status)
            K.paged_page_bounds(kd, pool, bounds=bounds, from_slot=start, status=status)
            K.kara_reset_tails(tail, ids, n_due)
            compressed += n_due
        assert K.read_status(status) == 0, step
    assert compressed == batch


def test_on_another_stream_and_captured():
    """Each call on a side stream without synchronising first against its allocations, and a
    captured step replayed on new inputs."""
    c, ptr = prefix_cache(62, [4, 2], [7, 3], 2, 128, least=2)
    q = bf16(c.gen, 6, 8, 128).cuda()
    gp, pp = i32(ptr), i32([7, 3])
    x = bf16(c.gen, 6, 12, 128).cuda()
    pos, freq = i32(np.arange(6)), inv_freq(128).cuda()
    bounds = c.bounds().cuda()

    def step(stream=None):
        r = K.paged_rope_append(x[:, :8], x[:, 8:10], x[:, 10:], c.kd, c.vd, c.pool, freq, pos,
                                bounds=bounds, stream=stream)
        b = K.paged_page_bounds(c.kd, c.pool, new_slots=1, stream=stream)
        s = K.paged_sparse_attn(q, c.kd, c.vd, bounds, c.pool, 4, new_slots=1, stream=stream)
        p = K.paged_prefix_attn(q, c.kd, c.vd, c.pool, gp, pp, new_slots=1, stream=stream)
        return r, b, s, p

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        junk = torch.full((1 << 22,), 3.0, device="cuda")    # reused by careless allocation
        got = step(side)
        del junk
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    q.copy_(bf16(c.gen, 6, 8, 128))
    x.copy_(bf16(c.gen, 6, 12, 128))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in out]
    for a, b in zip(replayed, step()):
        assert torch.equal(a, b)


# ------------------------------------------------------------------- far ends and odd callers

@pytest.mark.parametrize("kind", ["random", "equal", "two_values"])
@pytest.mark.parametrize("pages", [4500, 33000])
def test_sparse_selection_over_many_pages(pages, kind):
    """More pages than the selection keeps in shared memory, and hundreds of equal scores."""
    d, keep = 64, 700
    n = pages * PAGE - 7
    gen = torch.Generator().manual_seed(71)
    c = Cache(71, [16, n], 1, d)
    if kind == "equal":
        c.k[:] = c.k[0:1]
    elif kind == "two_values":
        c.k[:] = torch.where(torch.rand(c.num_blocks, 1, 1, 1, generator=gen) < 0.5, 1.0, -1.0)
    c.kd = c.k.cuda()
    q = bf16(gen, 2, 3, d)
    bounds = c.bounds()
    sel = torch.empty((2, 1, keep), dtype=torch.int32, device="cuda")
    status = K.new_status()
    out = K.paged_sparse_attn(q.cuda(), c.kd, c.vd, bounds.cuda(), c.pool, keep, sel=sel,
                              status=status)
    assert K.read_status(status) == 0
    for b, m in enumerate(c.lengths):
        s = op.page_scores(H.f64(q[b]), H.f64(bounds), c.table[b, :-(-int(m) // PAGE)])
        assert np.array_equal(H.i32(sel[b, 0]), op.select_pages(s[0], keep, 1, 2))
    ref, mag = op.sparse_attention(H.f64(q), c.k.float().numpy(), c.v.float().numpy(),
                                   H.i32(sel), c.table, c.lengths, 0.125, PAGE)
    attention_close(out, ref, mag)


def test_blocks_behind_32_bit_offsets():
    """The same sequences in blocks far up a pool of more than 2^31 elements: bit for bit what
    they give in a small pool."""
    hkv, d, hq, far = 8, 128, 16, 140_000
    c, ptr = prefix_cache(72, [3, 2], [5, 2], hkv, d)
    i = dict(dtype=torch.int32, device="cuda")
    big = far + c.num_blocks
    assert far * PAGE * hkv * d > 2 ** 31
    kd = torch.empty((big, PAGE, hkv, d), dtype=torch.bfloat16, device="cuda")
    vd = torch.empty_like(kd)
    kd[far:], vd[far:] = c.kd, c.vd
    pool = K.PagedPool(torch.tensor(np.where(c.table >= 0, c.table + far, -1), **i),
                       c.pool.ctx_len, torch.zeros(big, **i), c.pool.free_top, big, hkv, d)
    x = bf16(c.gen, 5, hq + 2 * hkv, d).cuda()
    args = (inv_freq(d).cuda(), i32(np.arange(5) * 1000))
    results = []
    for k, v, p in ((c.kd, c.vd, c.pool), (kd, vd, pool)):
        status = K.new_status()
        bounds = K.paged_page_bounds(k, p, status=status)
        q = K.paged_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], k, v, p, *args,
                                bounds=bounds, status=status)
        results.append((q, K.paged_sparse_attn(q, k, v, bounds, p, 4, new_slots=1, status=status),
                        K.paged_prefix_attn(q, k, v, p, i32(ptr), i32([5, 2]), new_slots=1,
                                            status=status),
                        bounds[-c.num_blocks:], k[-c.num_blocks:], v[-c.num_blocks:]))
        assert K.read_status(status) == 0
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_prefix_rows_outside_the_groups_and_empty_groups():
    c, _ = prefix_cache(73, [2, 3], [4, 6], 2, 64)
    q = bf16(c.gen, 5, 4, 64)
    for ptr in ([0, 0, 0], [5, 5, 5], [2, 2, 5], [2, 5, 5]):
        pages = [4, 6] if ptr[1] == ptr[0] else [6, 4]
        out = torch.full((5, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        status = K.new_status()
        K.paged_prefix_attn(q.cuda(), c.kd, c.vd, c.pool, i32(ptr), i32(pages), out=out,
                            status=status)
        assert K.read_status(status) == 0
        rows = np.arange(ptr[0], ptr[2])
        if len(rows):
            ref, mag = op.dense_attention(H.f64(q), H.f64(c.k), H.f64(c.v), c.table, c.lengths,
                                          0.125, PAGE)
            attention_close(out[rows], ref[rows], mag[rows])
        rest = [r for r in range(5) if r not in rows]
        assert (out[rest] == 3).all()


def test_nan_in_a_key_reaches_its_rows_only():
    """A NaN key inside the prefix makes the outputs of its group and KV head NaN, a NaN among a
    row's own keys those of the row; the others keep their values."""
    c, ptr = prefix_cache(74, [3, 3], [6, 6], 2, 128, least=20)
    q = bf16(c.gen, 6, 4, 128)
    good = check_prefix(c, q, ptr, [6, 6])
    c.kd[int(c.table[0, 3]), 5, 0] = float("nan")           # group 0, KV head 0
    c.kd[int(c.table[4, 6]), 1, 1] = float("nan")           # row 4's first own page, KV head 1
    got = K.paged_prefix_attn(q.cuda(), c.kd, c.vd, c.pool, i32(ptr), i32([6, 6]))
    bad = torch.zeros((6, 4), dtype=torch.bool, device="cuda")
    bad[:3, :2] = True
    bad[4, 2:] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], good[~bad])


def test_two_calls_at_once_and_no_room():
    """Calls on two streams at the same time, each with what it allocates itself."""
    c, ptr = prefix_cache(75, [40, 30], [60, 30], 2, 128, least=3)
    q = [bf16(c.gen, 70, 8, 128).cuda() for _ in range(2)]
    bounds = c.bounds().cuda()
    gp, pp = i32(ptr), i32([60, 30])
    want = [(K.paged_prefix_attn(x, c.kd, c.vd, c.pool, gp, pp),
             K.paged_sparse_attn(x, c.kd, c.vd, bounds, c.pool, 12)) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for s in range(2):
            got[s].append((K.paged_prefix_attn(q[s], c.kd, c.vd, c.pool, gp, pp, stream=streams[s]),
                           K.paged_sparse_attn(q[s], c.kd, c.vd, bounds, c.pool, 12,
                                               stream=streams[s])))
    torch.cuda.synchronize()
    for s in range(2):
        for pair in got[s]:
            assert torch.equal(pair[0], want[s][0]) and torch.equal(pair[1], want[s][1])
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for call in (lambda: K.paged_prefix_attn(q[0], c.kd, c.vd, c.pool, gp, pp, workspace=small),
                 lambda: K.paged_sparse_attn(q[0], c.kd, c.vd, bounds, c.pool, 12,
                                             workspace=small)):
        with pytest.raises(K.KaraError, match="workspace"):
            call()


def test_binding_refuses_tensors_that_do_not_fit():
    c = Cache(76, [20, 40], 2, 64, room=4)
    x = bf16(c.gen, 2, 8, 64).cuda()
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    freq, pos = inv_freq(64).cuda(), i32([1, 2])
    bounds = c.bounds().cuda()
    qc = q.contiguous()
    gp, pp = i32([0, 2]), i32([1])

    def append(**kw):
        a = dict(q=q, k=k, v=v, k_cache=c.kd, v_cache=c.vd, pool=c.pool, inv_freq=freq,
                 positions=pos)
        a.update(kw)
        return K.paged_rope_append(**a)

    def sparse(**kw):
        a = dict(q=qc, k_cache=c.kd, v_cache=c.vd, bounds=bounds, pool=c.pool, num_pages=4)
        a.update(kw)
        return K.paged_sparse_attn(**a)

    def prefix(**kw):
        a = dict(q=qc, k_cache=c.kd, v_cache=c.vd, pool=c.pool, group_ptr=gp, prefix_pages=pp)
        a.update(kw)
        return K.paged_prefix_attn(**a)

    wide = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")[..., :64]
    for call, bad in (
            (append, dict(q=wide)), (append, dict(q=q.float())), (append, dict(k=k[:1])),
            (append, dict(positions=pos[:1])), (append, dict(positions=pos.long())),
            (append, dict(inv_freq=freq[::2])), (append, dict(cu_tokens=i32([0, 1]))),
            (append, dict(k_cache=c.kd[:-1])), (append, dict(v_cache=c.vd.transpose(1, 2))),
            (append, dict(q_out=qc[:1])), (append, dict(bounds=bounds[:, :1])),
            (append, dict(q_ring=bounds, window=4)), (append, dict(status=pos.long())),
            (append, dict(q=q.cpu())), (append, dict(window=2 ** 40)),
            (sparse, dict(q=q)), (sparse, dict(sel=i32([1]))), (sparse, dict(out=qc[:1])),
            (sparse, dict(bounds=bounds.float())), (sparse, dict(workspace=pos)),
            (prefix, dict(group_ptr=i32([0, 1, 2]))), (prefix, dict(group_rows=i32([0]))),
            (prefix, dict(prefix_pages=pp.long())), (prefix, dict(q=qc.cpu()))):
        with pytest.raises(ValueError):
            call(**bad)
    for call, bad in ((append, dict(inv_freq=freq[:4].contiguous())), (sparse, dict(num_pages=2)),
                      (sparse, dict(scale=-1.0)), (prefix, dict(new_slots=-1))):
        with pytest.raises(K.KaraError):
            call(**bad)
    given = torch.empty_like(qc)
    assert sparse(out=given) is given and prefix(out=given) is given


def test_prefix_items_of_one_and_of_two_teams_in_turn():
    """Groups of 2 and of 40 rows by turns, several per block: items for one tensor-core tile
    follow items for two and the other way round. Run a few times: the result does not depend on
    who is ahead."""
    rows = [2, 40] * 24
    pages = [11, 9, 17, 24] * 12
    c, ptr = prefix_cache(77, rows, pages, 4, 128)
    q = bf16(c.gen, len(c.lengths), 32, 128)
    out = check_prefix(c, q, ptr, pages)
    for _ in range(20):
        again = K.paged_prefix_attn(q.cuda(), c.kd, c.vd, c.pool, i32(ptr), i32(pages))
        assert torch.equal(out, again)


def test_prefix_of_many_small_groups():
    """More groups than the plan keeps in shared memory, rows of one slot and of none."""
    rows = [1 + i % 3 for i in range(300)]
    pages = [(i * 7) % 5 for i in range(300)]
    c, ptr = prefix_cache(78, rows, pages, 1, 64)
    q = bf16(c.gen, len(c.lengths), 5, 64)
    check_prefix(c, q, ptr, pages)


def test_calls_in_a_row_share_a_workspace():
    """Calls of other shapes and lengths follow each other in one stream and one workspace, with no
    wait in between: a kernel starts before the one it follows has ended."""
    big = Cache(79, [900, 40, 3000, 700], 4, 128, room=32)
    small = Cache(80, [2500, 17], 2, 64, room=32)
    shared, ptr = prefix_cache(81, [9, 4], [30, 11], 2, 128)
    qb, qs, qp = (bf16(x.gen, len(x.lengths), h, x.d).cuda()
                  for x, h in ((big, 28), (small, 4), (shared, 8)))
    bb, bs = big.bounds().cuda(), small.bounds().cuda()
    gp, pp = i32(ptr), i32([30, 11])
    sel_b = torch.empty(4, 4, 20, dtype=torch.int32, device="cuda")
    sel_s = torch.empty(2, 2, 7, dtype=torch.int32, device="cuda")

    def sweep(**kw):
        out = []
        for step in range(6):
            for new in (0, 1):
                out.append(K.paged_sparse_attn(qb, big.kd, big.vd, bb, big.pool, 20, 1, 2,
                                               new_slots=new, sel=sel_b, **kw))
                out.append(sel_b.clone())
                out.append(K.paged_sparse_attn(qs, small.kd, small.vd, bs, small.pool, 7,
                                               new_slots=new, sel=sel_s, **kw))
                out.append(K.paged_prefix_attn(qp, shared.kd, shared.vd, shared.pool, gp, pp,
                                               new_slots=new, **kw))
                out.append(K.paged_sparse_attn(qb, big.kd, big.vd, bb, big.pool, 300, **kw))
                if "workspace" not in kw:
                    torch.cuda.synchronize()
            big.pool.ctx_len.add_(3)
            small.pool.ctx_len.add_(5)
        big.pool.ctx_len.sub_(18)
        small.pool.ctx_len.sub_(30)
        torch.cuda.synchronize()
        return out

    want = sweep()
    room = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(10):
        for a, b in zip(sweep(workspace=room), want):
            assert torch.equal(a, b)
