"""Oracle (fp64, CPU) of the operators around the paged cache: rotary append, page key bounds,
block-sparse page selection and attention, shared-prefix attention.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definitions: include/kara.h (paged_rope_append, paged_page_bounds, paged_sparse_attn,
paged_prefix_attn). Shared-prefix attention is ordinary decode attention over every row's own
table, so its oracle is that of decode attention with the lengths advanced by new_slots.

Parity pins (tests/test_oracle_paged_ops.py): a rotation keeps a pair's norm, composes by adding
positions and leaves q . k dependent on the distance only; the two channel layouts are
permutations of each other; a page's score bounds every logit of its keys; with every page
selected sparse attention is decode attention; equal scores select the lowest pages.
"""

from __future__ import annotations

import numpy as np


def rotate(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray,
           interleaved: bool) -> np.ndarray:
    """x [T, H, d] float64 rotated by positions [T]; inv_freq [rotary_dim / 2]."""
    half = len(inv_freq)
    angle = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)[None, :]
    c, s = np.cos(angle)[:, None, :], np.sin(angle)[:, None, :]
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    out = x.copy()
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., second] * c + x[..., first] * s
    return out


def append_slots(ctx_len: np.ndarray, cu_tokens: np.ndarray) -> np.ndarray:
    """(token row, sequence, slot) of every token, [T', 3]."""
    out = []
    for b in range(len(ctx_len)):
        for i, t in enumerate(range(int(cu_tokens[b]), int(cu_tokens[b + 1]))):
            out.append((t, b, int(ctx_len[b]) + i))
    return np.array(out, dtype=np.int64).reshape(-1, 3)


def page_bounds(k_pool: np.ndarray, block_table: np.ndarray, lengths: np.ndarray,
                from_slot: np.ndarray | None, bounds: np.ndarray, page: int) -> np.ndarray:
    """bounds [num_blocks, Hkv, 2, d] with the complete pages' entries replaced."""
    out = bounds.copy()
    for b in range(len(lengths)):
        first = 0 if from_slot is None else max(int(from_slot[b]), 0) // page
        for p in range(first, int(lengths[b]) // page):
            blk = block_table[b, p]
            out[blk, :, 0] = k_pool[blk].min(axis=0)
            out[blk, :, 1] = k_pool[blk].max(axis=0)
    return out


def page_scores(q: np.ndarray, bounds: np.ndarray, blocks: np.ndarray) -> np.ndarray:
    """q [Hq, d], bounds of the pages `blocks`: scores [Hkv, pages]."""
    hkv = bounds.shape[1]
    g = q.shape[0] // hkv
    out = np.full((hkv, len(blocks)), -np.inf)
    for kv in range(hkv):
        lo, hi = bounds[blocks, kv, 0], bounds[blocks, kv, 1]
        for h in range(kv * g, (kv + 1) * g):
            out[kv] = np.maximum(out[kv], np.maximum(q[h] * lo, q[h] * hi).sum(axis=1))
    return out


def select_pages(scores: np.ndarray, num_pages: int, sink: int, recent: int) -> np.ndarray:
    """scores [pages] of one KV head -> num_pages page numbers, ascending, -1 behind them."""
    n = len(scores)
    out = np.full(num_pages, -1, dtype=np.int64)
    if n <= num_pages:
        out[:n] = np.arange(n)
        return out
    free = np.arange(sink, n - recent)
    best = free[np.argsort(-scores[free], kind="stable")[:num_pages - sink - recent]]
    out[:] = np.sort(np.concatenate([np.arange(sink), best, np.arange(n - recent, n)]))
    return out


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float):
    """q [d], k and v [n, d]: the output and sum of weight * |v| (the error's scale)."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), np.zeros(v.shape[1])
    s = (k @ q) * scale
    e = np.exp(s - s.max())
    w = e / e.sum()
    return w @ v, w @ np.abs(v)


def sparse_attention(q: np.ndarray, k_pool: np.ndarray, v_pool: np.ndarray, sel: np.ndarray,
                     block_table: np.ndarray, lengths: np.ndarray, scale: float, page: int):
    """q [B, Hq, d] over the selected pages sel [B, Hkv, num_pages]: out and weight * |v|."""
    nb, hq, d = q.shape
    hkv = k_pool.shape[2]
    out, mag = np.zeros((nb, hq, d)), np.zeros((nb, hq, d))
    for b in range(nb):
        for h in range(hq):
            g = h // (hq // hkv)
            pages = sel[b, g][sel[b, g] >= 0]
            slots = (pages[:, None] * page + np.arange(page)).ravel()
            slots = slots[slots < lengths[b]]
            blk = block_table[b][slots // page]
            out[b, h], mag[b, h] = attend(q[b, h], k_pool[blk, slots % page, g],
                                          v_pool[blk, slots % page, g], scale)
    return out, mag


def dense_attention(q: np.ndarray, k_pool: np.ndarray, v_pool: np.ndarray,
                    block_table: np.ndarray, lengths: np.ndarray, scale: float, page: int):
    """Attention over all slots of every row: out and weight * |v|."""
    pages = max(1, -(-int(max(lengths)) // page))
    sel = np.full((len(lengths), k_pool.shape[2], pages), -1, dtype=np.int64)
    for b, n in enumerate(lengths):
        sel[b, :, :-(-int(n) // page)] = np.arange(-(-int(n) // page))
    return sparse_attention(q, k_pool, v_pool, sel, block_table, lengths, scale, page)
