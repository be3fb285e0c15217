"""Cases for the operators around a paged decode cache, with their plain forms.

Operators: ``paged_rope_append`` (new tokens rotated by position and written to the paged cache),
``paged_page_bounds`` (elementwise minimum and maximum of every page's keys), ``paged_sparse_attn``
(decode attention over the pages that a bound on the logits selects) and ``paged_prefix_attn``
(decode attention of rows that share their first pages). Head layouts, page size and context
lengths are those of the workloads in ``decode_kv_cache_kara_b200.synth``.

A case's lengths come from its ``layout`` number, its values from the seed.
"""

from __future__ import annotations

import math
import random

import torch

own = False

PAGE = 16


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence decoding one token, 8B-class heads: latency of a single call
        {"name": "append_one", "op": "append", "batch": 1, "hq": 32, "hkv": 8, "d": 128, "rd": 128,
         "interleaved": False, "ctx_lo": 4000, "ctx_hi": 4000, "new_lo": 1, "new_hi": 1,
         "bounds": False, "packed": True, "layout": 1},
        # a decode step of a full batch whose sequences were compressed (positions run ahead of
        # the slots), bounds of completed pages on the way
        {"name": "append_step", "op": "append", "batch": 128, "hq": 28, "hkv": 4, "d": 128,
         "rd": 128, "interleaved": False, "ctx_lo": 256, "ctx_hi": 2048, "new_lo": 1, "new_hi": 1,
         "bounds": True, "packed": True, "layout": 2},
        # prompts of six requests, ragged and unaligned, entering the cache in one call
        {"name": "append_prompts", "op": "append", "batch": 6, "hq": 28, "hkv": 4, "d": 128,
         "rd": 128, "interleaved": False, "ctx_lo": 0, "ctx_hi": 100, "new_lo": 500,
         "new_hi": 4096, "bounds": True, "packed": True, "layout": 3},
        # short continuations (a turn's few tokens) of many chats, rotation of neighbouring
        # channels on half of a small head
        {"name": "append_turns", "op": "append", "batch": 37, "hq": 16, "hkv": 2, "d": 64,
         "rd": 32, "interleaved": True, "ctx_lo": 1, "ctx_hi": 900, "new_lo": 0, "new_hi": 61,
         "bounds": False, "packed": False, "layout": 4},
        # after a window compression: the bounds of the rewritten pages of 32 sequences
        {"name": "bounds_window", "op": "bounds", "batch": 32, "hkv": 4, "d": 128, "ctx_lo": 3200,
         "ctx_hi": 3330, "tail": 220, "layout": 5},
        # a cache of ragged contexts, every page
        {"name": "bounds_cache", "op": "bounds", "batch": 64, "hkv": 4, "d": 128, "ctx_lo": 2048,
         "ctx_hi": 16384, "tail": -1, "layout": 6},
        # one long sequence, 8 KV heads: 128 of about 4000 pages
        {"name": "sparse_one", "op": "sparse", "batch": 1, "hq": 32, "hkv": 8, "d": 128,
         "ctx_lo": 65000, "ctx_hi": 65000, "pages": 128, "sink": 1, "recent": 4, "new_slots": 0,
         "layout": 7},
        # one 7B-class layer: batch 32, 4096-token caches, a quarter of the pages
        {"name": "sparse_layer", "op": "sparse", "batch": 32, "hq": 28, "hkv": 4, "d": 128,
         "ctx_lo": 4090, "ctx_hi": 4100, "pages": 64, "sink": 1, "recent": 2, "new_slots": 1,
         "layout": 8},
        # the step workload's batch: 128 ragged contexts of 2K to 16K tokens
        {"name": "sparse_step", "op": "sparse", "batch": 128, "hq": 28, "hkv": 4, "d": 128,
         "ctx_lo": 2048, "ctx_hi": 16384, "pages": 128, "sink": 4, "recent": 8, "new_slots": 1,
         "layout": 9},
        # eight samples of one prompt, early in their answers
        {"name": "prefix_samples", "op": "prefix", "groups": 1, "rows_lo": 8, "rows_hi": 8,
         "hq": 28, "hkv": 4, "d": 128, "prefix_lo": 1024, "prefix_hi": 1024, "suffix_lo": 1,
         "suffix_hi": 300, "new_slots": 1, "layout": 10},
        # sixteen prompts of different lengths with a few samples each, and rows on their own
        {"name": "prefix_groups", "op": "prefix", "groups": 16, "rows_lo": 1, "rows_hi": 15,
         "hq": 32, "hkv": 8, "d": 128, "prefix_lo": 0, "prefix_hi": 8192, "suffix_lo": 1,
         "suffix_hi": 2048, "new_slots": 0, "layout": 11},
        # a full batch behind one long shared document
        {"name": "prefix_batch", "op": "prefix", "groups": 1, "rows_lo": 128, "rows_hi": 128,
         "hq": 28, "hkv": 4, "d": 128, "prefix_lo": 32768, "prefix_hi": 32768, "suffix_lo": 64,
         "suffix_hi": 2048, "new_slots": 1, "layout": 12},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """A case of the listed ones' ranges, no larger than the largest of them."""
    while True:
        case = _draw(rng)
        cost = work(case)
        if cost["bytes"] <= 600e6 and cost["flops"] <= 50e9:
            return case


def _draw(rng):
    op = rng.choice(["append", "append", "bounds", "sparse", "sparse", "prefix", "prefix"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 4, 8])
    hq = hkv * rng.randint(1, 8)
    case = {"op": op, "hkv": hkv, "d": d, "layout": rng.randrange(1 << 20)}
    if op == "append":
        batch = _log_int(rng, 1, 128)
        most = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, 12000 // batch))
        case.update(batch=batch, hq=hq, rd=rng.choice([d, d, d // 2]),
                    interleaved=rng.random() < 0.3, ctx_lo=0, ctx_hi=_log_int(rng, 16, 2000),
                    new_lo=1 if most == 1 else rng.choice([0, 1, most // 2]), new_hi=most,
                    bounds=rng.random() < 0.5, packed=rng.random() < 0.6)
    elif op == "bounds":
        batch = _log_int(rng, 1, 64)
        top = _log_int(rng, 64, 14000)
        case.update(batch=batch, ctx_lo=top // rng.choice([1, 2, 8]), ctx_hi=top,
                    tail=rng.choice([-1, 1, _log_int(rng, 2, top)]))
    elif op == "sparse":
        batch = _log_int(rng, 1, 96)
        top = _log_int(rng, 40, min(65000, 1200000 // batch))
        case.update(batch=batch, hq=hq, ctx_lo=top // rng.choice([1, 2, 6]), ctx_hi=top,
                    pages=_log_int(rng, 6, 160), sink=rng.randint(0, 2),
                    recent=rng.randint(1, 4), new_slots=rng.randint(0, 1))
    else:
        groups = _log_int(rng, 1, 24)
        most = _log_int(rng, 1, max(1, 96 // groups))
        top = _log_int(rng, 16, 32000 // groups + 16)
        case.update(groups=groups, rows_lo=max(1, most // rng.choice([1, 3])), rows_hi=most, hq=hq,
                    prefix_lo=top // rng.choice([1, 2, 16]), prefix_hi=top,
                    suffix_lo=rng.choice([0, 1, 33]), suffix_hi=_log_int(rng, 40, 1800),
                    new_slots=rng.randint(0, 1))
    return case


def _span(rng, case, what):
    return rng.randint(case[what + "_lo"], case[what + "_hi"])


def _append_lens(case):
    rng = random.Random(case["layout"])
    ctx = [_span(rng, case, "ctx") for _ in range(case["batch"])]
    new = [_span(rng, case, "new") for _ in range(case["batch"])]
    if not any(new):
        new[-1] = 1
    return ctx, new


def _ctx_lens(case):
    rng = random.Random(case["layout"])
    return [_span(rng, case, "ctx") for _ in range(case["batch"])]


def _prefix_lens(case):
    """Rows per group, prefix pages per group, slots of every row behind its prefix."""
    rng = random.Random(case["layout"])
    rows = [_span(rng, case, "rows") for _ in range(case["groups"])]
    pages = [_span(rng, case, "prefix") // PAGE for _ in range(case["groups"])]
    suffix = [_span(rng, case, "suffix") for _ in range(sum(rows))]
    return rows, pages, suffix


# -------------------------------------------------------------------------------- preparation

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(counts, seed, spare=3):
    """Block tables of rows with these page counts over a permuted pool, as lists."""
    rng = random.Random(seed * 7919 + 17)
    num_blocks = sum(counts) + spare
    ids = list(range(num_blocks))
    rng.shuffle(ids)
    table, pos = [], 0
    width = max(counts) + 1
    for c in counts:
        table.append(ids[pos:pos + c] + [-1] * (width - c))
        pos += c
    return table, num_blocks


def _keys(gen, num_blocks, hkv, d):
    """Keys of a cache: runs of strong keys among ordinary ones, as in the synthetic workloads."""
    k = torch.randn((num_blocks, PAGE, hkv, d), generator=gen, device="cuda")
    strong = torch.rand((num_blocks, 1, hkv, 1), generator=gen, device="cuda") < 0.03
    return torch.where(strong, 4 * k, k).to(torch.bfloat16)


def _pool(state, table, ctx, num_blocks, hkv, d):
    state.update(block_table=_ints(table), ctx_len=_ints(ctx), num_blocks=num_blocks, hkv=hkv, d=d)
    state["free_list"] = torch.zeros(num_blocks, dtype=torch.int32, device="cuda")
    state["free_top"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def _library(state):
    """The handle that a user's program keeps: the pool and a workspace where the call takes one."""
    from decode_kv_cache_kara_b200 import kara as K
    pool = K.PagedPool(state["block_table"], state["ctx_len"], state["free_list"],
                       state["free_top"], state["num_blocks"], state["hkv"], state["d"])
    state["K"], state["pool"], state["status"] = K, pool, K.new_status()
    if state["op"] == "sparse":
        n = K.kara_workspace_bytes(K.OP_SPARSE, pool, 0, 0, state["hq"], state["pages"])
    elif state["op"] == "prefix":
        n = K.kara_workspace_bytes(K.OP_PREFIX, pool, 0, 0, state["hq"], 0)
    else:
        n = 0
    state["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"op": case["op"], "hkv": case["hkv"], "d": case["d"]}
    {"append": _prepare_append, "bounds": _prepare_bounds, "sparse": _prepare_sparse,
     "prefix": _prepare_prefix}[case["op"]](case, seed, gen, state)
    if own:
        _library(state)
    return state


def _prepare_append(case, seed, gen, state):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    ctx, new = _append_lens(case)
    table, nb = _tables([(c + n + PAGE - 1) // PAGE for c, n in zip(ctx, new)], seed)
    _pool(state, table, ctx, nb, hkv, d)
    rng = random.Random(seed)
    total = sum(new)
    seq, idx, pos, done = [], [], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        first = c + rng.randrange(0, 200000)      # slots dropped by earlier compressions
        seq += [b] * n
        idx += range(n)
        pos += range(first, first + n)
        done += [table[b][p] for p in range(c // PAGE, (c + n) // PAGE)]
    qkv = _normal(gen, total, hq + 2 * hkv, d)    # the projection's output: q, k, v heads
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not case["packed"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    state.update(
        q=q, k=k, v=v, positions=_ints(pos), interleaved=case["interleaved"], rd=case["rd"],
        inv_freq=torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
                           -torch.arange(0, case["rd"], 2, device="cuda").double() / case["rd"])
        .float(),
        cu_tokens=None if all(n == 1 for n in new) else _ints(cu),
        seq=_ints(seq).long(), idx=_ints(idx).long(), done=_ints(done).long(),
        k_cache=_normal(gen, nb, PAGE, hkv, d), v_cache=_normal(gen, nb, PAGE, hkv, d),
        bounds=torch.zeros((nb, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
        if case["bounds"] else None,
        q_out=torch.empty((total, hq, d), dtype=torch.bfloat16, device="cuda"))


def _prepare_bounds(case, seed, gen, state):
    ctx = _ctx_lens(case)
    table, nb = _tables([(c + PAGE - 1) // PAGE for c in ctx], seed)
    _pool(state, table, ctx, nb, case["hkv"], case["d"])
    first = [max(0, c - case["tail"]) if case["tail"] >= 0 else 0 for c in ctx]
    state.update(
        k_cache=_keys(gen, nb, case["hkv"], case["d"]),
        from_slot=_ints(first) if case["tail"] >= 0 else None,
        done=_ints([table[b][p] for b, c in enumerate(ctx)
                    for p in range(first[b] // PAGE, c // PAGE)]).long(),
        bounds=torch.zeros((nb, case["hkv"], 2, case["d"]), dtype=torch.bfloat16, device="cuda"))


def _prepare_sparse(case, seed, gen, state):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    ctx = _ctx_lens(case)
    length = [c + case["new_slots"] for c in ctx]
    table, nb = _tables([(n + PAGE - 1) // PAGE for n in length], seed)
    _pool(state, table, ctx, nb, hkv, d)
    k = _keys(gen, nb, hkv, d)
    # queries resemble some earlier key of their KV head, as a token that refers back does
    batch = case["batch"]
    at = (torch.rand((batch, hkv), generator=gen, device="cuda")
          * _ints([max(n // PAGE, 1) for n in length])[:, None]).long()
    blk = torch.gather(state["block_table"].long(), 1, at)
    near = k[blk, torch.randint(0, PAGE, (batch, hkv), generator=gen, device="cuda"),
             torch.arange(hkv, device="cuda")].float()
    q = near[:, :, None] + torch.randn((batch, hkv, hq // hkv, d), generator=gen, device="cuda")
    state.update(
        hq=hq, q=q.reshape(batch, hq, d).to(torch.bfloat16), k_cache=k,
        v_cache=_normal(gen, nb, PAGE, hkv, d),
        bounds=torch.stack([k.amin(1), k.amax(1)], 2).contiguous(), pages=case["pages"],
        sink=case["sink"], recent=case["recent"], new_slots=case["new_slots"],
        sel=torch.empty((batch, hkv, case["pages"]), dtype=torch.int32, device="cuda"),
        out=torch.empty((batch, hq, d), dtype=torch.bfloat16, device="cuda"))


def _prepare_prefix(case, seed, gen, state):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows, pages, suffix = _prefix_lens(case)
    new = case["new_slots"]
    suffix = [max(s, new) for s in suffix]
    own_pages = [(s + PAGE - 1) // PAGE for s in suffix]
    table, nb = _tables([p for p in pages] + own_pages, seed)
    shared, private = table[:len(pages)], table[len(pages):]
    group = [j for j, r in enumerate(rows) for _ in range(r)]
    width = max(pages[j] + own_pages[i] for i, j in enumerate(group)) + 1
    rowtab = []
    for i, j in enumerate(group):
        ids = shared[j][:pages[j]] + private[i][:own_pages[i]]
        rowtab.append(ids + [-1] * (width - len(ids)))
    ctx = [pages[j] * PAGE + suffix[i] - new for i, j in enumerate(group)]
    _pool(state, rowtab, ctx, nb, hkv, d)
    ptr = [0]
    for r in rows:
        ptr.append(ptr[-1] + r)
    most = max(rows)
    # the groups padded to one size, for the plain form
    pad = [[min(ptr[j] + i, ptr[j + 1] - 1) for i in range(most)] for j in range(len(rows))]
    back = [j * most + i - ptr[j] for i, j in enumerate(group)]
    deep, wide = max(max(pages), 1), max(max(own_pages), 1)
    state.update(
        hq=hq, q=_normal(gen, len(group), hq, d), k_cache=_keys(gen, nb, hkv, d),
        v_cache=_normal(gen, nb, PAGE, hkv, d), group_ptr=_ints(ptr), prefix_pages=_ints(pages),
        new_slots=new, pad=_ints(pad).long(), back=_ints(back).long(),
        shared=_ints([(s[:p] + [0] * deep)[:deep] for s, p in zip(shared, pages)]).long(),
        private=_ints([(s[:p] + [0] * wide)[:wide] for s, p in zip(private, own_pages)]).long(),
        suffix=_ints(suffix), out=torch.empty((len(group), hq, d), dtype=torch.bfloat16,
                                              device="cuda"))


# ------------------------------------------------------------------------------------- a pass

def run(state):
    if own:
        return {"append": _own_append, "bounds": _own_bounds, "sparse": _own_sparse,
                "prefix": _own_prefix}[state["op"]](state)
    return {"append": _plain_append, "bounds": _plain_bounds, "sparse": _plain_sparse,
            "prefix": _plain_prefix}[state["op"]](state)


def _own_append(s):
    s["K"].paged_rope_append(
        s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pool"], s["inv_freq"],
        s["positions"], cu_tokens=s["cu_tokens"], interleaved=s["interleaved"],
        bounds=s["bounds"], q_out=s["q_out"], status=s["status"])
    return _append_outputs(s)


def _own_bounds(s):
    return s["K"].paged_page_bounds(s["k_cache"], s["pool"], bounds=s["bounds"],
                                    from_slot=s["from_slot"], status=s["status"])


def _own_sparse(s):
    s["K"].paged_sparse_attn(
        s["q"], s["k_cache"], s["v_cache"], s["bounds"], s["pool"], s["pages"],
        sink_pages=s["sink"], recent_pages=s["recent"], new_slots=s["new_slots"], sel=s["sel"],
        out=s["out"], workspace=s["workspace"], status=s["status"])
    return {"out": s["out"], "sel": s["sel"]}


def _own_prefix(s):
    return s["K"].paged_prefix_attn(
        s["q"], s["k_cache"], s["v_cache"], s["pool"], s["group_ptr"], s["prefix_pages"],
        new_slots=s["new_slots"], out=s["out"], workspace=s["workspace"], status=s["status"])


def _append_outputs(s):
    out = {"q_out": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["bounds"] is not None:
        out["bounds"] = s["bounds"]
    return out


def _rotate(x, cos, sin, rd, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rd:]], -1).to(torch.bfloat16)


def _plain_append(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, s["rd"], s["interleaved"]))
    slot = s["ctx_len"].long()[s["seq"]] + s["idx"]
    blk = s["block_table"].long()[s["seq"], slot // PAGE]
    s["k_cache"][blk, slot % PAGE] = _rotate(s["k"], cos, sin, s["rd"], s["interleaved"])
    s["v_cache"][blk, slot % PAGE] = s["v"]
    if s["bounds"] is not None:
        _plain_bounds(s)
    return _append_outputs(s)


def _plain_bounds(s):
    page = s["k_cache"][s["done"]]
    s["bounds"][s["done"]] = torch.stack([page.amin(1), page.amax(1)], 2)
    return s["bounds"]


def _softmax_parts(logits, ok):
    """exp(logits - maximum) where ok, and the maximum (0 for a row with nothing)."""
    logits = torch.where(ok, logits, -torch.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    return torch.exp(logits - top), top


def _plain_sparse(s):
    batch, hq, d = s["q"].shape
    hkv, count = s["hkv"], s["pages"]
    g = hq // hkv
    length = s["ctx_len"].long() + s["new_slots"]
    pages = (length + PAGE - 1) // PAGE
    width = s["block_table"].shape[1]
    p = torch.arange(width, device="cuda")
    there = p < pages[:, None]
    bounds = s["bounds"][s["block_table"].long().clamp(min=0)].double()     # [B, P, Hkv, 2, d]
    q = s["q"].double().view(batch, hkv, g, d)
    score = (torch.einsum("bpkd,bkgd->bkgp", bounds[..., 0, :], q.clamp(max=0))
             + torch.einsum("bpkd,bkgd->bkgp", bounds[..., 1, :], q.clamp(min=0))).amax(2)
    fixed = there & ((p < s["sink"]) | (p >= (pages - s["recent"])[:, None]))
    score = torch.where(fixed[:, None], torch.inf, torch.where(there[:, None], score, -torch.inf))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :count]
    order = torch.cat([order, order.new_full((batch, hkv, max(0, count - width)), width)], -1)
    order = torch.where(order < pages[:, None, None], order, width)
    order = torch.sort(order, dim=-1).values
    s["sel"].copy_(torch.where(order < width, order, -1))
    safe = order.clamp(max=width - 1)
    blk = torch.gather(s["block_table"].long()[:, None].expand(-1, hkv, -1), 2, safe).clamp(min=0)
    head = torch.arange(hkv, device="cuda")[None, :, None]
    k = s["k_cache"].transpose(1, 2)[blk, head].float().flatten(2, 3)       # [B, Hkv, n, d]
    v = s["v_cache"].transpose(1, 2)[blk, head].float().flatten(2, 3)
    slot = (order[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(2)
    ok = (slot < length[:, None, None])[:, :, None]
    logits = s["q"].float().view(batch, hkv, g, d) @ k.transpose(-1, -2) / math.sqrt(d)
    e, _ = _softmax_parts(logits, ok)
    total = e.sum(-1, keepdim=True)
    out = (e @ v) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(out.reshape(batch, hq, d))
    return {"out": s["out"], "sel": s["sel"]}


def _plain_prefix(s):
    n, hq, d = s["q"].shape
    hkv = s["hkv"]
    g = hq // hkv
    scale = 1.0 / math.sqrt(d)
    q = s["q"].float().view(n, hkv, g, d)
    # the shared pages once per group
    groups, most = s["pad"].shape
    k = s["k_cache"][s["shared"]].float().flatten(1, 2).transpose(1, 2)     # [groups, Hkv, P, d]
    v = s["v_cache"][s["shared"]].float().flatten(1, 2).transpose(1, 2)
    qg = q[s["pad"]].permute(0, 2, 1, 3, 4).reshape(groups, hkv, most * g, d)
    slot = torch.arange(k.shape[2], device="cuda")
    ok = (slot < s["prefix_pages"][:, None] * PAGE)[:, None, None]
    e, m1 = _softmax_parts(qg @ k.transpose(-1, -2) * scale, ok)

    def rows(x):
        return x.view(groups, hkv, most, g, -1).transpose(1, 2).flatten(0, 1)[s["back"]]

    l1, o1, m1 = rows(e.sum(-1, keepdim=True)), rows(e @ v), rows(m1)
    # every row's own pages
    k = s["k_cache"][s["private"]].float().flatten(1, 2).transpose(1, 2)
    v = s["v_cache"][s["private"]].float().flatten(1, 2).transpose(1, 2)
    ok = (torch.arange(k.shape[2], device="cuda") < s["suffix"][:, None])[:, None, None]
    e, m2 = _softmax_parts(q @ k.transpose(-1, -2) * scale, ok)
    l2, o2 = e.sum(-1, keepdim=True), e @ v
    m1 = torch.where(l1 > 0, m1, -torch.inf)
    m2 = torch.where(l2 > 0, m2, -torch.inf)
    top = torch.maximum(m1, m2)
    top = torch.where(top == -torch.inf, 0.0, top)
    a, b = torch.exp(m1 - top), torch.exp(m2 - top)
    total = a * l1 + b * l2
    out = (a * o1 + b * o2) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(out.reshape(n, hq, d))
    return s["out"]


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "bounds": _exact_bounds, "sparse": _exact_sparse,
            "prefix": _exact_prefix}[case["op"]](case, s)


def _exact_append(case, s):
    rd = case["rd"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * s["inv_freq"].double()[None, :])[:, None]

    def rotated(x):
        x = x.double()
        y = x.clone()
        if case["interleaved"]:
            first, second = slice(0, rd, 2), slice(1, rd, 2)
        else:
            first, second = slice(0, rd // 2), slice(rd // 2, rd)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k, v = s["k_cache"].double(), s["v_cache"].double()
    knew = rotated(s["k"])
    table = s["block_table"].tolist()
    ctx, new = _append_lens(case)
    out, t = {"q_out": rotated(s["q"])}, 0
    blocks, rows, done = [], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        blocks += [table[b][(c + i) // PAGE] for i in range(n)]
        rows += [(c + i) % PAGE for i in range(n)]
        done += [table[b][p] for p in range(c // PAGE, (c + n) // PAGE)]
        t += n
    k[blocks, rows], v[blocks, rows] = knew, s["v"].double()
    out.update(k_cache=k, v_cache=v)
    if case["bounds"]:
        bounds = s["bounds"].double()
        if done:
            bounds[done, :, 0] = k[done].min(dim=1).values
            bounds[done, :, 1] = k[done].max(dim=1).values
        out["bounds"] = bounds
    return out


def _exact_bounds(case, s):
    bounds = s["bounds"].double()
    table = s["block_table"].tolist()
    for b, n in enumerate(_ctx_lens(case)):
        first = max(0, n - case["tail"]) if case["tail"] >= 0 else 0
        ids = table[b][first // PAGE:n // PAGE]
        if ids:
            page = s["k_cache"][ids].double()
            bounds[ids, :, 0] = page.min(dim=1).values
            bounds[ids, :, 1] = page.max(dim=1).values
    return bounds


def _attend(q, k, v, d):
    """q [Hkv, G, d], k and v [n, Hkv, d] in 64 bits: softmax attention, zeros where n = 0."""
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    w = torch.softmax(torch.einsum("kgd,nkd->kgn", q, k) / math.sqrt(d), -1)
    return torch.einsum("kgn,nkd->kgd", w, v)


def _exact_sparse(case, s):
    d, hkv, count = case["d"], case["hkv"], case["pages"]
    table = s["block_table"].tolist()
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    sel = torch.full_like(s["sel"], -1)
    for b, c in enumerate(_ctx_lens(case)):
        n = c + case["new_slots"]
        pages = (n + PAGE - 1) // PAGE
        if pages == 0:
            continue
        ids = torch.tensor(table[b][:pages], device="cuda")
        q = s["q"][b].double().view(hkv, -1, d)
        lo, hi = s["bounds"][ids].double().unbind(2)
        score = torch.stack([torch.maximum(q[:, h] * lo, q[:, h] * hi).sum(-1)
                             for h in range(q.shape[1])]).amax(0)            # [pages, Hkv]
        score[:case["sink"]] = math.inf
        score[max(0, pages - case["recent"]):] = math.inf
        for kv in range(hkv):
            order = torch.argsort(score[:, kv], descending=True, stable=True)[:count]
            pick = torch.sort(order).values
            sel[b, kv, :len(pick)] = pick
            slots = (pick[:, None] * PAGE + torch.arange(PAGE, device="cuda")) < n
            k = s["k_cache"][ids[pick], :, kv].double()[slots]
            v = s["v_cache"][ids[pick], :, kv].double()[slots]
            g = q.shape[1]
            out[b, kv * g:(kv + 1) * g] = _attend(q[kv:kv + 1], k[:, None], v[:, None], d)[0]
    return {"out": out, "sel": sel}


def _exact_prefix(case, s):
    d, hkv = case["d"], case["hkv"]
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    ctx = s["ctx_len"].tolist()
    for b, c in enumerate(ctx):
        n = c + case["new_slots"]
        ids = s["block_table"][b, :(n + PAGE - 1) // PAGE].long()
        k = s["k_cache"][ids].double().flatten(0, 1)[:n]
        v = s["v_cache"][ids].double().flatten(0, 1)[:n]
        out[b] = _attend(s["q"][b].double().view(hkv, -1, d), k, v, d).view(-1, d)
    return out


# ---------------------------------------------------------------------- bytes and operations

def work(case):
    d, hkv = case["d"], case["hkv"]
    row = hkv * d * 2                                         # one slot's K (or V) in bytes
    if case["op"] == "append":
        ctx, new = _append_lens(case)
        t, hq, rd = sum(new), case["hq"], case["rd"]
        nbytes = t * (2 * hq * d * 2 + 4 * row + 4) + rd * 2
        if case["bounds"]:
            for c, n in zip(ctx, new):
                done = (c + n) // PAGE - c // PAGE
                nbytes += done * 2 * row + (c % PAGE * row if done else 0)
        return {"bytes": nbytes, "flops": 3 * t * (hq + hkv) * rd}
    if case["op"] == "bounds":
        pages = 0
        for n in _ctx_lens(case):
            first = max(0, n - case["tail"]) if case["tail"] >= 0 else 0
            pages += max(0, n // PAGE - first // PAGE)
        return {"bytes": pages * (PAGE + 2) * row, "flops": 2 * pages * PAGE * hkv * d}
    hq = case["hq"]
    if case["op"] == "sparse":
        nbytes = flops = 0
        for c in _ctx_lens(case):
            n = c + case["new_slots"]
            pages = (n + PAGE - 1) // PAGE
            used = min(n, case["pages"] * PAGE)
            nbytes += 2 * used * row + 4 * hq * d + 4 * hkv * case["pages"]
            flops += 4 * used * hq * d
            if pages > case["pages"]:
                free = pages - case["sink"] - case["recent"]
                nbytes += free * 2 * row
                flops += 4 * free * hq * d
        return {"bytes": nbytes, "flops": flops}
    rows, pages, suffix = _prefix_lens(case)
    nbytes = flops = 0
    at = 0
    for r, p in zip(rows, pages):
        own_slots = sum(max(x, case["new_slots"]) for x in suffix[at:at + r])
        at += r
        nbytes += 2 * row * (p * PAGE + own_slots) + r * 4 * hq * d
        flops += 4 * hq * d * (r * p * PAGE + own_slots)
    return {"bytes": nbytes, "flops": flops}
