"""What the operators around the paged cache refuse on the host, before any launch (CPU)."""

import ctypes

import pytest
import torch

from decode_kv_cache_kara_b200 import kara as K

NULL, ONE = ctypes.c_void_p(0), ctypes.c_void_p(256)


def pool(**kw):
    f = dict(table=256, ctx=256, batch=3, width=64, blocks=64, page=16, hkv=2, d=128)
    f.update(kw)
    return K._Pool(f["table"], f["ctx"], 0, 0, f["batch"], f["width"], f["blocks"], f["page"],
                   f["hkv"], f["d"])


def append(**kw):
    f = dict(q=ONE, k=ONE, v=ONE, qs=512, ks=256, vs=256, t=3, cu=NULL, pos=ONE, freq=ONE, rd=128,
             kc=ONE, vc=ONE, pool=pool(), hq=4, bounds=NULL, ring=NULL, w=0, qo=ONE, ko=NULL,
             st=ONE)
    f.update(kw)
    return K.lib().paged_rope_append(f["q"], f["k"], f["v"], f["qs"], f["ks"], f["vs"], f["t"],
                                     f["cu"], f["pos"], f["freq"], f["rd"], 0, f["kc"], f["vc"],
                                     ctypes.byref(f["pool"]), f["hq"], f["bounds"], f["ring"],
                                     f["w"], f["qo"], f["ko"], f["st"], None)


def page_bounds(**kw):
    f = dict(kc=ONE, pool=pool(), frm=NULL, new=0, bounds=ONE, st=ONE)
    f.update(kw)
    return K.lib().paged_page_bounds(f["kc"], ctypes.byref(f["pool"]), f["frm"], f["new"],
                                     f["bounds"], f["st"], None)


def sparse(**kw):
    f = dict(q=ONE, kc=ONE, vc=ONE, bounds=ONE, pool=pool(), hq=4, scale=1.0, n=8, sink=1,
             recent=2, new=0, sel=NULL, out=ONE, ws=ONE, wsn=1 << 40, st=ONE)
    f.update(kw)
    return K.lib().paged_sparse_attn(f["q"], f["kc"], f["vc"], f["bounds"],
                                     ctypes.byref(f["pool"]), f["hq"], f["scale"], f["n"],
                                     f["sink"], f["recent"], f["new"], f["sel"], f["out"],
                                     f["ws"], f["wsn"], f["st"], None)


def prefix(**kw):
    f = dict(q=ONE, kc=ONE, vc=ONE, pool=pool(), hq=4, scale=1.0, ptr=ONE, pages=ONE, groups=2,
             rows=NULL, new=0, out=ONE, ws=ONE, wsn=1 << 40, st=ONE)
    f.update(kw)
    return K.lib().paged_prefix_attn(f["q"], f["kc"], f["vc"], ctypes.byref(f["pool"]), f["hq"],
                                     f["scale"], f["ptr"], f["pages"], f["groups"], f["rows"],
                                     f["new"], f["out"], f["ws"], f["wsn"], f["st"], None)


ODD = ctypes.c_void_p(264)       # not 16-byte aligned
INVALID = {
    append: [dict(t=2), dict(t=-1, cu=ONE), dict(q=NULL), dict(k=NULL), dict(v=NULL),
             dict(pos=NULL), dict(freq=NULL), dict(kc=NULL), dict(vc=NULL), dict(qo=NULL),
             dict(st=NULL), dict(q=ODD), dict(kc=ODD), dict(bounds=ODD), dict(ko=ODD),
             dict(qs=511), dict(qs=504), dict(ks=260), dict(vs=128), dict(ring=ONE, w=0),
             dict(ring=ONE, w=4097), dict(hq=5), dict(pool=pool(table=0))],
    page_bounds: [dict(kc=NULL), dict(bounds=NULL), dict(st=NULL), dict(bounds=ODD),
                  dict(new=-1), dict(new=64 * 16 + 1), dict(pool=pool(ctx=0))],
    sparse: [dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(n=0),
             dict(sink=-1), dict(recent=0), dict(sink=9), dict(sink=7), dict(recent=9),
             dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(new=-1), dict(q=NULL),
             dict(bounds=NULL), dict(out=NULL), dict(st=NULL), dict(out=ODD), dict(hq=3)],
    prefix: [dict(groups=-1), dict(groups=4), dict(new=-2), dict(ptr=NULL), dict(pages=NULL),
             dict(q=NULL), dict(out=NULL), dict(st=NULL), dict(vc=ODD), dict(hq=7)],
}


@pytest.mark.parametrize("call", list(INVALID), ids=lambda c: c.__name__)
def test_invalid_arguments_launch_nothing(lib_path, call):
    before = K.kara_launch_count()
    for bad in INVALID[call]:
        assert call(**bad) == K.ERR_INVALID_ARG, bad
    for bad in (dict(pool=pool(page=32)), dict(pool=pool(d=96))):
        assert call(**bad) == K.ERR_UNSUPPORTED, bad
    if call is not page_bounds:
        assert call(hq=18) == K.ERR_UNSUPPORTED
    assert K.kara_launch_count() == before


def test_unsupported_rotary_sizes_and_small_workspaces(lib_path):
    before = K.kara_launch_count()
    for rd in (0, 8, 24, 136, 144, -16):
        assert append(rd=rd) == K.ERR_UNSUPPORTED
    for call, op, k in ((sparse, K.OP_SPARSE, 8), (prefix, K.OP_PREFIX, 0)):
        need = K.lib().kara_workspace_bytes(op, ctypes.byref(pool()), 0, 0, 4, k)
        assert need > 0
        assert call(wsn=need - 1) == K.ERR_WORKSPACE
        assert call(ws=NULL) == K.ERR_WORKSPACE
        assert call(ws=ctypes.c_void_p(128), wsn=need) == K.ERR_WORKSPACE
    assert K.kara_launch_count() == before


def test_empty_calls_return_ok_without_a_launch(lib_path):
    before = K.kara_launch_count()
    empty = pool(batch=0)
    assert append(t=0, cu=ONE, q=NULL) == K.OK
    assert append(pool=empty, t=0, q=NULL) == K.OK
    assert page_bounds(pool=empty, kc=NULL) == K.OK
    assert sparse(pool=empty, q=NULL) == K.OK
    assert prefix(groups=0, q=NULL) == K.OK
    assert prefix(pool=empty, groups=0, q=NULL) == K.OK
    assert K.kara_launch_count() == before


def test_binding_refuses_host_tensors():
    i = dict(dtype=torch.int32)
    p = K.PagedPool(torch.zeros((2, 4), **i), torch.zeros(2, **i), torch.zeros(4, **i),
                    torch.zeros(1, **i), 4, 2, 64)
    kv = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    calls = [lambda: K.paged_rope_append(q, q[:, :2], q[:, 2:], kv, kv, p, torch.zeros(32),
                                         torch.zeros(2, **i)),
             lambda: K.paged_page_bounds(kv, p),
             lambda: K.paged_sparse_attn(q, kv, kv, kv, p, 4),
             lambda: K.paged_prefix_attn(q, kv, kv, p, torch.zeros(2, **i), torch.zeros(1, **i))]
    for fn in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn()


def test_workspace_sizes_hold_the_partials(lib_path):
    """The sizes grow with what the calls leave there: partials of every unit, scores of every
    page; the prefix partials are bounded by the rows and the blocks, not by the prefix."""
    def size(op, k=0, **kw):
        return K.lib().kara_workspace_bytes(op, ctypes.byref(pool(**kw)), 0, 0, 4, k)

    ranges = 148 * 3 * 4 // 2                        # warps of the streaming kernel per KV head
    assert size(K.OP_SPARSE, 8) >= (3 + ranges) * 4 * 130 * 4 + 3 * 2 * 64 * 20 + 3 * 2 * 8 * 4
    assert size(K.OP_PREFIX) >= (3 * 4 + 256 * 148 + (3 + ranges) * 4) * 130 * 4
    assert size(K.OP_PREFIX, width=65536) == size(K.OP_PREFIX)
    assert size(K.OP_SPARSE, 0) == 0 and size(K.OP_PREFIX, batch=0) == 0
    big = size(K.OP_SPARSE, 64, batch=4096, width=65536, hkv=8)
    assert big > 2 ** 32 * 8
