"""The paged 8-bit cache and the attention over it: refusals (host checks only: no kernel runs, the device pointers are
made up)."""
import ctypes as C
import math

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, OOM = 0, -1, -2, -3, -6
D = 0x7F0000000000  # a 16-byte aligned address that nothing here reads


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import build
    build.build()
    from weight_streaming_nf4_gb300 import ops as o
    return o


def _args(ops, **kw):
    a = dict(data=D, table=D, T=20, n_seq=4, max_pages=7, max_new=9, nh=12, nkv=4, hd=64, past=D, start=D,
             ck=D, cv=D, scale=D, pages=100, cnkv=None, chd=None, k=D, sk=256, v=D, sv=256, q=D, sq=768, sl=0.125, o=D, so=768,
             lse=D, ws=D, bytes=1 << 40)
    a.update(kw)
    plan = ops.KVPlanC(a["data"], a["table"], a["T"], a["n_seq"], a["max_pages"], a["max_new"], a["nh"], a["nkv"], a["hd"])
    cache = ops.KVCacheC(a["ck"], a["cv"], a["scale"], a["pages"], a["cnkv"] or a["nkv"], a["chd"] or a["hd"])
    return a, C.byref(plan), C.byref(cache)


def _size(ops, **kw):
    n = C.c_size_t(0)
    return ops._lib.ws_kv_plan_size(_args(ops, **kw)[1], C.byref(n)), n.value


def _work(ops, **kw):
    n = C.c_size_t(0)
    return ops._lib.ws_attention_kv_workspace_size(_args(ops, **kw)[1], C.byref(n)), n.value


def _init(ops, **kw):
    a, p, _ = _args(ops, **kw)
    return ops._lib.ws_kv_plan_init(p, a["past"], a["start"], None)


def _append(ops, **kw):
    a, p, c = _args(ops, **kw)
    return ops._lib.ws_kv_append(c, p, a["k"], a["sk"], a["v"], a["sv"], None)


def _attend(ops, **kw):
    a, p, c = _args(ops, **kw)
    return ops._lib.ws_attention_kv(c, p, a["q"], a["sq"], a["sl"], a["o"], a["so"], a["lse"], a["ws"], a["bytes"], None)


SHAPES = [
    dict(T=0), dict(T=(1 << 20) + 1), dict(n_seq=0), dict(n_seq=4097), dict(max_pages=0), dict(max_pages=(1 << 20) + 1),
    dict(n_seq=4096, max_pages=(1 << 16) + 1), dict(max_new=0), dict(max_new=21), dict(nkv=0), dict(nkv=257, nh=257), dict(nh=0),
    dict(nh=14), dict(nh=1028), dict(hd=32), dict(hd=256), dict(hd=0),
]


@pytest.mark.parametrize("kw", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_shapes_that_no_call_takes(ops, kw):
    assert _size(ops, **kw)[0] == _work(ops, **kw)[0] == _init(ops, **kw) == _append(ops, **kw) == _attend(ops, **kw) == SHAPE


@pytest.mark.parametrize("kw", [
    dict(), dict(T=1 << 20, max_new=1 << 20, nh=1024, nkv=1), dict(n_seq=4096, max_pages=1 << 16, T=4096, max_new=1),
    dict(n_seq=1, max_pages=1 << 20, T=1, max_new=1), dict(nh=256, nkv=256, hd=128), dict(T=1, n_seq=4096, max_new=1)])
def test_sizes_of_shapes_that_are_taken(ops, kw):
    (st, n), (sw, w) = _size(ops, **kw), _work(ops, **kw)
    assert st == sw == OK and n > 0 and w > 0
    # nothing of the memory is reached: the workspace is one byte short
    assert _attend(ops, **dict(dict(sq=1 << 20, so=1 << 20), **kw), bytes=w - 1) == OOM


def test_plan_refusals(ops):
    assert ops._lib.ws_kv_plan_size(None, None) == INVALID and ops._lib.ws_kv_plan_size(_args(ops)[1], None) == INVALID
    assert ops._lib.ws_attention_kv_workspace_size(_args(ops)[1], None) == INVALID
    assert ops._lib.ws_kv_plan_init(None, D, D, None) == INVALID
    for kw in (dict(data=None), dict(table=None), dict(past=None), dict(start=None)):
        assert _init(ops, **kw) == INVALID
    for kw in (dict(data=D + 8), dict(table=D + 2), dict(past=D + 1), dict(start=D + 2)):
        assert _init(ops, **kw) == ALIGN


CACHE = [(dict(ck=None), INVALID), (dict(cv=None), INVALID), (dict(scale=None), INVALID), (dict(data=None), INVALID),
         (dict(table=None), INVALID), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(cnkv=2), SHAPE), (dict(chd=128), SHAPE),
         (dict(ck=D + 8), ALIGN), (dict(cv=D + 4), ALIGN), (dict(scale=D + 4), ALIGN), (dict(data=D + 4), ALIGN), (dict(table=D + 2), ALIGN)]


@pytest.mark.parametrize("kw,want", CACHE, ids=[str(i) for i in range(len(CACHE))])
def test_cache_refusals(ops, kw, want):
    assert _append(ops, **kw) == _attend(ops, **kw) == want


def test_append_refusals(ops):
    for kw, want in ((dict(k=None), INVALID), (dict(v=None), INVALID), (dict(sk=248), SHAPE), (dict(sv=260), SHAPE), (dict(k=D + 2), ALIGN),
                     (dict(v=D + 8), ALIGN)):
        assert _append(ops, **kw) == want


def test_attention_refusals(ops):
    for kw, want in ((dict(q=None), INVALID), (dict(o=None), INVALID), (dict(ws=None), INVALID), (dict(sl=0.0), INVALID), (dict(sl=-1.0), INVALID),
                     (dict(sl=math.nan), INVALID), (dict(sl=math.inf), INVALID), (dict(sq=760), SHAPE), (dict(so=772), SHAPE), (dict(q=D + 8), ALIGN),
                     (dict(o=D + 2), ALIGN), (dict(ws=D + 8), ALIGN), (dict(lse=D + 2), ALIGN), (dict(bytes=0), OOM)):
        assert _attend(ops, **kw) == want


def test_python_refusals(ops):
    f8 = torch.float8_e4m3fn
    k, v, s = torch.zeros(3, 2, 64, 128, dtype=f8), torch.zeros(3, 2, 128, 64, dtype=f8), torch.zeros(3, 2, 2)
    for bad in ((k, k, s), (k.float(), v, s), (k, v, s[:2]), (k, v, s.double()), (k[:, :, :32], v, s), (k, v, s)):
        with pytest.raises(ValueError):  # the last is right but for its device
            ops.KVCache(*bad)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.kv_plan(i, i, torch.zeros(4, 2, dtype=torch.int32), 4, 1, 4, 2, 64)
