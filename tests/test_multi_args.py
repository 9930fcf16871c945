"""Refusals of the many-adapter linear and of AdamW (host checks only: no kernel
runs, the device pointers are made up), and the chunk plan that
ws_adamw_plan_init writes on the host."""
import ctypes as C

import numpy as np
import pytest
import torch

OK, INVALID, SHAPE, ALIGN, OOM, UNSUPPORTED = 0, -1, -2, -3, -6, -7
D = 0x7F0000000000  # a 16-byte aligned address that nothing here reads


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import build
    build.build()
    from weight_streaming_nf4_gb300 import ops as o
    return o


def _linear(ops, **kw):
    """Arguments of a valid forward, changed by kw, and the status of the call."""
    a = dict(codes=D, absmax=D, N=128, K=192, A=D, B=D, scale=D, sa=16 * 192, sb=128 * 16, n=3, r=16, dtype=0 + 1,
             data=D, M=5, pn=3, x=D, mask=None, y=D, U=D, ws=D, bytes=1 << 40)
    a.update(kw)
    w = ops.Nf4(a["codes"], a["absmax"], a["N"], a["K"])
    s = ops.LoraSetC(a["A"], a["B"], a["scale"], a["sa"], a["sb"], a["n"], a["r"], a["dtype"])
    p = ops.LoraPlanC(a["data"], a["M"], a["pn"])
    return a, w, s, p


def _fwd(ops, **kw):
    a, w, s, p = _linear(ops, **kw)
    return ops._lib.ws_lora_linear_fwd_multi(C.byref(w), a["x"], C.byref(s), C.byref(p), a["mask"], a["y"], a["U"],
                                             a["ws"], a["bytes"], None)


def _bwd(ops, dX=D, dt=1, acc=0, dA=D, dB=D, dY=D, **kw):
    a, w, s, p = _linear(ops, **kw)
    return ops._lib.ws_lora_linear_bwd_multi(C.byref(w), a["x"], C.byref(s), C.byref(p), a["mask"], a["U"], dY, dX,
                                             dt, acc, dA, dB, a["ws"], a["bytes"], None)


SHARED = [
    (dict(codes=None), INVALID), (dict(A=None), INVALID), (dict(scale=None), INVALID), (dict(data=None), INVALID),
    (dict(x=None), INVALID), (dict(ws=None), INVALID), (dict(U=None), INVALID), (dict(dtype=7), INVALID),
    (dict(N=100), SHAPE), (dict(K=0), SHAPE), (dict(K=32), SHAPE), (dict(r=8), SHAPE), (dict(M=0), SHAPE),
    (dict(M=(1 << 20) + 1), SHAPE), (dict(n=4), SHAPE), (dict(n=0, pn=0), SHAPE), (dict(n=4097, pn=4097), SHAPE),
    (dict(sa=16 * 192 - 8), SHAPE), (dict(sb=128 * 16 + 4), SHAPE), (dict(sa=0), SHAPE),
    (dict(codes=D + 8), ALIGN), (dict(A=D + 4), ALIGN), (dict(mask=D + 4), ALIGN), (dict(scale=D + 2), ALIGN),
    (dict(x=D + 2), ALIGN), (dict(U=D + 8), ALIGN), (dict(ws=D + 1), ALIGN), (dict(data=D + 4), ALIGN),
    (dict(bytes=16), OOM),
]


@pytest.mark.parametrize("kw,want", SHARED, ids=[str(i) for i in range(len(SHARED))])
def test_linear_refusals(ops, kw, want):
    assert _fwd(ops, **kw) == want
    assert _bwd(ops, **kw) == want


def test_linear_refusals_of_one_direction(ops):
    assert _fwd(ops, y=None) == INVALID and _fwd(ops, y=D + 8) == ALIGN
    assert _bwd(ops, dX=None) == INVALID and _bwd(ops, dY=None) == INVALID and _bwd(ops, dA=None) == INVALID
    assert _bwd(ops, dt=2) == INVALID and _bwd(ops, acc=4) == INVALID
    assert _bwd(ops, dt=0, acc=1) == INVALID           # accumulating needs an fp32 dX
    assert _bwd(ops, dtype=0) == UNSUPPORTED           # bf16 adapters are for serving
    assert _bwd(ops, dB=D + 4) == ALIGN


def test_plan_and_mask_refusals(ops):
    n = C.c_size_t(0)
    size, init = ops._lib.ws_lora_multi_plan_size, ops._lib.ws_lora_multi_plan_init
    assert size(0, 1, C.byref(n)) == SHAPE and size(5, 0, C.byref(n)) == SHAPE and size(5, 4097, C.byref(n)) == SHAPE
    assert size(5, 3, None) == INVALID and size(5, 3, C.byref(n)) == OK and n.value > 0
    assert init(C.byref(ops.LoraPlanC(D, 5, 3)), None, None) == INVALID
    assert init(C.byref(ops.LoraPlanC(D, 5, 3)), D + 2, None) == ALIGN
    assert init(C.byref(ops.LoraPlanC(D + 8, 5, 3)), D, None) == ALIGN
    key = ops.dropout_key(p=0.1)
    m = ops._lib.ws_dropout_mask
    assert m(key, 4, 100, D, None) == SHAPE and m(key, 4, 64, None, None) == INVALID and m(key, 4, 64, D + 4, None) == ALIGN
    assert m(ops.dropout_key(p=1.0), 4, 64, D, None) == INVALID
    w = ops._lib.ws_lora_multi_workspace_size
    assert w(0, 64, 64, 1, C.byref(n)) == SHAPE and w(4, 60, 64, 1, C.byref(n)) == SHAPE and w(4, 64, 64, 1, None) == INVALID


def test_tensors_that_are_not_on_the_gpu_are_refused(ops):
    A, B, s = torch.zeros(2, 16, 64), torch.zeros(2, 64, 16), torch.ones(2)
    with pytest.raises(ValueError):
        ops.LoraSet(A, B, s)
    with pytest.raises(ValueError):
        ops.lora_multi_plan(torch.zeros(4, dtype=torch.int32), 2)
    p = [torch.zeros(8)]
    with pytest.raises(ValueError):
        ops.adamw_plan(p, p, p, p)
    with pytest.raises(ValueError):
        ops.adamw_encode8(torch.zeros(8), False)
    for bad in (dict(A=A[:, :8]), dict(B=B.bfloat16()), dict(scale=s.double()), dict(A=A[:1])):
        with pytest.raises(ValueError):
            ops.LoraSet(**{**dict(A=A, B=B, scale=s), **bad})


# ------------------------------------------------------------------------------ AdamW
def _tensors(ops, sizes, groups, bits=32, at=D):
    arr = (ops.AdamwTensorC * len(sizes))()
    for i, (n, g) in enumerate(zip(sizes, groups)):
        room = -(-n * 4 // 256) * 256
        p = [at + k * room for k in range(6)]
        at += 6 * room
        arr[i] = ops.AdamwTensorC(p[0], p[1], p[2], p[3], p[4] if bits == 8 else None, p[5] if bits == 8 else None,
                                  n, g, 0)
    return arr


def _init(ops, arr, n_groups=1, types=(1, 1, 32), n=None):
    n = len(arr) if n is None else n
    pb, wb = C.c_size_t(0), C.c_size_t(0)
    ty = ops.AdamwTypesC(*types)
    st = ops._lib.ws_adamw_plan_size(arr, n, n_groups, ty, C.byref(pb), C.byref(wb))
    if st:
        return st, None, None
    image = np.zeros(pb.value, np.uint8)
    plan = ops.AdamwPlanC()
    st = ops._lib.ws_adamw_plan_init(arr, n, n_groups, ty, image.ctypes.data, image.size, C.byref(plan))
    return st, image, plan


def test_adamw_plan_lists_every_chunk_once_by_group(ops):
    sizes = [1, 4096, 4097, 3, 20000, 8192, 5]
    groups = [2, 0, 2, 0, 3, 2, 0]   # group 1 has no tensor
    arr = _tensors(ops, sizes, groups)
    st, image, plan = _init(ops, arr, 4)
    assert st == OK
    per = [-(-s // 4096) for s in sizes]
    assert plan.n_chunks == sum(per)
    c = image[:plan.n_chunks * 64]
    first = image[plan.n_chunks * 64:plan.n_chunks * 64 + 20].view(np.int32)
    assert first[0] == 0 and first[-1] == sum(per)
    ptr, num = c.view(np.uint64).reshape(-1, 8), c.view(np.int32).reshape(-1, 16)
    want = [(arr[i].p + 4 * e, arr[i].g + 4 * e, arr[i].m + 4 * e, arr[i].v + 4 * e, min(4096, sizes[i] - e), g)
            for g in range(4) for i in range(len(sizes)) if groups[i] == g for e in range(0, sizes[i], 4096)]
    assert [(*map(int, p[:4]), int(q[12]), int(q[13])) for p, q in zip(ptr, num)] == want
    for g in range(4):
        assert first[g + 1] - first[g] == sum(p for p, h in zip(per, groups) if h == g)


def test_adamw_plan_refusals(ops):
    T = lambda **kw: _tensors(ops, kw.pop("sizes", [100, 300]), kw.pop("groups", [0, 0]), **kw)
    assert _init(ops, T())[0] == OK and _init(ops, T(bits=8), types=(0, 1, 8))[0] == OK
    assert _init(ops, T(), types=(1, 1, 16))[0] == INVALID and _init(ops, T(), types=(5, 1, 32))[0] == INVALID
    assert _init(ops, T(), types=(1, 1, 8))[0] == INVALID             # 8-bit states without scales
    assert _init(ops, T(groups=[0, 1]))[0] == INVALID                 # group out of range
    assert _init(ops, T(groups=[0, -1]))[0] == INVALID
    assert _init(ops, T(), n=0)[0] == SHAPE and _init(ops, T(), n_groups=0)[0] == SHAPE
    assert _init(ops, T(sizes=[100, 0]))[0] == SHAPE
    for field in ("p", "g", "m", "v"):
        a = T()
        setattr(a[1], field, None)
        assert _init(ops, a)[0] == INVALID
        a = T()
        setattr(a[1], field, getattr(a[1], field) + 4)
        assert _init(ops, a)[0] == ALIGN
    a = T()
    a[1].p = a[0].p                                                    # the same parameter twice
    assert _init(ops, a)[0] == INVALID
    a = T()
    a[1].m = a[0].p + 384                                              # the end of another tensor
    assert _init(ops, a)[0] == INVALID
    a = T()
    a[0].g = a[0].p                                                    # a gradient that the step overwrites
    assert _init(ops, a)[0] == INVALID
    a = T()
    a[0].g = a[1].g                                                    # two readers of one gradient
    assert _init(ops, a)[0] == OK
    a = T(bits=8)
    a[1].v_scale = a[0].v_scale
    assert _init(ops, a, types=(1, 1, 8))[0] == INVALID
    st, image, plan = _init(ops, T())
    assert ops._lib.ws_adamw_plan_init(T(), 2, 1, ops.AdamwTypesC(1, 1, 32), image.ctypes.data, 64, C.byref(plan)) == OOM


def test_adamw_step_and_codec_refusals(ops):
    _, _, plan = _init(ops, _tensors(ops, [100], [0]))
    step = ops._lib.ws_adamw_step
    assert step(C.byref(plan), D, 0, None, D, 1 << 20, None) == INVALID   # the image is not set
    plan.image = D
    assert step(None, D, 0, None, D, 1 << 20, None) == INVALID
    assert step(C.byref(plan), None, 0, None, D, 1 << 20, None) == INVALID
    assert step(C.byref(plan), D, 2, None, D, 1 << 20, None) == INVALID
    assert step(C.byref(plan), D + 8, 0, None, D, 1 << 20, None) == ALIGN
    assert step(C.byref(plan), D, 0, D + 2, D, 1 << 20, None) == ALIGN
    assert step(C.byref(plan), D, 0, None, D, 16, None) == OOM
    enc, dec = ops._lib.ws_adamw_encode8, ops._lib.ws_adamw_decode8
    assert enc(D, 0, 0, D, D, None) == SHAPE and enc(D, 8, 2, D, D, None) == INVALID and enc(D + 4, 8, 0, D, D, None) == ALIGN
    assert dec(D, D, 8, 0, D, 3, None) == INVALID and dec(D, None, 8, 0, D, 0, None) == INVALID and dec(D, D + 2, 8, 0, D, 0, None) == ALIGN


def test_adamw_groups_refuses_unknown_settings(ops):
    with pytest.raises(ValueError):
        ops.adamw_groups([dict(lr=1e-3, momentum=0.9)], device="cpu")
    with pytest.raises(ValueError):
        ops.adamw_groups([dict(beta1=0.9)], device="cpu")
    for bad in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1e-8), dict(step=-1), dict(step=0.5)):
        with pytest.raises(ValueError):
            ops.adamw_groups([dict(lr=1e-3, **bad)], device="cpu")
    g = ops.adamw_groups([dict(lr=1e-3), dict(lr=2e-3, step=7, max_norm=0.5)], device="cpu")
    assert g.shape == (2, 8) and g[0].tolist() == [1e-3, 0.9, 0.999, 1e-8, 0.01, 0.0, 0.0, 0.0] and g[1, 6] == 7
