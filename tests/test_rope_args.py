"""The norm and rotary positions of query and key heads: refusals (host checks only: no kernel runs, the device pointers
are made up), and the frequencies and turns made on the host."""
import ctypes as C
import math
from fractions import Fraction

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


def _args(**kw):
    a = dict(turns=D, rot=64, il=0, factor=1.0, reserved=0, rope=True, pos=D, M=5, nh=6, nkv=2, hd=64, eps=1e-6, gq=D, gk=D,
             q=D, sq=384, k=D, sk=128, oq=D + 64, soq=384, ok=D + 64, sok=128, uq=D, suq=384, uk=D, suk=128,
             dgq=D, dgk=D, acc=0, ws=D, bytes=1 << 30)
    a.update(kw)
    return a


def _fwd(ops, **kw):
    a = _args(**kw)
    r = C.byref(ops.RopeC(a["turns"], a["rot"], a["il"], a["factor"], a["reserved"])) if a["rope"] else None
    return ops._lib.ws_qk_norm_rope_fwd(r, a["pos"], a["M"], a["nh"], a["nkv"], a["hd"], a["eps"], a["gq"], a["gk"], a["q"], a["sq"],
                                        a["k"], a["sk"], a["oq"], a["soq"], a["ok"], a["sok"], None)


def _bwd(ops, **kw):
    a = _args(**kw)
    r = C.byref(ops.RopeC(a["turns"], a["rot"], a["il"], a["factor"], a["reserved"])) if a["rope"] else None
    return ops._lib.ws_qk_norm_rope_bwd(r, a["pos"], a["M"], a["nh"], a["nkv"], a["hd"], a["eps"], a["gq"], a["gk"], a["q"], a["sq"],
                                        a["k"], a["sk"], a["uq"], a["suq"], a["uk"], a["suk"], a["oq"], a["soq"], a["ok"], a["sok"],
                                        a["dgq"], a["dgk"], a["acc"], a["ws"], a["bytes"], None)


SHARED = [
    (dict(M=0), SHAPE), (dict(M=(1 << 30) + 1), SHAPE), (dict(nh=0), SHAPE), (dict(nkv=0), SHAPE), (dict(nh=1025), SHAPE),
    (dict(hd=96), SHAPE), (dict(hd=256), SHAPE), (dict(hd=0), SHAPE), (dict(rot=8), SHAPE), (dict(rot=72), SHAPE), (dict(rot=80), SHAPE),
    (dict(rot=24), SHAPE), (dict(turns=None), INVALID), (dict(pos=None), INVALID), (dict(il=2), INVALID), (dict(reserved=1), INVALID),
    (dict(factor=math.inf), INVALID), (dict(factor=math.nan), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(rope=False, gq=None, gk=None, dgq=None, dgk=None), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(oq=None), INVALID), (dict(ok=None), INVALID), (dict(sq=376), SHAPE), (dict(sk=132), SHAPE),
    (dict(soq=64), SHAPE), (dict(sok=130), SHAPE), (dict(turns=D + 8), ALIGN), (dict(pos=D + 2), ALIGN), (dict(gq=D + 4), ALIGN),
    (dict(q=D + 8), ALIGN), (dict(k=D + 2), ALIGN), (dict(oq=D + 8), ALIGN), (dict(ok=D + 4), ALIGN),
    (dict(oq=D, soq=392), INVALID), (dict(ok=D, sok=136), INVALID),
]


@pytest.mark.parametrize("kw,want", SHARED, ids=[str(i) for i in range(len(SHARED))])
def test_refusals(ops, kw, want):
    assert _fwd(ops, **kw) == want
    assert _bwd(ops, **kw) == want


def test_refusals_of_the_backward(ops):
    assert _bwd(ops, uq=None) == INVALID and _bwd(ops, suk=120) == SHAPE and _bwd(ops, uk=D + 8) == ALIGN
    assert _bwd(ops, acc=1) == INVALID and _bwd(ops, acc=4) == INVALID
    assert _bwd(ops, gq=None) == INVALID                     # a gradient of a gain that is not there
    assert _bwd(ops, dgk=D + 2) == ALIGN and _bwd(ops, ws=None) == INVALID and _bwd(ops, ws=D + 4) == ALIGN
    n = C.c_size_t(0)
    size = ops._lib.ws_qk_norm_rope_workspace_size
    assert size(5, 6, 2, 64, C.byref(n)) == OK and n.value > 0
    assert _bwd(ops, bytes=n.value - 1) == OOM
    assert size(5, 6, 2, 64, None) == INVALID and size(0, 6, 2, 64, C.byref(n)) == SHAPE and size(5, 6, 2, 32, C.byref(n)) == SHAPE
    assert size(1 << 30, 1024, 1024, 128, C.byref(n)) == OK


def test_python_refusals(ops):
    q, k = torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(3, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.qk_norm_rope_fwd(q.float(), k, 64)
    with pytest.raises(ValueError):
        ops.qk_norm_rope_fwd(q, k[:2], 64)
    with pytest.raises(ValueError):
        ops.qk_norm_rope_fwd(q, k, 64)                       # not on a CUDA device
    for bad in (dict(rot=24), dict(rot=64, base=1.0), dict(rot=64, scaling="other"), dict(rot=64, scaling="yarn"),
                dict(rot=64, factor=0.5)):
        with pytest.raises(ValueError):
            ops.rope_frequencies(**bad)
    with pytest.raises(ValueError):
        ops.rope(64, inv_freq=[1.0] * 16, device="cpu")
    with pytest.raises(ops.WsError):
        ops.rope(16, inv_freq=[math.inf] * 8, device="cpu")


def test_turns_are_the_fraction_of_a_turn(ops):
    r = ops.rope(128, base=1e6, device="cpu")
    tau = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572418")
    for i, t in enumerate(r.turns.tolist()):
        want = Fraction(1e6 ** (-2.0 * i / 128)) / tau % 1 * (1 << 64)
        got = Fraction(t % (1 << 64))
        # double arithmetic: two roundings of a value below one turn
        assert abs(got - want) <= Fraction(1 << 64, 1 << 52)
    neg = ops.rope(16, inv_freq=[-0.25] * 8, device="cpu").turns.tolist()[0]
    pos = ops.rope(16, inv_freq=[0.25] * 8, device="cpu").turns.tolist()[0]
    d = (neg + pos) % (1 << 64)
    assert min(d, (1 << 64) - d) <= 1 << 12
    assert ops.rope(16, inv_freq=[0.0] * 8, device="cpu").turns.tolist() == [0] * 8


def test_scaled_frequencies(ops):
    plain, one = ops.rope_frequencies(64, base=1e4)
    assert one == 1.0 and plain[0] == 1.0 and math.isclose(plain[1], 1e4 ** (-1 / 32))
    lin, _ = ops.rope_frequencies(64, base=1e4, scaling="linear", factor=4.0)
    assert all(math.isclose(4 * a, b) for a, b in zip(lin, plain))
    ntk, _ = ops.rope_frequencies(64, base=1e4, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and math.isclose(4 * ntk[-1], plain[-1])
    yarn, f = ops.rope_frequencies(64, base=1e4, scaling="yarn", factor=4.0, original=2048)
    assert math.isclose(f, 0.1 * math.log(4) + 1)
    turns = [2048 * p / (2 * math.pi) for p in plain]
    for y, p, t in zip(yarn, plain, turns):
        if t > 40:
            assert y == p
        elif t < 0.5:
            assert math.isclose(4 * y, p)
        else:
            assert p / 4 * (1 - 1e-12) <= y <= p * (1 + 1e-12)
    assert ops.rope_frequencies(64, scaling="yarn", factor=4.0, original=2048, attention_factor=1.5)[1] == 1.5
    r = ops.rope(64, base=1e4, scaling="linear", scale=4.0, device="cpu")
    assert r.rot == 64 and r.turns.tolist() == ops.rope(64, inv_freq=lin, device="cpu").turns.tolist()
