"""Limits of the many-adapter linear (host checks only): the workspace of a shape has a size exactly where the calls take
that shape."""
import ctypes as C

import pytest

from test_multi_args import OK, OOM, SHAPE, _bwd, _fwd, ops  # noqa: F401

SHAPES = [
    (1, 64, 64, 1, True), (1 << 20, 64, 64, 4096, True), (5, 1 << 30, 64, 1, True), (5, 64, 1 << 30, 3, True),
    ((1 << 20) + 1, 64, 64, 1, False), (1, 64, 64, 4097, False), (1, 64, 64, 0, False), (0, 64, 64, 1, False),
    (5, (1 << 30) + 64, 64, 1, False), (5, 64, (1 << 30) + 64, 1, False), (5, 1 << 40, 64, 1, False),
    (1 << 20, 64, (1 << 14) - 64, 9, True), (1 << 20, 64, 1 << 14, 9, False), (1 << 20, 1 << 14, 64, 9, False),
    (16, 1 << 30, 64, 1, False), (15, 1 << 30, 64, 1, True), (5, 96, 64, 1, False), (5, 64, 32, 1, False),
]


@pytest.mark.parametrize("M,N,K,n,ok", SHAPES)
def test_a_workspace_has_a_size_where_the_call_takes_the_shape(ops, M, N, K, n, ok):  # noqa: F811
    size = C.c_size_t(0)
    assert ops._lib.ws_lora_multi_workspace_size(M, N, K, n, C.byref(size)) == (OK if ok else SHAPE)
    # nothing of it is reached: the workspace of a shape that is taken is one byte short
    kw = dict(M=M, N=N, K=K, n=n, pn=n, sa=16 * K, sb=16 * N, bytes=max(size.value, 1) - 1)
    assert _fwd(ops, **kw) == _bwd(ops, **kw) == (OOM if ok else SHAPE)
    if ok:
        assert size.value > 0
