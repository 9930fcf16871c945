"""Tokens taken back from the 8-bit cache (a smaller past[s]), those among them that were not finite: a page goes on as if
they had not been.  Codes, scales and results against the plain 64-bit cache that never saw them."""
import math

import pytest
import torch

from test_gpu_kv import DEV, Model, check_attention, empty_cache, ints, rows

pytestmark = pytest.mark.gpu
NKV, HD, G = 2, 64, 3


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import ops as o
    return o


def put(ops, cache, past, k, v, table):
    n = k.shape[0]
    plan = ops.kv_plan(ints([past]), ints([0, n]), ints([table]), n, n, G * NKV, NKV, HD)
    ops.kv_append(cache, plan, k, v)
    return plan


def codes(cache, model, table, tokens):
    """The scales, and the codes of the sequence's tokens (behind them the proposed ones' may lie)."""
    full, rest = divmod(tokens, 64)
    for p, n in [(table[i], 64) for i in range(full)] + ([(table[full], rest)] if rest else []):
        for a, b in ((cache.k[p].double()[:, :n], model.k[p][:, :n]), (cache.v[p].double().transpose(1, 2)[:, :n], model.v[p][:, :n]),
                     (cache.scale[p].double(), model.s[p])):
            assert ((a == b) | (a.isnan() & b.isnan())).all()


# tokens at first, then steps of (past, rows of the call, rows that are not finite); a step without such rows is kept
CASES = [
    (10, [(10, 4, [2]), (10, 3, [])]),                                  # the whole proposal taken back
    (10, [(10, 4, [0, 3]), (7, 5, [])]),                                # and older tokens
    (10, [(10, 1, [0]), (10, 1, [0]), (10, 1, [])]),                    # twice
    (10, [(10, 4, [2]), (14, 2, []), (16, 3, [1]), (10, 6, [])]),       # gone on behind it first
    (62, [(62, 5, [1]), (62, 5, [])]),                                  # over a page's end
    (62, [(62, 5, [3]), (62, 5, [])]),
    (100, [(100, 40, [20]), (100, 60, [])]), (64, [(64, 2, [0]), (64, 2, [])]), (30, [(30, 2, [1]), (0, 3, [])]),
    (20, [(20, 3, [1]), (18, 2, [0]), (12, 1, [0]), (12, 30, [])]),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("what", ["k", "v", "both"])
@pytest.mark.parametrize("std", [1.0, 64.0])
def test_tokens_that_are_not_finite_taken_back(ops, case, what, std):
    first, steps = case
    table = [2, 0, 3]
    cache = empty_cache(ops, 4, NKV, HD)
    model = Model(cache)  # never sees what is taken back
    k, v = rows(1, first, NKV, HD), rows(2, first, NKV, HD)
    put(ops, cache, 0, k, v, table)
    model.append([0], [first], [table], k, v)
    for i, (past, n, bad) in enumerate(steps):
        last = i == len(steps) - 1
        k, v = rows(10 + i, n, NKV, HD, std if last else 1.0), rows(20 + i, n, NKV, HD, std if last else 1.0)
        k[:, 5], v[:, 70] = 0.25, -0.5
        for r in bad:
            if what != "v":
                k[r, 9] = math.inf if r % 2 else math.nan
            if what != "k":
                v[r, 64 + 9] = -math.inf
        if not last:  # small, so that the scales of pages that stay finite do not grow
            k, v = k * 2.0 ** -8, v * 2.0 ** -8
        plan = put(ops, cache, past, k, v, table)
        if bad:
            page = table[past // 64 + (1 if past % 64 + bad[0] >= 64 else 0)]
            if what != "v":
                assert cache.scale[page, 0, 0].isnan() and cache.scale[page, 1, 0].isfinite()
            if what != "k":
                assert cache.scale[page, 1, 1].isnan() and cache.scale[page, 0, 1].isfinite()
    past, n, _ = steps[-1]
    model.append([past], [n], [table], k, v)
    codes(cache, model, table, past + n)
    check_attention(ops, cache, model, plan, [past], [n], [table], rows(30, n, NKV * G, HD), normwise=False)


def test_a_token_that_is_not_finite_stays_until_it_is_taken_back(ops):
    """Behind the first row of the call that brought it, a page stays what it is; a page begun with it too."""
    table = [0, 1]
    for first, past in ((10, 11), (10, 40), (0, 1), (0, 3)):
        cache = empty_cache(ops, 2, NKV, HD)
        if first:
            put(ops, cache, 0, rows(1, first, NKV, HD), rows(2, first, NKV, HD), table)
        k = rows(3, 4, NKV, HD)
        k[2, 9] = math.nan
        put(ops, cache, first, k, rows(4, 4, NKV, HD), table)
        put(ops, cache, past, rows(5, 2, NKV, HD), rows(6, 2, NKV, HD), table)
        assert cache.scale[0, 0, 0].isnan() and cache.scale[0, 1].isfinite().all() and cache.scale[0, 0, 1].isfinite()


def test_scales_that_are_nan_by_other_means_stay(ops):
    """A caller's own NaN, of any kind, says nothing about an earlier scale: the page is lost until it is begun anew."""
    for bits in (0x7fc00000, 0x7fffffff, 0x7f800001, -1, 0x7fc00001, -0x400000):
        cache = empty_cache(ops, 1, NKV, HD)
        put(ops, cache, 0, rows(1, 5, NKV, HD), rows(2, 5, NKV, HD), [0])
        cache.k[:, 0] = 0
        cache.scale.view(torch.int32)[0, 0, 0] = bits
        put(ops, cache, 5, rows(3, 2, NKV, HD), rows(4, 2, NKV, HD), [0])
        assert cache.scale[0, 0, 0].isnan() and cache.scale[0, 0, 1].isfinite()
        put(ops, cache, 1, rows(3, 2, NKV, HD), rows(4, 2, NKV, HD), [0])
        assert cache.scale[0, 0, 0].isnan()
        put(ops, cache, 0, rows(3, 2, NKV, HD), rows(4, 2, NKV, HD), [0])
        assert cache.scale.isfinite().all()
