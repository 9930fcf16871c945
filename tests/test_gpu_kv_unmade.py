"""Calls with a plan that was never made, or made for other sizes: nothing is read by it or written, the device error word
says so, and the next call with a plan that was made works.  (Memory of a plan holds anything before it is made.)"""
import pytest
import torch

from test_gpu_kv import DEV, Model, check_attention, empty_cache, ints, rows, starts

pytestmark = pytest.mark.gpu
NKV, HD = 2, 64


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import ops as o
    return o


def run(ops, cache, plan, G, T, stored):
    """Append and attention; returns what the device error word says after each."""
    k, v, q = rows(1, T, NKV, HD), rows(2, T, NKV, HD), rows(3, T, G * NKV, HD)
    o, lse = torch.full((T, G * NKV * HD), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((G * NKV, T), 7.0, device=DEV)
    before = [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.scale.view(torch.int32))]
    said = []
    ops.kv_append(cache, plan, k, v)
    said.append(ops.device_error())
    ops.attention_kv(q, cache, plan, o=o, lse=lse)
    said.append(ops.device_error())
    if stored is None:
        assert all(torch.equal(a, b) for a, b in zip(before, (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.scale.view(torch.int32))))
        assert (o == 7).all() and (lse == 7).all()
    return said


@pytest.mark.parametrize("G,new", [(2, [1, 2]), (8, [30, 1])], ids=["few", "chunks"])
def test_a_plan_that_was_not_made(ops, G, new):
    past, table, T = [70, 3], [[0, 1], [2, 3]], sum(new)
    cache = empty_cache(ops, 4, NKV, HD)
    model = Model(cache)
    step_plan = ops.kv_plan(ints([0, 0]), ints(starts(past)), ints(table), sum(past), max(past), G * NKV, NKV, HD)
    k, v = rows(8, sum(past), NKV, HD), rows(9, sum(past), NKV, HD)
    ops.kv_append(cache, step_plan, k, v)
    model.append([0, 0], past, table, k, v)
    tab = ints(table)
    args = (T, max(new), G * NKV, NKV, HD)
    plan = ops.KVPlan(tab, *args, None)  # never made
    plan.data = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)  # room for the larger ones below too
    plan.c.data = plan.data.data_ptr()
    g = torch.Generator(DEV).manual_seed(1)
    for fill in (0, 255, None):
        if fill is None:
            plan.data.random_(generator=g)
        else:
            plan.data.fill_(fill)
        assert run(ops, cache, plan, G, T, None) == [ops.WS_DERR_BAD_CONFIG] * 2
    # one captured and not yet replayed is not made either
    start, had = ints(starts(new)), ints(past)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.kv_plan(had, start, tab, *args, plan=plan)
    assert run(ops, cache, plan, G, T, None) == [ops.WS_DERR_BAD_CONFIG] * 2
    graph.replay()
    ops.kv_append(cache, plan, rows(1, T, NKV, HD), rows(2, T, NKV, HD))
    model.append(past, new, table, rows(1, T, NKV, HD), rows(2, T, NKV, HD))
    model.check(cache)
    check_attention(ops, cache, model, plan, past, new, table, rows(3, T, G * NKV, HD))
    # the struct changed since: other rows, other bounds, other heads
    for name, value in (("T", T + 1), ("max_new", max(new) - 1 or 2), ("n_seq", 1), ("max_pages", 1), ("n_heads", 2 * G * NKV)):
        old = getattr(plan.c, name)
        setattr(plan.c, name, value)
        k, q = rows(1, T + 1, NKV, HD), rows(3, T + 1, 2 * G * NKV, HD)
        o = torch.full_like(q, 7.0)
        ws = torch.empty(ops.attention_kv_workspace_size(plan), dtype=torch.uint8, device=DEV)
        stream = torch.cuda.current_stream().cuda_stream
        assert ops._lib.ws_kv_append(cache.ref, plan.ref, k.data_ptr(), NKV * HD, k.data_ptr(), NKV * HD, stream) == 0
        assert ops.device_error() == ops.WS_DERR_BAD_CONFIG
        assert ops._lib.ws_attention_kv(cache.ref, plan.ref, q.data_ptr(), q.shape[1], 0.125, o.data_ptr(), q.shape[1], None, ws.data_ptr(),
                                        ws.nbytes, stream) == 0
        assert ops.device_error() == ops.WS_DERR_BAD_CONFIG
        assert (o == 7).all()
        setattr(plan.c, name, old)
    model.check(cache)
    check_attention(ops, cache, model, plan, past, new, table, rows(3, T, G * NKV, HD))
