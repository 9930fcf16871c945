"""Lengths, row ranges and tables that no caller should give, through plan, append and attention: all memory that the calls
get lies inside larger buffers, of which nothing else may change; rows and pages of no sequence stay as they were; and what
can be served is.  Row ranges that name rows twice, more often than a plan has room for among them."""
import pytest
import torch

from test_gpu_kv import DEV, PAGE, Model, attention, ints, rows

pytestmark = pytest.mark.gpu
NKV, HD = 2, 64


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import ops as o
    return o


class Guarded:
    """Tensors that lie in larger buffers, 4096 bytes from either end."""

    def __init__(self):
        self.all = []

    def make(self, shape, dtype, fill=0xa5):
        n = torch.empty(shape, dtype=dtype, device="meta").nbytes
        big = torch.full((n + 8192,), 0xa5, dtype=torch.uint8, device=DEV)
        big[4096:4096 + n] = fill
        self.all.append((big, n))
        return big[4096:4096 + n].view(dtype).view(shape)

    def like(self, t):
        out = self.make(tuple(t.shape), t.dtype)
        out.copy_(t)
        return out

    def check(self):
        for big, n in self.all:
            assert (big[:4096] == 0xa5).all() and (big[4096 + n:] == 0xa5).all()


BIG = 1 << 30
CASES = {  # query heads of a kv head, rows, most new rows, pages of a row of the table, tokens before, row starts
    "few": (2, 8, 3, 2, [[70, -9, 70], [BIG, 70, 70], [70, 70, 70], [127, 128, 126], [70, 70, 70], [0, 0, 0]],
            [[0, 1, 2, 3], [0, 1, 2, 3], [5, 2, 400, -7], [0, 4, 6, 8], [-(1 << 31), (1 << 31) - 1, 8, 8], [0, 8, 0, 8]]),
    "chunks": (8, 100, 40, 3, [[70, -9, 70, 0], [BIG, 70, 192, 191], [70] * 4, [150, 3, 64, 191], [-BIG, BIG, 70, 70]],
               [[0, 30, 60, 99, 100], [0, 40, 80, 99, 100], [0, 100, 0, 100, 0], [-50, 20, 90, 70, 1 << 20], [100, -1, 60, 61, 200]]),
    "more than there is room for": (8, 20, 20, 2, [[0, 0] * 32, [60, 3] * 32], [[0, 20] * 32 + [0]] * 2),
    "more single rows than there is room for": (2, 1, 1, 2, [[0, 0] * 32, [60, 3] * 32], [[0, 1] * 32 + [0]] * 2),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("holes", [False, True])
def test_arrays_out_of_range_change_nothing_else(ops, name, holes):
    G, T, most, width, pasts, begins = CASES[name]
    n = len(pasts[0])
    spare = 3
    pages = n * width + spare  # the last ones are in no table
    for past, start in zip(pasts, begins):
        guard = Guarded()
        cache = ops.KVCache(guard.make((pages, NKV, PAGE, HD), torch.float8_e4m3fn), guard.make((pages, NKV, HD, PAGE), torch.float8_e4m3fn),
                            guard.make((pages, NKV, 2), torch.float32))
        cache.k.view(torch.uint8).copy_(torch.randint(0, 0x7f, cache.k.shape, dtype=torch.uint8))
        cache.v.view(torch.uint8).copy_(torch.randint(0, 0x7f, cache.v.shape, dtype=torch.uint8))
        cache.scale.fill_(2.0 ** -6)
        table = [[i * width + j for j in range(width)] for i in range(n)]
        if holes:  # pages that are none, of every kind
            table[0][0], table[1][-1], table[2][0] = -1, pages, (1 << 31) - 1
            table[n - 1][width - 1] = -(1 << 31)
        model = Model(cache)
        tab = guard.like(ints(table))
        plan = ops.kv_plan(ints([0] * n), ints([0] * (n + 1)), tab, T, most, G * NKV, NKV, HD)
        plan.data = guard.like(plan.data)
        plan.c.data = plan.data.data_ptr()
        ops.kv_plan(guard.like(ints(past)), guard.like(ints(start)), tab, T, most, G * NKV, NKV, HD, plan=plan)
        k, v, q = (guard.like(rows(s, T, h, HD)) for s, h in ((1, NKV), (2, NKV), (3, G * NKV)))
        o, lse = guard.make((T, G * NKV * HD), torch.bfloat16), guard.make((G * NKV, T), torch.float32)
        o.fill_(7)
        lse.fill_(7)
        ws = guard.make((ops.attention_kv_workspace_size(plan),), torch.uint8)
        ops.kv_append(cache, plan, k, v)
        ops.attention_kv(q, cache, plan, o=o, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        assert ops.device_error() == 0
        guard.check()
        # the plan's own reading of them
        room = width * PAGE
        p = [min(max(a, 0), room) for a in past]
        lo = [min(max(a, 0), T) for a in start[:-1]]
        c = [max(0, min(min(max(b, a), T) - a, most, room - x)) for a, b, x in zip(lo, start[1:], p)]
        named = torch.zeros(T, dtype=torch.int32, device=DEV)
        for a, m in zip(lo, c):
            named[a:a + m] += 1
        assert (o[named == 0] == 7).all() and (lse[:, named == 0] == 7).all()
        before = [t.clone() for t in (model.k, model.v, model.s)]
        for i in range(n):
            model.append([p[i]], [c[i]], [table[i]], k[lo[i]:lo[i] + c[i]], v[lo[i]:lo[i] + c[i]])
        held = (cache.k.double(), cache.v.double().transpose(2, 3), cache.scale.double())
        if "more" in name:  # which of them get a place is open; each page is one or the other, whole
            for page in range(pages):
                old, new = ([bool(((a[page] == b[page]) | (a[page].isnan() & b[page].isnan())).all()) for a, b in zip(held, x)]
                            for x in (before, (model.k, model.v, model.s)))
                assert all(old) or all(new)
            assert all(torch.equal(a[-spare:], b[-spare:]) for a, b in zip(held, before))
            # something is appended, unless the page that comes first is none: one row has one place, and table[0][0] is -1
            assert holes or any(not torch.equal(a, b) for a, b in zip(held, before))
            continue
        model.check(cache)
        assert all(torch.equal(a[-spare:], b[-spare:]) for a, b in zip(held, before))
        for ro, tol, rl, ltol, r0 in attention(model, p, c, table, q, G, HD, HD ** -0.5, start=lo):
            m = ro.shape[0]
            once = named[r0:r0 + m] == 1
            got, glse = o[r0:r0 + m].double().view(m, -1, HD)[once], lse.t()[r0:r0 + m].double()[once]
            assert (got - ro[once]).abs().le(tol[once]).all()
            real = rl[once].isfinite()
            assert torch.equal(glse[~real], rl[once][~real]) and (glse - rl[once]).abs()[real].le(ltol[once][real]).all()
