"""The paged 8-bit cache (append) and the attention over it, against plain 64-bit forms.

Tolerances.  Appended codes and scales are exact.  Attention: the result is rounded to bf16 once (2^-8 of it; the norm of
such roundings is below 2e-3 of the result's).  Before that, probabilities are rounded to fp16 (2^-11 of themselves) and
a score is off by at most
    delta = 2^-17 scale max|q| max_j sum|k_j|,
which covers queries held with an absolute error of 2^-18 of the row's largest element and as much again for the fp32
sums; 2^x and the sums after it add less than 2^-19.  Below 2^-14 fp16 has steps of 2^-24: a probability, relative to the
row's largest and times its page's scale over the largest scale S, enters as 2^7 times itself, so it is off by as much as
2^-25 2^-7 = 2^-32 there however small it is, which a code of at most 448 makes 2^-32 448 S for each of the N tokens seen
(it shows where the large probabilities meet zeros among the values).  So an element is off by 2^-8 of itself,
(2^-11 + 2 delta + 2^-18) sum_j p_j |v_j| and 2^-32 448 S N; lse by delta + 2^-18 + 2^-22 |lse|."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import ops as o
    return o


def power(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def e4m3(y):
    """The nearest e4m3 values (ties to even) of finite values of at most 448."""
    unit = power(torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(y / unit) * unit


def scale_of(top):
    """The smallest power of two 2^e, e >= -126, with top <= 448 2^e."""
    s = torch.full_like(top, 2.0 ** -126)
    while bool((s * 448 < top).any()):
        s = torch.where(s * 448 < top, 2 * s, s)
    return s


class Model:
    """The cache as the definition has it, in 64 bits: values, not codes."""

    def __init__(self, cache):
        self.k = cache.k.double() * 1.0
        self.v = cache.v.double().transpose(2, 3).contiguous()
        self.s = cache.scale.double()

    def append(self, past, new, table, k, v):
        nkv, hd = self.k.shape[1], self.k.shape[3]
        row = 0
        for i, (a, n) in enumerate(zip(past, new)):
            for t in range(a // PAGE, -(-(a + n) // PAGE) if n else 0):
                page = table[i][t]
                lo, hi = max(a, t * PAGE), min(a + n, (t + 1) * PAGE)
                if not 0 <= page < self.k.shape[0]:
                    continue
                p = lo - t * PAGE
                for c, codes, rows in ((0, self.k, k), (1, self.v, v)):
                    x = rows[row + lo - a:row + hi - a].double().view(hi - lo, nkv, hd).transpose(0, 1)
                    s = scale_of(x.abs().amax((1, 2)).nan_to_num(posinf=0))
                    s[~x.isfinite().flatten(1).all(1)] = math.nan
                    if p:
                        old = self.s[page, :, c]
                        s = torch.where(old.isnan() | s.isnan(), math.nan, torch.maximum(old, s))
                        grown = e4m3(codes[page, :, :p] * (old / s)[:, None, None])
                        codes[page, :, :p] = torch.where((s > old)[:, None, None], grown, codes[page, :, :p])
                    y = x / s[:, None, None]
                    codes[page, :, p:p + hi - lo] = torch.where(y.isnan(), 0.0, e4m3(y.nan_to_num()))  # under a NaN scale
                    self.s[page, :, c] = s
            row += n

    def check(self, cache):
        for a, b in ((cache.k.double(), self.k), (cache.v.double().transpose(2, 3), self.v), (cache.scale.double(), self.s)):
            off = ((a != b) & ~(a.isnan() & b.isnan())).nonzero()
            assert off.shape[0] == 0, (off.shape[0], off[0].tolist(), a[tuple(off[0])].item(), b[tuple(off[0])].item())


def attention(m, past, new, table, q, G, hd, scale, start=None):
    """Rows' (o, lse, bound of o, bound of lse), per sequence rows [n, heads, ...]; pages that are none hold nothing."""
    nkv = m.k.shape[1]
    out, row = [], 0
    for i, (a, n) in enumerate(zip(past, new)):
        r0 = row if start is None else start[i]
        row += n
        if n == 0:
            continue
        pages = table[i][:-(-(a + n) // PAGE)]
        good = torch.tensor([0 <= p < m.k.shape[0] for p in pages], device=DEV).repeat_interleave(PAGE)[:a + n]
        at = torch.tensor([min(max(p, 0), m.k.shape[0] - 1) for p in pages], device=DEV)
        k = (m.k[at] * m.s[at, :, 0, None, None]).transpose(0, 1).reshape(nkv, -1, hd)[:, :a + n]
        v = (m.v[at] * m.s[at, :, 1, None, None]).transpose(0, 1).reshape(nkv, -1, hd)[:, :a + n]
        k, v = (torch.where(good[None, :, None], t, 0.0) for t in (k, v))
        kn, vn = k.isnan().any(-1), v.isnan()  # what is not finite reaches the rows that see it, and no others
        k, v = k.nan_to_num(), v.nan_to_num()
        x = q[r0:r0 + n].double().view(n, nkv, G, hd).permute(1, 2, 0, 3)
        s = torch.einsum("hgnd,hjd->hgnj", x, k) * scale
        seen = (torch.arange(a + n, device=DEV) <= a + torch.arange(n, device=DEV)[:, None]) & good
        s = s.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None])
        o = torch.einsum("hgnj,hjd->hgnd", p, v)
        size = torch.einsum("hgnj,hjd->hgnd", p, v.abs())
        lost = torch.einsum("nj,hj->hn", seen.double(), kn.double())[:, None] > 0
        lse = torch.where(lost, math.nan, lse)
        o = torch.where(lost[..., None] | (torch.einsum("nj,hjd->hnd", seen.double(), vn.double())[:, None] > 0), math.nan, o)
        delta = 2.0 ** -17 * scale * x.abs().amax(-1) * k.abs().sum(-1).amax(-1)[:, None, None]
        top = torch.where((good[::PAGE])[:, None], m.s[at, :, 1], 0.0).nan_to_num().amax(0)[:, None, None, None]
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -18 + 2 * delta)[..., None] * size + 2.0 ** -32 * 448 * top * (a + n)
        out.append([t.permute(2, 0, 1, 3).reshape(n, nkv * G, hd) for t in (o, tol)]
                   + [t.permute(2, 0, 1).reshape(n, nkv * G) for t in (lse, delta + 2.0 ** -18 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0))] + [r0])
    return out


def pages_for(past, new, seed=3, spare=5):
    """A page table with the pages in any order, and how many pages there are."""
    n = [-(-(a + b) // PAGE) for a, b in zip(past, new)]
    order = torch.randperm(sum(n) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for c in n:
        table.append(order[at:at + c] + [-1] * (max(n + [1]) - c))
        at += c
    return table, len(order)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(new):
    return torch.tensor([0] + new).cumsum(0).tolist()


def empty_cache(ops, n, nkv, hd):
    """A cache whose memory holds NaN everywhere."""
    c = ops.kv_cache(n, nkv, hd)
    c.k.view(torch.uint8).fill_(0x7f)
    c.v.view(torch.uint8).fill_(0xff)
    c.scale.fill_(math.nan)
    return c


def rows(seed, T, heads, hd, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, heads, hd, generator=g) * std * (0.25 + torch.rand(T, heads, 1, generator=g) * 2)).bfloat16().view(T, heads * hd).to(DEV)


def step(ops, cache, model, past, new, table, T=None, max_new=None, G=2, seed=0, vstd=1.0, kstd=1.0):
    """Plan and append of one step; the model too.  Returns (plan, row starts)."""
    nkv, hd = cache.n_kv_heads, cache.head_dim
    T = sum(new) if T is None else T
    k, v = rows(seed + 1, T, nkv, hd, kstd), rows(seed + 2, T, nkv, hd, vstd)
    plan = ops.kv_plan(ints(past), ints(starts(new)), ints(table), T, max(new) if max_new is None else max_new, G * nkv, nkv, hd)
    ops.kv_append(cache, plan, k, v)
    model.append(past, new, table, k, v)
    return plan


def check_attention(ops, cache, model, plan, past, new, table, q, scale=None, normwise=True):
    nkv, hd = cache.n_kv_heads, cache.head_dim
    G = plan.n_heads // nkv
    o = torch.full((plan.T, plan.n_heads * hd), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((plan.n_heads, plan.T), 7.0, device=DEV)
    size = ops.attention_kv_workspace_size(plan)
    ws = torch.full((16 + size + 16,), 255, dtype=torch.uint8, device=DEV)  # 16-byte aligned, and no more
    ops.attention_kv(q, cache, plan, scale=scale, o=o, lse=lse, workspace=ws[16:16 + size])
    assert (ws[:16] == 255).all() and (ws[16 + size:] == 255).all()
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    got, glse = o.double().view(plan.T, plan.n_heads, hd), lse.double().t()
    mine = torch.zeros(plan.T, dtype=torch.bool, device=DEV)
    for ro, tol, rl, ltol, r0 in attention(model, past, new, table, q, G, hd, hd ** -0.5 if scale is None else scale):
        n = ro.shape[0]
        mine[r0:r0 + n] = True
        a, b = got[r0:r0 + n], glse[r0:r0 + n]
        assert torch.equal(a.isnan(), ro.isnan()) and torch.equal(b.isnan(), rl.isnan())
        fine = ~ro.isnan()
        assert (a - ro).abs()[fine].le(tol[fine]).all()
        real = rl.isfinite()
        assert torch.equal(b[~real & ~rl.isnan()], rl[~real & ~rl.isnan()])
        assert (b - rl).abs()[real].le(ltol[real]).all()
        if normwise:
            assert (a - ro)[fine].norm() <= 2e-3 * ro[fine].norm()
    assert (got[~mine] == 7).all() and (glse[~mine] == 7).all()
    return o, lse


APPENDS = [  # kv heads, head size, then steps of (tokens before, new rows) for each sequence
    (1, 64, [([0], [1]), ([1], [1]), ([2], [61]), ([63], [1]), ([64], [1]), ([65], [200])]),
    (2, 128, [([0, 0, 0], [64, 0, 63]), ([64, 0, 63], [1, 5, 2]), ([65, 5, 65], [128, 59, 0]), ([193, 64, 65], [3, 1, 70])]),
    (8, 128, [([0] * 9, [1, 2, 3, 4, 17, 100, 64, 128, 129]), ([1, 2, 3, 4, 17, 100, 64, 128, 129], [1] * 9)]),
    (3, 64, [([0, 0], [1000, 999]), ([1000, 999], [1, 1])]),
]


@pytest.mark.parametrize("case", APPENDS, ids=[str(i) for i in range(len(APPENDS))])
@pytest.mark.parametrize("std", [1.0, 1e-3, 3e37])
def test_append(ops, case, std):
    nkv, hd, steps = case
    last = [a + b for a, b in zip(*steps[-1])]
    table, n = pages_for(last, [0] * len(last))
    cache = empty_cache(ops, n, nkv, hd)
    model = Model(cache)
    for i, (past, new) in enumerate(steps):  # later rows are larger, then smaller: scales grow and stay
        s = min(std * (4.0 ** (i % 3)), 2e37)
        step(ops, cache, model, past, new, table, seed=10 * i, kstd=s, vstd=s / 3)
        model.check(cache)


def test_append_rounds_older_codes_once_more_only_into_subnormals(ops):
    """Small tokens, then one that is 2^12 times larger: the page's scale grows by a power of two."""
    cache = empty_cache(ops, 2, 1, 64)
    model = Model(cache)
    for past, std in ((0, 1.0), (7, 4096.0), (8, 0.01), (9, 1e6)):
        step(ops, cache, model, [past], [7 if past == 0 else 1], [[1, 0]], seed=past, kstd=std, vstd=std)
        model.check(cache)


def test_append_of_zeros_infinities_and_nan(ops):
    cache = empty_cache(ops, 4, 2, 64)
    model = Model(cache)
    k, v = rows(1, 4, 2, 64), rows(2, 4, 2, 64)
    k[0] = 0                       # sequence 0: an all-zero row
    v[1, 3] = math.nan             # sequence 1, kv head 0: its values
    k[2, 70] = -math.inf           # sequence 2, kv head 1: its keys
    table = [[0], [1], [2]]
    for past, new in (([0, 0, 0], [1, 1, 2]), ([1, 1, 2], [1, 2, 1]), ([0, 3, 0], [1, 1, 2])):
        plan = ops.kv_plan(ints(past), ints(starts(new)), ints(table), 4, 2, 4, 2, 64)
        ops.kv_append(cache, plan, k, v)
        model.append(past, new, table, k, v)
        model.check(cache)
        k, v = rows(past[1] + 5, 4, 2, 64), rows(past[1] + 6, 4, 2, 64)  # the poisoned pages stay so until begun anew
    assert cache.scale[1, 0, 1].isnan() and cache.scale[1, 0, 0].isfinite() and cache.scale[2].isfinite().all()


ATTEND = [  # kv heads, query heads of each, head size, tokens before, new rows
    (1, 1, 64, [0], [1]), (1, 1, 128, [1], [1]), (2, 7, 64, [332], [1]), (8, 5, 128, [0, 63, 64, 65, 500], [1, 1, 1, 1, 1]),
    (4, 7, 128, [100, 0, 700], [2, 2, 2]), (8, 8, 128, [1000, 31], [1, 1]), (2, 16, 64, [77, 3000], [1, 1]), (1, 64, 128, [130, 0], [1, 3]),
    (3, 3, 64, [10, 0, 5, 200], [0, 4, 0, 6]), (2, 2, 128, [0, 0, 900], [63, 64, 65]), (8, 5, 128, [70, 1500], [40, 1]),
    (1, 5, 64, [0], [257]), (2, 7, 128, [333, 0, 64], [100, 129, 1]), (2, 4, 128, [6000], [1]), (4, 1, 64, [20000, 3], [1, 1]),
    (2, 8, 64, [1, 2, 3] * 40, [1, 2, 1] * 40), (1, 3, 128, [5000], [300]), (2, 5, 128, [0], [700]), (2, 8, 128, [4000], [33]),
]


@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
def test_attention(ops, case):
    nkv, G, hd, past, new = case
    table, n = pages_for(past, new)
    cache = empty_cache(ops, n, nkv, hd)
    model = Model(cache)
    if max(past):  # what the cache holds before
        step(ops, cache, model, [0] * len(past), past, table, G=G, seed=50)
    plan = step(ops, cache, model, past, new, table, G=G, seed=60)
    q = rows(70, plan.T, nkv * G, hd, 1.5)
    a = check_attention(ops, cache, model, plan, past, new, table, q)
    b = check_attention(ops, cache, model, plan, past, new, table, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_behind_the_last_sequence_and_sequences_without_rows(ops):
    past, new, table = [40, 9, 100], [3, 0, 2], [[0, 1], [2, -1], [3, 4]]
    cache = empty_cache(ops, 5, 2, 64)
    model = Model(cache)
    step(ops, cache, model, [0] * 3, past, table)
    plan = step(ops, cache, model, past, new, table, T=9, max_new=5)
    check_attention(ops, cache, model, plan, past, new, table, rows(4, 9, 4, 64))


def test_pages_that_are_none(ops):
    """Pages below 0 and beyond the cache: append drops their rows, attention passes over them; a row that sees none
    gets zeros and -infinity."""
    for G, n1 in ((2, 3), (8, 90)):
        past, new = [130, 0, 64, 10], [n1, 5, 1, 2]
        table = [[0, 77, 1, 2], [-1, 3, -1, -1], [-5, 1 << 30, -1, -1], [4, -1, -1, -1]]
        cache = empty_cache(ops, 5, 2, 64)
        model = Model(cache)
        step(ops, cache, model, [0] * 4, past, table, G=G)
        plan = step(ops, cache, model, past, new, table, G=G, seed=9)
        model.check(cache)
        o, lse = check_attention(ops, cache, model, plan, past, new, table, rows(4, plan.T, 2 * G, 64))
        assert (o[n1:n1 + 6] == 0).all() and (lse[:, n1:n1 + 6] == -math.inf).all()


def test_arrays_out_of_range_stay_inside(ops):
    """Lengths, rows and tables that no caller should give: nothing but the given memory is touched, and what can be
    served is."""
    cache = empty_cache(ops, 6, 2, 64)
    model = Model(cache)
    table = [[0, 1], [2, 3], [4, 5]]
    step(ops, cache, model, [0] * 3, [70, 70, 70], table)
    q = rows(4, 8, 4, 64)
    for past, start in (([70, -9, 70], [0, 1, 2, 3]), ([1 << 30, 70, 70], [0, 1, 2, 3]), ([70, 70, 70], [5, 2, 400, -7]),
                        ([127, 128, 126], [0, 4, 6, 8]), ([70, 70, 70], [-(1 << 31), (1 << 31) - 1, 8, 8])):
        plan = ops.kv_plan(ints(past), ints(start), ints(table), 8, 3, 4, 2, 64)
        o = torch.full((8, 256), 7.0, dtype=torch.bfloat16, device=DEV)
        ops.attention_kv(q, cache, plan, o=o)
        torch.cuda.synchronize()
        assert ops.device_error() == 0
        # the plan's own reading of them
        p = [min(max(a, 0), 128) for a in past]
        lo = [min(max(a, 0), 8) for a in start[:-1]]
        n = [max(0, min(min(max(b, a), 8) - a, 3, 128 - c)) for a, b, c in zip(lo, start[1:], p)]
        for ro, tol, _, _, r0 in attention(model, p, n, table, q, 2, 64, 0.125, start=lo):
            c = ro.shape[0]
            assert torch.equal(ro.isnan(), o[r0:r0 + c].double().view(c, 4, 64).isnan())
            fine = ~ro.isnan()
            assert (o[r0:r0 + c].double().view(c, 4, 64) - ro).abs()[fine].le(tol[fine]).all()


def test_scales_that_differ_widely_between_pages(ops):
    """Pages whose values are 2^20 apart, among them all-zero ones, and keys likewise."""
    for G, n in ((3, 1), (8, 40)):
        table = [[0, 1, 2, 3, 4, 5, 6]]
        cache = empty_cache(ops, 7, 2, 128)
        model = Model(cache)
        for i, (ks, vs) in enumerate(((1.0, 1.0), (0.5, 2.0 ** -20), (0.0, 0.0), (1.0, 2.0 ** 10), (2.0, 1.0))):
            step(ops, cache, model, [64 * i], [64], table, seed=i, kstd=ks, vstd=vs)
        plan = step(ops, cache, model, [320], [n], table, G=G, seed=9, vstd=2.0 ** -10)
        check_attention(ops, cache, model, plan, [320], [n], table, rows(5, n, 2 * G, 128, 1.5))


def test_scores_that_grow_from_page_to_page(ops):
    """Every page's largest score is far above the ones before it, in one kv head; far below in the other."""
    for G, n in ((2, 1), (8, 40)):
        table = [[0, 1, 2, 3, 4, 5]]
        cache = empty_cache(ops, 6, 2, 128)
        model = Model(cache)
        for i in range(5):
            k, v = rows(i, 64, 2, 128), rows(i + 20, 64, 2, 128)
            k.view(64, 2, 128)[:, 0] *= 2.0 ** i
            k.view(64, 2, 128)[:, 1] *= 2.0 ** (4 - i)
            plan = ops.kv_plan(ints([64 * i]), ints([0, 64]), ints(table), 64, 64, 2 * G, 2, 128)
            ops.kv_append(cache, plan, k, v)
            model.append([64 * i], [64], table, k, v)
        plan = step(ops, cache, model, [320], [n], table, G=G, seed=9)
        check_attention(ops, cache, model, plan, [320], [n], table, rows(5, n, 2 * G, 128, 1.5), normwise=False)


def test_large_and_tiny_queries_and_peaked_rows(ops):
    for n in (1, 60):
        table = [[3, 1, 0, 2, 4]]
        cache = empty_cache(ops, 5, 1, 64)
        model = Model(cache)
        step(ops, cache, model, [0], [200], table, seed=1)
        plan = step(ops, cache, model, [200], [n], table, G=4, seed=2)
        for std, scale in ((40.0, None), (1e-30, None), (0.0, None), (3e30, 1e-30), (1.0, 20.0)):
            q = rows(6, n, 4, 64, std)
            check_attention(ops, cache, model, plan, [200], [n], table, q, scale=scale, normwise=False)


def test_non_finite_queries_and_pages_reach_their_own_rows_only(ops):
    for n in (2, 50):
        past, new, table = [90, 90], [n, n], [[0, 1, 2], [3, 4, 5]]
        cache = empty_cache(ops, 6, 2, 64)
        model = Model(cache)
        step(ops, cache, model, [0, 0], past, table, G=3)
        plan = step(ops, cache, model, past, new, table, G=3, seed=5)
        q = rows(6, 2 * n, 6, 64)
        ref = check_attention(ops, cache, model, plan, past, new, table, q)[0]
        q2 = q.clone()
        q2[1, 64 * 4 + 5] = math.nan
        o = ops.attention_kv(q2, cache, plan)[0]
        bad = o.view(2 * n, 6, 64).isnan()
        assert bad[1, 4].all() and bad.sum() == 64
        good = ~bad
        assert torch.equal(o.view(2 * n, 6, 64)[good], ref.view(2 * n, 6, 64)[good])
        cache.scale[4, 1, 0] = math.nan  # what append makes of a key that is not finite
        model.s[4, 1, 0] = math.nan
        check_attention(ops, cache, model, plan, past, new, table, q)


def test_a_page_that_is_not_finite_stays_out_of_the_rows_before_it(ops):
    """A new page whose keys, values or both are not finite: rows of the same tile that end before it are untouched."""
    for n in (2, 40):
        past, table = [127 if n == 2 else 100], [[0, 1, 2]]
        for bad_k, bad_v in ((True, False), (False, True), (True, True)):
            cache = empty_cache(ops, 3, 2, 64)
            model = Model(cache)
            step(ops, cache, model, [0], past, table, G=3)
            k, v = rows(1, n, 2, 64), rows(2, n, 2, 64)
            if bad_k:
                k[n - 1, 70] = math.inf
            if bad_v:
                v[n - 1, 3] = math.nan
            plan = ops.kv_plan(ints(past), ints([0, n]), ints(table), n, n, 6, 2, 64)
            ops.kv_append(cache, plan, k, v)
            model.append(past, [n], table, k, v)
            model.check(cache)
            o, _ = check_attention(ops, cache, model, plan, past, [n], table, rows(6, n, 6, 64), normwise=False)
            new_page = [past[0] + i >= 128 for i in range(n)]
            assert o.view(n, 6, 64).isnan().any(2).any(1).tolist() == new_page


def test_strided_rows(ops):
    past, new, table = [70, 5], [2, 45], [[0, 1], [2, 3]]
    cache = empty_cache(ops, 4, 2, 64)
    model = Model(cache)
    wide = torch.full((47, 2048), 7.0, dtype=torch.bfloat16, device=DEV)
    q, k, v, o = wide[:, 8:520], wide[:, 520:648], wide[:, 712:840], wide[:, 1024:1536]
    q.copy_(rows(1, 47, 8, 64))
    k.copy_(rows(2, 47, 2, 64))
    v.copy_(rows(3, 47, 2, 64))
    step(ops, cache, model, [0, 0], past, table, G=4)
    plan = ops.kv_plan(ints(past), ints(starts(new)), ints(table), 47, 45, 8, 2, 64)
    ops.kv_append(cache, plan, k, v)
    model.append(past, new, table, k, v)
    model.check(cache)
    want, _ = check_attention(ops, cache, model, plan, past, new, table, q.contiguous())
    ops.attention_kv(q, cache, plan, o=o)
    assert torch.equal(o, want) and (wide[:, 1536:] == 7).all() and (wide[:, 840:1024] == 7).all()


def test_streams_and_replays_of_a_whole_step(ops):
    """Plan, append and attention captured once; lengths, table and rows change between replays."""
    nkv, G, hd, n = 2, 5, 128, 6
    table = ints([[4 * i + j for j in range(4)] for i in range(n)])
    past, start = ints([0] * n), ints([0, 3, 4, 4, 5, 6, 40])
    cache = empty_cache(ops, 4 * n, nkv, hd)
    q, k, v = rows(1, 40, nkv * G, hd), rows(2, 40, nkv, hd), rows(3, 40, nkv, hd)
    plan = ops.kv_plan(past, start, table, 40, 34, nkv * G, nkv, hd)
    ws = torch.full((ops.attention_kv_workspace_size(plan),), 255, dtype=torch.uint8, device=DEV)
    o = torch.zeros(40, nkv * G * hd, dtype=torch.bfloat16, device=DEV)

    def call(stream=None):
        ops.kv_plan(past, start, table, 40, 34, nkv * G, nkv, hd, plan=plan, stream=stream)
        ops.kv_append(cache, plan, k, v, stream=stream)
        ops.attention_kv(q, cache, plan, o=o, workspace=ws, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    for i, lens in enumerate(([3, 1, 0, 1, 1, 34], [30, 90, 64, 127, 1, 100])):
        past.copy_(ints(lens))
        table.copy_(table.flip(0) if i else table)
        q.copy_(rows(20 + i, 40, nkv * G, hd))
        k.copy_(rows(30 + i, 40, nkv, hd))
        saved = [t.clone() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.scale)]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.scale)]
        for t, x in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.scale), saved):
            t.copy_(x)
        o.zero_()
        call()
        torch.cuda.synchronize()
        for x, y in zip(got, (o, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.scale)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    with pytest.raises(ValueError):
        ops.kv_plan(past, start, table, 40, 33, nkv * G, nkv, hd, plan=plan)
    with pytest.raises(ValueError):
        ops.attention_kv(q[:39], cache, plan)
    with pytest.raises(ValueError):
        ops.attention_kv(q, empty_cache(ops, 3, 4, hd), plan)


def test_offsets_past_32_bits(ops):
    """A cache of more than 2^32 bytes of keys, its last pages in use."""
    n, nkv, hd = 66000, 8, 128  # 4.3 GB of keys
    cache = ops.kv_cache(n, nkv, hd)
    table = [[n - 1, 0, n - 2]]
    for t in (cache.k, cache.v):
        t.view(torch.uint8)[[0, n - 1, n - 2]] = 0
    small = ops.KVCache(cache.k[[0, 0, 0]].contiguous(), cache.v[[0, 0, 0]].contiguous(), cache.scale[[0, 0, 0]].contiguous())
    k, v, q = rows(1, 150, nkv, hd), rows(2, 150, nkv, hd), rows(3, 150, 16, hd)
    outs = []
    for c, tb in ((cache, table), (small, [[2, 0, 1]])):
        plan = ops.kv_plan(ints([0]), ints([0, 150]), ints(tb), 150, 150, 16, nkv, hd)
        ops.kv_append(c, plan, k, v)
        outs.append(ops.attention_kv(q, c, plan)[0])
    assert torch.equal(*outs)


WIDE = [(1, 1024, 128, [70], [1]), (1, 1024, 64, [5, 0], [2, 1]), (256, 1, 64, [3, 64], [1, 2]), (256, 4, 64, [90], [20]),
        (2, 17, 128, [200, 64], [1, 1]), (4, 8, 128, [640, 127, 0], [2, 3, 2]), (8, 1, 64, [0] * 20, [17] * 20),
        (2, 3, 128, [37 * i % 150 for i in range(60)], [(5, 6, 43, 44, 90)[i % 5] for i in range(60)]), (2, 5, 128, [0], [1639])]


@pytest.mark.parametrize("case", WIDE, ids=[str(i) for i in range(len(WIDE))])
def test_many_heads_and_rows_about_a_tile_s(ops, case):
    test_attention(ops, case)


def test_as_many_sequences_as_a_plan_takes(ops):
    """Elements' bounds only: over one sequence's 128 elements the norm of the roundings may pass 2e-3 of the result's.
    A rounding is spread over 2^-8 of a power of two that the value is one to two times of: 2^-8 / sqrt(3) = 2.3e-3 of it
    where the large values lie just above theirs."""
    nkv, G, hd, n = 1, 2, 64, 4096
    past = [(0, 1, 63, 64, 130)[i * 7 % 5] for i in range(n)]
    new = [0 if i % 11 == 3 else 1 for i in range(n)]
    table, pages = pages_for(past, new)
    cache = empty_cache(ops, pages, nkv, hd)
    for t in (cache.k, cache.v):  # what the cache holds before: any finite codes above zero
        t.view(torch.uint8).copy_(torch.randint(0, 0x7f, t.shape, dtype=torch.uint8, generator=torch.Generator().manual_seed(1)))
    cache.scale.fill_(2.0 ** -7)
    T = sum(new)
    k, v, q = rows(1, T, nkv, hd), rows(2, T, nkv, hd), rows(3, T, nkv * G, hd)
    plan = ops.kv_plan(ints(past), ints(starts(new)), ints(table), T, 1, G * nkv, nkv, hd)
    ops.kv_append(cache, plan, k, v)
    o, lse = ops.attention_kv(q, cache, plan, want_lse=True)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    live = torch.tensor(new, device=DEV) > 0
    last, tab = torch.tensor(past, device=DEV)[live], torch.tensor(table, device=DEV)[live].clamp(min=0)
    ck = (cache.k.double() * cache.scale[..., 0, None, None])[tab, 0].view(T, -1, hd)
    cv = (cache.v.double() * cache.scale[..., 1, None, None]).transpose(2, 3)[tab, 0].reshape(T, -1, hd)
    mine = tab.gather(1, (last // PAGE)[:, None])[:, 0]
    for c, (x, held) in enumerate(((k, ck), (v, cv))):
        s = cache.scale[mine, 0, c].double()[:, None]
        assert torch.equal(held[torch.arange(T, device=DEV), last], e4m3(x.double() / s) * s)
    seen = torch.arange(ck.shape[1], device=DEV) <= last[:, None]
    ck, cv = (torch.where(seen[..., None], x, 0.0) for x in (ck, cv))
    x = q.double().view(T, G, hd)
    s = torch.einsum("tgd,tjd->tgj", x, ck).masked_fill(~seen[:, None], -math.inf) * hd ** -0.5
    p = s.softmax(-1)
    want, size = torch.einsum("tgj,tjd->tgd", p, cv), torch.einsum("tgj,tjd->tgd", p, cv.abs())
    delta = 2.0 ** -17 * hd ** -0.5 * x.abs().amax(-1) * ck.abs().sum(-1).amax(-1)[:, None]
    top = cache.scale[tab, 0, 1].double().masked_fill(~seen[:, ::PAGE], 0).amax(-1)[:, None, None]
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -18 + 2 * delta)[..., None] * size + 2.0 ** -32 * 448 * top * (last + 1)[:, None, None]
    assert ((o.double().view(T, G, hd) - want).abs() <= tol).all()
    ref = torch.logsumexp(s, -1)
    assert ((lse.t().double() - ref).abs() <= delta + 2.0 ** -18 + 2.0 ** -22 * ref.abs()).all()


def test_two_calls_at_once_and_two_graphs_in_turn(ops):
    """One plan and one cache, read by calls on two streams with a workspace each, and by two captured calls that share
    one and are replayed in turn: the bits of single calls."""
    nkv, G, hd, past, new = 4, 5, 128, [9000, 300, 77], [1, 90, 2]
    table, n = pages_for(past, new)
    cache = empty_cache(ops, n, nkv, hd)
    model = Model(cache)
    step(ops, cache, model, [0] * 3, past, table, G=G)
    plan = step(ops, cache, model, past, new, table, G=G, seed=9)
    qs = [rows(i, plan.T, nkv * G, hd) for i in (4, 5)]
    want = [check_attention(ops, cache, model, plan, past, new, table, q)[0] for q in qs]
    size = ops.attention_kv_workspace_size(plan)
    spaces = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in qs]
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(8):
        for q, ws, o, s in zip(qs, spaces, outs, streams):
            ops.attention_kv(q, cache, plan, o=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert ops.device_error() == 0 and all(torch.equal(a, b) for a, b in zip(outs, want))
    graphs = []
    for q, o in zip(qs, outs):
        o.zero_()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            ops.attention_kv(q, cache, plan, o=o, workspace=spaces[0])
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert ops.device_error() == 0 and all(torch.equal(a, b) for a, b in zip(outs, want))
