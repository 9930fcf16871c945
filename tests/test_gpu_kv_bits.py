"""The precision of attention over the 8-bit cache, held to what the header states: results whose large terms cancel, so
that the rounding to bf16 does not hide what is lost before it.

Tolerance.  An element is rounded to bf16 once, 2^-8 of it.  Before that, with N tokens seen and p_j their probabilities:
- a probability enters the second product as two fp16 numbers, hi and the rest: off by at most 2^-11 2^-11 = 2^-22 of itself,
  and by 2^-31 of the row's largest p_j S_j (S_j the scale of its page's values) however small it is: the rest's steps end at
  2^-24, half of one is 2^-25, and the largest enters as 2^6 or more.  Codes are 448 at most, so N times 448 2^-31 max_j p_j S_j;
- 2^x and the rounding of x, |x| <= 16: 2^-22 + 2^-24 16 < 2^-19; the sums of p_j and of p_j v_j, N roundings of 2^-24 each;
- a score, delta = scale (2^-18 max_j sum_i |q_i k_ij| + 2^-21 max|q| max_j sum_{i small} |k_ij|): fp32 sums of hd products in two
  parts, and queries that are exact down to 2^-14 of their row's largest element and off by 2^-21.8 of it below (small)."""
import math

import pytest
import torch

from test_gpu_kv import DEV, PAGE, Model, empty_cache, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import ops as o
    return o


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf16(x):
    return x.bfloat16().to(DEV)


def check(ops, k, v, q, past, G, scale=None, pages=None):
    """One sequence: k, v [past + n, nkv, hd] appended, its last n rows' q [n, nkv*G, hd] against 64 bits of the cached values."""
    total, nkv, hd = k.shape
    n, scale = total - past, hd ** -0.5 if scale is None else scale
    pages = list(range(-(-total // PAGE)))[::-1] if pages is None else pages
    cache = empty_cache(ops, len(pages), nkv, hd)
    model = Model(cache)
    flat = [t.reshape(total, nkv * hd) for t in (k, v)]
    for a, b in ((0, past), (past, total)):
        if b > a:
            plan = ops.kv_plan(ints([a]), ints([0, b - a]), ints([pages]), b - a, b - a, nkv * G, nkv, hd)
            ops.kv_append(cache, plan, flat[0][a:b], flat[1][a:b])
            model.append([a], [b - a], [pages], flat[0][a:b], flat[1][a:b])
    model.check(cache)
    o, lse = ops.attention_kv(q.reshape(n, -1), cache, plan, scale=scale, want_lse=True)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    at = torch.tensor(pages, device=DEV)
    kk, vv = ((t[at] * model.s[at, :, c, None, None]).transpose(0, 1).reshape(nkv, -1, hd)[:, :total] for c, t in ((0, model.k), (1, model.v)))
    S = model.s[at, :, 1].t().repeat_interleave(PAGE, 1)[:, :total]
    x = q.double().view(n, nkv, G, hd).permute(1, 2, 0, 3)
    seen = torch.arange(total, device=DEV) <= past + torch.arange(n, device=DEV)[:, None]
    s = (torch.einsum("hgnd,hjd->hgnj", x, kk) * scale).masked_fill(~seen, -math.inf)
    ref = torch.logsumexp(s, -1)
    p = s.softmax(-1)
    want, size = torch.einsum("hgnj,hjd->hgnd", p, vv), torch.einsum("hgnj,hjd->hgnd", p, vv.abs())
    top = x.abs().amax(-1, keepdim=True)
    small = (x.abs() < 2.0 ** -14 * top).double()
    delta = scale * (2.0 ** -18 * torch.einsum("hgnd,hjd->hgnj", x.abs(), kk.abs()).amax(-1)
                     + 2.0 ** -21 * top[..., 0] * torch.einsum("hgnd,hjd->hgnj", small, kk.abs()).amax(-1))
    floor = 2.0 ** -31 * 448 * total * (p * S[:, None, None]).amax(-1)
    rel = 2.0 ** -22 + 2.0 ** -19 + 2 * total * 2.0 ** -24
    tol = 2.0 ** -8 * want.abs() + (rel + 2 * delta)[..., None] * size + floor[..., None]
    got = o.double().view(n, nkv, G, hd).permute(1, 2, 0, 3)
    worst = ((got - want).abs() / tol).max().item()
    assert worst <= 1, worst
    assert ((lse.double().view(nkv, G, n) - ref).abs() <= delta + 2.0 ** -19 + total * 2.0 ** -24 + 2.0 ** -22 * ref.abs()).all()
    return o


FORMS = [  # kv heads, query heads of each, head size, tokens before, new rows: up to 8, up to 16, up to 128 rows a tile, more
    (4, 2, 64, 30, 1), (4, 5, 128, 40, 1), (4, 8, 64, 20, 2), (2, 16, 128, 40, 1), (4, 4, 64, 3, 20), (2, 5, 128, 20, 25),
    (2, 8, 64, 0, 40), (2, 8, 128, 8, 40), (4, 2, 64, 150, 1), (2, 8, 128, 100, 40)]


@pytest.mark.parametrize("form", FORMS, ids=[str(i) for i in range(len(FORMS))])
def test_probabilities_are_not_rounded_to_a_half(ops, form):
    """Values of both signs cancel; scores differ little, so no token decides alone."""
    nkv, G, hd, past, n = form
    g = gen(sum(form))
    k, q = bf16(torch.randn(past + n, nkv, hd, generator=g) * 0.2), bf16(torch.randn(n, nkv * G, hd, generator=g) * 0.5)
    check(ops, k, bf16(torch.randn(past + n, nkv, hd, generator=g)), q, past, G)


WEIGHTS = [  # for each page of the cache: its values' size 2^e, its scores' distance from the others' in powers of two
    [(30, -90), (0, 0), (0, 0)], [(0, 0), (30, -90), (0, 0)], [(0, 0), (0, 0), (30, -90)], [(60, -90), (0, 0), (-3, 0)],
    [(100, -250), (0, 0), (0, 0)], [(0, 0), (100, -250), (0, 0)], [(30, -30), (0, 0), (0, 0)], [(0, 0), (0, 0), (30, -30)],
    [(-45, 45), (45, -45), (0, 0)], [(45, -45), (0, 0), (-45, 45)], [(0, 0), (-40, 12), (-20, 12)], [(-20, -12), (-40, -25), (20, -80)],
    [(8, -8), (12, -12), (4, -4)], [(3, 0), (-4, 7), (12, -9)]]


# With few pages each is a share of its own for up to 16 rows, so their forms have 256 kv heads (whose pages share four
# to a head) and the pattern four times.
@pytest.mark.parametrize("form", [(256, 2, 64, 1, 4), (256, 4, 64, 4, 4), (130, 1, 128, 2, 4), (2, 2, 64, 1, 1), (2, 4, 64, 20, 1), (1, 8, 128, 40, 1)],
                         ids=["8rows", "16rows", "2rows", "whole", "slot", "tile"])
@pytest.mark.parametrize("pages", WEIGHTS, ids=[str(i) for i in range(len(WEIGHTS))])
def test_a_page_counts_by_its_weight_times_its_scale(ops, form, pages):
    """Pages of large values that hardly count, and of small ones that decide: in any order, each keeps its bits."""
    nkv, G, hd, n, times = form
    pages = pages * times
    past = PAGE * len(pages)
    g = gen(n + hd)
    k, v = torch.randn(past + n, nkv, hd, generator=g) * 0.2, torch.randn(past + n, nkv, hd, generator=g)
    k[..., 0] = 0
    for i, (e, d) in enumerate(pages):
        at = slice(PAGE * i, PAGE * (i + 1))
        v[at] *= 2.0 ** e
        k[at, :, 0] = d * math.log(2)
    q = torch.randn(n, nkv * G, hd, generator=g) * 0.3
    q[..., 0] = hd ** 0.5
    check(ops, bf16(k), bf16(v), bf16(q), past, G)


@pytest.mark.parametrize("form", FORMS, ids=[str(i) for i in range(len(FORMS))])
@pytest.mark.parametrize("large", [2.0 ** 6, 448 * 2.0 ** -5, 2.0 ** 20])
def test_small_elements_of_a_query_beside_a_large_one(ops, form, large):
    """One channel of the queries is 2^11 to 2^13 times the others, and the keys hold nothing there: what counts are the
    others' bits.  They are exact down to 2^-14 of the largest."""
    nkv, G, hd, past, n = form
    g = gen(sum(form) + 1)
    k = torch.randn(past + n, nkv, hd, generator=g) * 2
    k[..., 5] = 0
    size = torch.rand(n, nkv * G, hd, generator=g) * 3 + 1  # 1 to 4, 2^-13 to 2^-11 of the largest
    q = size * torch.sign(torch.randn(n, nkv * G, hd, generator=g)) * 2.0 ** -13 * large
    q[..., 5] = large
    scale = 2.0 ** 11 / large * hd ** -0.5
    check(ops, bf16(k), bf16(torch.randn(past + n, nkv, hd, generator=g)), bf16(q), past, G, scale=scale)


@pytest.mark.parametrize("hd,G,n", [(64, 2, 1), (64, 8, 2), (128, 2, 1), (128, 4, 4)], ids=["64-8rows", "64-16rows", "128-8rows", "128-16rows"])
def test_long_sums_of_single_tokens_are_rounded_not_cut_off(ops, hd, G, n):
    """Shares of 128 pages whose first half has positive values and whose second half negative ones: a sum rises, and falls
    to nearly nothing, so the result shows what its additions lose.  The tensor cores' additions cut off: in a page eight,
    each by up to 2^-23 of the page's sum, 2^-20 of the sizes in all; pages are added in fp32, rounded to nearest, 128
    roundings of up to 2^-24 of half the sizes and of either sign, 2^-22 in the mean.  2^-19 of the sizes (root mean
    square), and the rounding to bf16; additions that cut off all the way lose 1024 times up to 2^-24 of a quarter in the
    mean, 2^-16."""
    nkv, share = 8, 128
    units = torch.cuda.get_device_properties(0).multi_processor_count * (8 if hd == 128 else 12) // nkv
    pages = units * share
    g = torch.Generator(DEV).manual_seed(hd + n)
    cache = ops.kv_cache(pages, nkv, hd)
    cache.k.view(torch.uint8).copy_(torch.randint(0, 0x38, cache.k.shape, dtype=torch.uint8, generator=g, device=DEV))  # 0 to 1
    cache.v.view(torch.uint8).copy_(torch.randint(0x30, 0x40, cache.v.shape, dtype=torch.uint8, generator=g, device=DEV))  # 1/2 to 2
    sign = (torch.arange(pages, device=DEV) % share >= share // 2).to(torch.uint8) << 7
    cache.v.view(torch.uint8).bitwise_or_(sign[:, None, None, None])
    cache.scale.fill_(1.0)
    total = pages * PAGE
    q = (torch.randn(n, nkv * G, hd, generator=g, device=DEV) * 0.5).bfloat16()
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    plan = ops.kv_plan(ints([total - n]), ints([0, n]), table, n, n, nkv * G, nkv, hd)
    o, lse = ops.attention_kv(q.view(n, -1), cache, plan, want_lse=True)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    err = own = size = 0.0
    for h in (0, nkv - 1):
        k, v = cache.k[:, h].double().view(total, hd), cache.v[:, h].double().transpose(1, 2).reshape(total, hd)
        x = q.view(n, nkv, G, hd)[:, h].double().reshape(n * G, hd)
        s = x @ k.t() * hd ** -0.5
        s.view(n, G, total)[:, :, total - n:].masked_fill_(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)[:, None], -math.inf)
        ref = torch.logsumexp(s, 1)
        p = s.softmax(1)
        want = p @ v
        got = o.view(n, nkv, G, hd)[:, h].double().reshape(n * G, hd)
        err, own, size = err + (got - want).square().sum().item(), own + want.square().sum().item(), size + (p @ v.abs()).square().sum().item()
        got = lse.view(nkv, G, n)[h].t().reshape(-1).double()
        assert ((got - ref).abs() <= 2.0 ** -19 + 2.0 ** -22 * ref.abs()).all()
    assert own < 2.0 ** -12 * size  # it does cancel
    assert err ** 0.5 <= 2.0 ** -9 * own ** 0.5 + 2.0 ** -19 * size ** 0.5, (err / size) ** 0.5
