"""Cases of the operators between the projections and the attention core, and of serving from a
cache: the norm of each query and key head with the rotary positions in one pass and its backward
pass, rows appended to an 8-bit paged cache, and attention over that cache.

Plain forms are elementary torch operations in 32 bits (angles in 64); ``own`` switches to the
framework's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
PAGE = 64      # tokens of one page: one scale for its keys and one for its values, for each kv head
TOP = 448.0    # largest e4m3 value
LOW = -126     # smallest exponent of a scale
EPS = 1e-6
BASE = 1e6

# Query heads, kv heads and head size of the stacks this repository builds.
STACKS = {"0.5b": (14, 2, 64), "7b": (28, 4, 128), "32b": (40, 8, 128), "72b": (64, 8, 128)}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token, far into its context: latency
        dict(name="rope 1 row", op="rope", stack="32b", M=1, norm=True, rot=128, interleaved=False, scaling="none", ctx=40000),
        # a ragged batch of prompts; half of each head rotated, neighbouring elements paired, stretched
        # to four times its context, no norm
        dict(name="rope 333 rows", op="rope", stack="7b", M=333, norm=False, rot=64, interleaved=True, scaling="yarn", ctx=120000),
        # the prompts of one large serving batch
        dict(name="rope 16384 rows", op="rope", stack="32b", M=16384, norm=True, rot=128, interleaved=False, scaling="none", ctx=32768),
        # the training step of this repository's stack: 512 tokens, gradients of the gains too
        dict(name="rope back 512 rows", op="back", stack="32b", M=512, norm=True, rot=128, interleaved=False, scaling="none", ctx=512, gains=True),
        # a long training batch, frozen gains
        dict(name="rope back 8192 rows", op="back", stack="7b", M=8192, norm=True, rot=128, interleaved=True, scaling="linear", ctx=8192, gains=False),
        # one token of each of 48 users into the cache
        dict(name="append 48 rows", op="append", stack="32b", prompts=0, new=0, decodes=48, step=1, ctx=4000),
        # prompts of eight users into the cache, some of them continued
        dict(name="append 8 prompts", op="append", stack="32b", prompts=8, new=4096, decodes=0, step=1, ctx=700),
        # one user's next token in a short conversation: latency
        dict(name="decode 1 user", op="attend", stack="0.5b", prompts=0, new=0, decodes=1, step=1, ctx=332, lse=False),
        # a decode batch of 48 users with contexts of very different lengths
        dict(name="decode 48 users", op="attend", stack="32b", prompts=0, new=0, decodes=48, step=1, ctx=16000, lse=False),
        # two users with very long contexts, two proposed tokens each
        dict(name="decode 2 long", op="attend", stack="7b", prompts=0, new=0, decodes=2, step=2, ctx=130000, lse=True),
        # a chunk of two users' prompts behind what the cache holds already: the most arithmetic
        dict(name="chunk 2 prompts", op="attend", stack="32b", prompts=2, new=1800, decodes=0, step=1, ctx=6000, lse=True),
        # prompts and decode rows in one ragged batch
        dict(name="mixed 33 users", op="attend", stack="7b", prompts=3, new=700, decodes=30, step=1, ctx=4000, lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "back", "append", "attend", "attend"))
    stack = rng.choice(sorted(STACKS))
    nh, nkv, hd = STACKS[stack]
    if op in ("rope", "back"):
        norm, rot = rng.random() < 0.7, 16 * rng.randint(1, hd // 16)
        c = dict(op=op, stack=stack, M=_log(rng, 1, 8192), norm=norm, rot=rot, interleaved=rng.random() < 0.5,
                 scaling=rng.choice(("none", "linear", "yarn")), ctx=_log(rng, 16, 200000))
        return dict(c, gains=norm and rng.random() < 0.6) if op == "back" else c
    if op == "append":
        return dict(op=op, stack=stack, prompts=rng.randint(0, 6), new=_log(rng, 1, 4096), decodes=rng.randint(1, 64), step=rng.randint(1, 4),
                    ctx=_log(rng, 1, 8192))
    while True:
        many = rng.random() < 0.5
        c = dict(op=op, stack=stack, prompts=rng.randint(1, 4) if many else 0, new=_log(rng, 2, 2048), decodes=rng.randint(0 if many else 1, 48),
                 step=rng.randint(1, 3), ctx=_log(rng, 1, 60000), lse=rng.random() < 0.5)
        past, new = _batch(c)
        if work(c)["flops"] <= 2.5e11 and len(past) * max(past) * nkv * hd <= 6e8 and sum(new) * nh * max(past) <= 7e8:
            return c


def _batch(case):
    """Tokens in the cache and new rows of each sequence: prompts first, then decoding ones."""
    rng = random.Random(17)
    p, d, n, c = case["prompts"], case["decodes"], case["new"], case["ctx"]
    new = [n if i == 0 else rng.randint(max(1, n // 4), n) for i in range(p)] + [case["step"]] * d
    past = [c if i == 0 else rng.randint(0, c) for i in range(p)] + [c if i == 0 else rng.randint(c // 8, c) for i in range(d)]
    return past, new


# ------------------------------------------------------------------------------ states
def _inv_freq(case):
    """Rotary frequencies (64 bits) and the factor of cosine and sine: plain, positions divided by
    eight (linear), or YaRN from 32768 positions to four times as many."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = BASE ** (-2 * i / rot)
    if case["scaling"] == "linear":
        return f / 8, 1.0
    if case["scaling"] == "yarn":
        def at(turns):
            return rot * math.log(32768 / (2 * math.pi * turns)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / 4 * ramp, 0.1 * math.log(4) + 1
    return f, 1.0


def _prepare_rope(case, seed):
    g, h = torch.Generator(DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
    nh, nkv, hd = STACKS[case["stack"]]
    m = case["M"]

    def rows(heads, std):  # projections' outputs: the heads' sizes differ
        x = torch.randn(m, heads, hd, generator=g, device=DEV) * (std * (0.5 + torch.rand(heads, 1, generator=g, device=DEV)))
        return x.bfloat16().view(m, heads * hd)
    s = dict(case=case, q=rows(nh, 2.0), k=rows(nkv, 4.0), gq=None, gk=None)
    if case["norm"]:
        s["gq"], s["gk"] = (1 + 0.2 * torch.randn(hd, generator=g, device=DEV) for _ in range(2))
    # sequences of up to ctx tokens behind one another, each from a place of its own
    start = torch.randint(0, case["ctx"], (m,), generator=h)
    length = torch.randint(1, max(2, min(case["ctx"], m)), (m,), generator=h)
    end = torch.cumsum(length, 0)
    seq = torch.searchsorted(end, torch.arange(m), right=True)
    pos = start[seq] + torch.arange(m) - (end - length)[seq]
    s["pos"] = pos.to(torch.int32).to(DEV)
    freq, s["factor"] = _inv_freq(case)
    s["freq"] = freq.to(DEV)
    if case["op"] == "back":
        s["dq"], s["dk"] = rows(nh, 1e-3), rows(nkv, 1e-3)
    if own:
        from weight_streaming_nf4_gb300 import ops
        s["rope"] = ops.rope(case["rot"], inv_freq=freq.tolist(), interleaved=case["interleaved"], factor=s["factor"])
        s["oq"], s["ok"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if case["op"] == "back":
            s["dgq"], s["dgk"] = (torch.empty(hd, device=DEV) if case["gains"] else None for _ in range(2))
            s["ws"] = torch.empty(ops.qk_norm_rope_workspace_size(m, nh, nkv, hd), dtype=torch.uint8, device=DEV)
    return s


def _power(top):
    """Scales: the smallest powers of two that hold the largest sizes, NaN where one is not finite."""
    f, e = torch.frexp(top.double() / TOP)
    e = torch.where(top > 0, e - (f == 0.5).to(e.dtype), torch.full_like(e, LOW)).clamp(min=LOW)
    return torch.where(top.isfinite(), torch.ldexp(torch.ones((), device=top.device), e), torch.full((), math.nan, device=top.device))


def _prepare_cache(case, seed):
    g, h = torch.Generator(DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
    nh, nkv, hd = STACKS[case["stack"]]
    past, new = _batch(case)
    n, t = len(past), sum(new)
    pages = [-(-(a + b) // PAGE) for a, b in zip(past, new)]
    total = sum(pages) + 3  # some pages are nobody's
    order = torch.randperm(total, generator=h).to(torch.int32)
    table = torch.full((n, max(pages)), -1, dtype=torch.int32)
    first = 0
    for i, p in enumerate(pages):
        table[i, :p] = order[first:first + p]
        first += p
    s = dict(case=case, table=table.to(DEV), past=torch.tensor(past, dtype=torch.int32, device=DEV), T=t, pages=pages,
             start=torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(DEV))
    s["k"] = torch.empty(total, nkv, PAGE, hd, dtype=torch.float8_e4m3fn, device=DEV)
    s["v"] = torch.empty(total, nkv, hd, PAGE, dtype=torch.float8_e4m3fn, device=DEV)
    s["scale"] = torch.empty(total, nkv, 2, device=DEV)
    for a in range(0, total, 4096):  # what the cache holds; the places behind a sequence's end hold older tokens
        for i, x in enumerate((s["k"][a:a + 4096], s["v"][a:a + 4096])):
            y = torch.randn(x.shape, generator=g, device=DEV) * (0.5 + torch.rand(1, nkv, 1, 1, generator=g, device=DEV))
            sc = _power(y.abs().amax((2, 3)))
            s["scale"][a:a + 4096, :, i] = sc
            x.copy_(y / sc[:, :, None, None])
    if case["op"] == "append":
        s["nk"], s["nv"] = ((torch.randn(t, nkv * hd, generator=g, device=DEV) * 1.5).bfloat16() for _ in range(2))
        # the touched pages, what of each is older and what is new
        at = [(i, p) for i in range(n) for p in range(past[i] // PAGE, pages[i])]
        begin = torch.tensor([0] + new).cumsum(0).tolist()
        tok = torch.tensor([begin[i] + p * PAGE - past[i] for i, p in at])[:, None] + torch.arange(PAGE)
        inside = (tok >= torch.tensor([begin[i] for i, _ in at])[:, None]) & (tok < torch.tensor([begin[i + 1] for i, _ in at])[:, None])
        older = torch.arange(PAGE) < torch.tensor([past[i] - p * PAGE for i, p in at])[:, None]
        s["page"] = torch.tensor([int(table[i, p]) for i, p in at]).to(DEV)
        s["tok"], s["new"], s["old"] = tok.clamp(0, t - 1).to(DEV), inside.to(DEV), older.to(DEV)
    else:
        # queries after their norm: a few keys stand out
        s["q"] = (torch.randn(t, nh, hd, generator=g, device=DEV) * 1.5).bfloat16().view(t, nh * hd)
        p = case["prompts"]
        s["groups"] = [(a, b, max(new[a:b]), max(pages[a:b])) for a, b in ((0, p), (p, n)) if b > a]
    if own:
        from weight_streaming_nf4_gb300 import ops
        s["cache"] = ops.KVCache(s["k"], s["v"], s["scale"])
        s["plan"] = ops.kv_plan(s["past"], s["start"], s["table"], t, max(new), nh, nkv, hd)  # one for a step: all layers share it
        if case["op"] == "attend":
            s["o"] = torch.empty(t, nh * hd, dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty(nh, t, device=DEV) if case["lse"] else None
            s["ws"] = torch.empty(ops.attention_kv_workspace_size(s["plan"]), dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    return _prepare_rope(case, seed) if case["op"] in ("rope", "back") else _prepare_cache(case, seed)


# ------------------------------------------------------------------------- plain forms
def _turned(x, s, back):
    """x [M, heads, hd] with its first elements rotated in pairs by the rows' angles, or back."""
    c = s["case"]
    rot = c["rot"]
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = ((t * s["factor"]).float()[:, None, :] for t in (angle.cos(), angle.sin()))
    if back:
        sin = -sin
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _heads(x, hd):
    return x.float().view(x.shape[0], -1, hd)


def _rope_fwd(x, gain, s):
    hd = STACKS[s["case"]["stack"]][2]
    y = _heads(x, hd)
    if gain is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gain
    return _turned(y, s, False).bfloat16().view(x.shape)


def _rope_bwd(x, dy, gain, s):
    """Gradients of x and of the gain."""
    hd = STACKS[s["case"]["stack"]][2]
    d = _turned(_heads(dy, hd), s, True)
    if gain is None:
        return d.bfloat16().view(x.shape), None
    y = _heads(x, hd)
    r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    y = y * r
    e = d * gain
    dx = r * (e - y * (e * y).mean(-1, keepdim=True))
    return dx.bfloat16().view(x.shape), (d * y).sum((0, 1))


def _plain_rope(s):
    if s["case"]["op"] == "rope":
        return dict(q=_rope_fwd(s["q"], s["gq"], s), k=_rope_fwd(s["k"], s["gk"], s))
    (dq, dgq), (dk, dgk) = _rope_bwd(s["q"], s["dq"], s["gq"], s), _rope_bwd(s["k"], s["dk"], s["gk"], s)
    return dict(dq=dq, dk=dk, dgq=dgq, dgk=dgk) if s["case"]["gains"] else dict(dq=dq, dk=dk)


def _put(codes, scale, rows, s):
    """New rows into the touched pages [n, kv heads, PAGE, hd]: a page that goes on keeps a scale no
    smaller than it had, and its older codes are rounded again where the scale grows."""
    old, new = s["old"][:, None, :, None], s["new"][:, None, :, None]
    zero = torch.zeros((), device=DEV)
    x = torch.where(new, rows.float()[s["tok"]].view(*s["tok"].shape, -1, codes.shape[3]).transpose(1, 2), zero)
    now = _power(x.abs().amax((2, 3)))
    now = torch.where(s["old"][:, :1], torch.where(scale > now, scale, now), now)
    ratio = torch.where(s["old"][:, :1], scale / now, torch.ones((), device=DEV))[:, :, None, None]
    again = (torch.where(old, codes.float(), zero) * ratio).to(torch.float8_e4m3fn)
    fresh = (x / now[:, :, None, None]).to(torch.float8_e4m3fn)
    out = torch.where(new, fresh.float(), torch.where(old, again.float(), codes.float()))
    return out.to(torch.float8_e4m3fn), now


def _plain_append(s):
    p = s["page"]
    k, ks = _put(s["k"][p], s["scale"][p, :, 0], s["nk"], s)
    v, vs = _put(s["v"][p].transpose(2, 3), s["scale"][p, :, 1], s["nv"], s)
    s["k"].view(torch.uint8)[p] = k.view(torch.uint8)
    s["v"].view(torch.uint8)[p] = v.transpose(2, 3).contiguous().view(torch.uint8)
    s["scale"][p] = torch.stack([ks, vs], -1)
    return dict(k=s["k"], v=s["v"], scale=s["scale"])


def _attend(s, a, b, rows, pages, o, lse):
    """Sequences a to b - 1, padded to `rows` new rows and `pages` pages."""
    nh, nkv, hd = STACKS[s["case"]["stack"]]
    n, g = b - a, nh // nkv
    at = s["table"][a:b, :pages].clamp(min=0).long()
    sc = s["scale"][at].permute(0, 2, 1, 3)[..., None]  # [n, nkv, pages, 2, 1]
    k = (s["k"][at].float().permute(0, 2, 1, 3, 4) * sc[:, :, :, 0:1]).reshape(n, nkv, pages * PAGE, hd)
    v = (s["v"][at].float().permute(0, 2, 1, 4, 3) * sc[:, :, :, 1:2]).reshape(n, nkv, pages * PAGE, hd)
    i = torch.arange(rows, device=DEV)
    start, count = s["start"][a:b].long(), (s["start"][a + 1:b + 1] - s["start"][a:b]).long()
    row = (start[:, None] + i).clamp(max=s["T"] - 1)
    q = s["q"].view(-1, nkv, g, hd)[row].float().permute(0, 2, 1, 3, 4).reshape(n, nkv, rows * g, hd)
    x = (q @ k.transpose(2, 3)).view(n, nkv, rows, g, -1) / math.sqrt(hd)
    seen = torch.arange(pages * PAGE, device=DEV) <= (s["past"][a:b, None] + i)[:, :, None]
    x = x.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    y = (x.view(n, nkv, rows * g, -1) @ v).view(n, nkv, rows, g, hd) / total
    real = i < count[:, None]
    o[row[real]] = y.permute(0, 2, 1, 3, 4).reshape(n, rows, nh * hd)[real]
    lse[row[real]] = (top + total.log()).permute(0, 2, 1, 3, 4).reshape(n, rows, nh)[real]


def _plain_attend(s):
    nh, nkv, hd = STACKS[s["case"]["stack"]]
    o, lse = torch.empty(s["T"], nh * hd, device=DEV), torch.empty(s["T"], nh, device=DEV)
    [_attend(s, *group, o, lse) for group in s["groups"]]
    o = o.bfloat16()
    return dict(o=o, lse=lse.t().contiguous()) if s["case"]["lse"] else dict(o=o)


def _own(s):
    from weight_streaming_nf4_gb300 import ops
    c = s["case"]
    hd = STACKS[c["stack"]][2]
    if c["op"] == "rope":
        q, k = ops.qk_norm_rope_fwd(s["q"], s["k"], hd, s["rope"], s["pos"], q_gain=s["gq"], k_gain=s["gk"], eps=EPS, q_out=s["oq"], k_out=s["ok"])
        return dict(q=q, k=k)
    if c["op"] == "back":
        dq, dk, dgq, dgk = ops.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], hd, s["rope"], s["pos"], q_gain=s["gq"], k_gain=s["gk"], eps=EPS,
                                                dq=s["oq"], dk=s["ok"], dq_gain=s["dgq"], dk_gain=s["dgk"], want_gains=c["gains"], workspace=s["ws"])
        return dict(dq=dq, dk=dk, dgq=dgq, dgk=dgk) if c["gains"] else dict(dq=dq, dk=dk)
    if c["op"] == "append":
        ops.kv_append(s["cache"], s["plan"], s["nk"], s["nv"])
        return dict(k=s["k"], v=s["v"], scale=s["scale"])
    o, lse = ops.attention_kv(s["q"], s["cache"], s["plan"], o=s["o"], lse=s["lse"], workspace=s["ws"])
    return dict(o=o, lse=lse) if c["lse"] else dict(o=o)


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "back": _plain_rope, "append": _plain_append, "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ work
def work(case):
    nh, nkv, hd = STACKS[case["stack"]]
    if case["op"] in ("rope", "back"):
        each, m = case["M"] * (nh + nkv) * hd, case["M"]
        if case["op"] == "rope":
            return dict(bytes=4 * each + 4 * m + (8 * hd if case["norm"] else 0), flops=each * (8 if case["norm"] else 4))
        x = 2 * each if case["norm"] else 0  # without a norm the inputs are not needed
        return dict(bytes=4 * each + x + 4 * m + (16 * hd if case["gains"] else 0), flops=each * 16)
    past, new = _batch(case)
    row = nkv * hd
    if case["op"] == "append":
        pages = sum(-(-(a + b) // PAGE) - a // PAGE for a, b in zip(past, new))
        return dict(bytes=sum(new) * row * 6 + pages * nkv * 8 + 8 * len(past), flops=sum(new) * row * 6)
    seen = sum(a + b for a, b in zip(past, new))
    pairs = sum(a * b + b * (b + 1) // 2 for a, b in zip(past, new))
    table = sum(-(-(a + b) // PAGE) for a, b in zip(past, new))
    return dict(bytes=seen * row * 2 + table * (nkv * 8 + 4) + sum(new) * nh * (4 * hd + (4 if case["lse"] else 0)), flops=4 * pairs * nh * hd)


# ------------------------------------------------------------------------------ exact
def _exact_turn(case, pos, hd):
    """[M, hd, hd] turned round: what a row's rotation does to a head, as cosines and sines of every element."""
    rot = case["rot"]
    freq, factor = _inv_freq(case)
    cos = torch.ones(pos.numel(), hd, dtype=torch.float64, device=DEV)
    sin = torch.zeros(pos.numel(), hd, dtype=torch.float64, device=DEV)
    other = torch.arange(hd, device=DEV)
    for i, f in enumerate(freq.tolist()):
        x, y = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        angle = torch.remainder(pos.double() * f, 2 * math.pi)
        cos[:, x] = cos[:, y] = factor * torch.cos(angle)
        sin[:, y] = factor * torch.sin(angle)
        sin[:, x] = -sin[:, y]
        other[x], other[y] = y, x
    return cos[:, None], sin[:, None], other


def _exact_rope(case, s):
    hd = STACKS[case["stack"]][2]
    cos, sin, other = _exact_turn(case, s["pos"], hd)
    out = {}
    for n, gain in (("q", s["gq"]), ("k", s["gk"])):
        x = s[n].double().view(case["M"], -1, hd)
        w = torch.ones(hd, dtype=torch.float64, device=DEV) if gain is None else gain.double()
        size = torch.ones(case["M"], x.shape[1], 1, dtype=torch.float64, device=DEV) if gain is None else ((x ** 2).sum(2, keepdim=True) / hd + EPS).sqrt()
        if case["op"] == "rope":
            y = x / size * w
            out[n] = (cos * y + sin * y[:, :, other]).view(case["M"], -1)
            continue
        d = s["d" + n].double().view(case["M"], -1, hd)
        d = cos * d - sin * d[:, :, other]
        dx = d * w / size
        if gain is not None:
            dx = dx - x * (d * w * x).sum(2, keepdim=True) / (hd * size ** 3)
        out["d" + n] = dx.reshape(case["M"], -1)
        if case["gains"]:
            out["dg" + n] = (d * x / size).sum((0, 1))
    return out


def _exact_code(y):
    """The nearest e4m3 values (ties to even)."""
    unit = torch.ldexp(torch.ones_like(y), torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return torch.round(y / unit) * unit


def _exact_append(case, s):
    k, v, scale = s["k"].double(), s["v"].double().transpose(2, 3).contiguous(), s["scale"].double()
    past, new = _batch(case)
    nkv, hd = k.shape[1], k.shape[3]
    row = 0
    for i, (a, b) in enumerate(zip(past, new)):
        for p in range(a // PAGE, s["pages"][i]):
            page = int(s["table"][i, p])
            lo, hi = max(a, p * PAGE), min(a + b, (p + 1) * PAGE)
            kept = lo - p * PAGE
            for which, codes, rows in ((0, k, s["nk"]), (1, v, s["nv"])):
                x = rows[row + lo - a:row + hi - a].double().view(hi - lo, nkv, hd).transpose(0, 1)
                top = x.abs().amax((1, 2)).clamp(min=TOP * 2.0 ** LOW)
                now = torch.ldexp(torch.ones_like(top), torch.frexp(top).exponent - 9)  # 2^-9 TOP < 1: holds most
                now = torch.where(now * TOP < top, 2 * now, now)
                if kept:
                    was = scale[page, :, which]
                    now = torch.maximum(now, was)
                    codes[page, :, :kept] = _exact_code(codes[page, :, :kept] * (was / now)[:, None, None])
                codes[page, :, kept:kept + hi - lo] = _exact_code(x / now[:, None, None])
                scale[page, :, which] = now
        row += b
    return dict(k=k, v=v.transpose(2, 3).contiguous(), scale=scale)


def _exact_attend(case, s):
    nh, nkv, hd = STACKS[case["stack"]]
    o = torch.zeros(s["T"], nh, hd, dtype=torch.float64, device=DEV)
    lse = torch.zeros(nh, s["T"], dtype=torch.float64, device=DEV)
    past, new = _batch(case)
    row = 0
    for i, (a, b) in enumerate(zip(past, new)):
        page = s["table"][i, :s["pages"][i]].long()
        for h in range(nkv):
            k = (s["k"][page, h].double() * s["scale"][page, h, 0].double()[:, None, None]).reshape(-1, hd)[:a + b]
            v = (s["v"][page, h].double() * s["scale"][page, h, 1].double()[:, None, None]).transpose(1, 2).reshape(-1, hd)[:a + b]
            for j in range(h * (nh // nkv), (h + 1) * (nh // nkv)):
                x = s["q"][row:row + b].double().view(b, nh, hd)[:, j] @ k.t() * hd ** -0.5
                later = torch.arange(a + b, device=DEV) > a + torch.arange(b, device=DEV)[:, None]
                x[later] = -math.inf
                lse[j, row:row + b] = torch.logsumexp(x, 1)
                o[row:row + b, j] = torch.softmax(x, 1) @ v
        row += b
    return dict(o=o.view(s["T"], -1), lse=lse) if case["lse"] else dict(o=o.view(s["T"], -1))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "back"):
        return _exact_rope(case, s)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attend(case, s)
