"""Cases of the operators for many adapters: the linear with the low-rank adapters of many
requests beside one frozen NF4 projection, its backward pass, and the AdamW step over many
tensors with 32-bit or 8-bit states and gradient clipping for each group of tensors.

Plain forms are elementary torch operations in 32 bits; ``own`` switches to the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda:0"
R = 16  # the framework's adapter rank
BLOCK = 256  # elements of one 8-bit state block
LEVELS = (-1.0, -0.6962, -0.5251, -0.3949, -0.2844, -0.1848, -0.0911, 0.0,
          0.0796, 0.1609, 0.2461, 0.3379, 0.4407, 0.5626, 0.7230, 1.0)
M_TOP = 448.0    # largest e4m3 value
V_TOP = 1.9375   # largest value of the unsigned 4 + 4 bit code
V_LOW = (1 + 1 / 16) * 2.0 ** -15  # its smallest non-zero value

# Linear widths (hidden, kv, intermediate) of the stacks this repository builds.
STACKS = {"0.5b": (896, 128, 4864), "7b": (3584, 512, 18944), "32b": (5120, 1024, 27648)}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token through the 32B attention-output projection: latency
        dict(name="decode 1 row", op="fwd", M=1, N=5120, K=5120, adapters=8, requests=1, adapter="f32"),
        # a decode batch of many users, nearly every row another adapter, kept in bf16 for serving
        dict(name="decode 48 rows", op="fwd", M=48, N=27648, K=5120, adapters=64, requests=48, adapter="bf16"),
        # prompts and decode rows in one ragged batch through the 32B down projection
        dict(name="mixed 333 rows", op="fwd", M=333, N=5120, K=27648, adapters=12, requests=40, adapter="f32"),
        # prompts of eight users through the 7B gate projection
        dict(name="prompts 2048 rows", op="fwd", M=2048, N=18944, K=3584, adapters=8, requests=8, adapter="bf16"),
        # four adapters trained in one batch, 32B attention-output projection, with dropout
        dict(name="train 512 rows", op="bwd", M=512, N=5120, K=5120, adapters=4, requests=4, dropout=0.1, dx="bf16"),
        # a small ragged training batch, 0.5B key projection, no dropout
        dict(name="train 77 rows", op="bwd", M=77, N=128, K=896, adapters=3, requests=5, dropout=0.0, dx="f32"),
        # the largest backward: 32B down projection, six adapters
        dict(name="train 2048 rows", op="bwd", M=2048, N=5120, K=27648, adapters=6, requests=16, dropout=0.1, dx="f32"),
        # the tensors of one layer's adapters of the 0.5B stack: latency
        dict(name="adamw32 one layer", op="adamw", stack="0.5b", layers=1, groups=1, odd=0, bits=32, grad="f32", clip=True, step=3),
        # every adapter tensor of the 32B stack, 32-bit states
        dict(name="adamw32 64 layers", op="adamw", stack="32b", layers=64, groups=1, odd=0, bits=32, grad="f32", clip=True, step=100),
        # four adapters of the 7B stack, one group each, 8-bit states, bf16 gradients, odd tensors beside them
        dict(name="adamw8 four groups", op="adamw", stack="7b", layers=7, groups=4, odd=5, bits=8, grad="bf16", clip=True, step=0),
        # every adapter tensor of the 32B stack, 8-bit states, no clipping
        dict(name="adamw8 64 layers", op="adamw", stack="32b", layers=64, groups=1, odd=0, bits=8, grad="f32", clip=False, step=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "adamw"))
    if op == "adamw":
        return dict(op=op, stack=rng.choice(sorted(STACKS)), layers=_log(rng, 1, 40), groups=rng.randint(1, 6),
                    odd=rng.randint(0, 40), bits=rng.choice((8, 32)), grad=rng.choice(("f32", "bf16")),
                    clip=rng.random() < 0.5, step=rng.randint(0, 2000))
    while True:
        m, n, k = _log(rng, 1, 2048), 64 * _log(rng, 1, 432), 64 * _log(rng, 1, 432)
        if 1 << 22 <= m * n * k <= 2048 * 5120 * 27648:
            break
    c = dict(op=op, M=m, N=n, K=k, adapters=_log(rng, 1, 64), requests=_log(rng, 1, m))
    if op == "fwd":
        return dict(c, adapter=rng.choice(("f32", "bf16")))
    return dict(c, dropout=rng.choice((0.0, 0.05, 0.1)), dx=rng.choice(("f32", "bf16")))


# ------------------------------------------------------------------------------ states
def _rows(case, g):
    """Adapter of each row: requests are runs of rows; now and then one has no adapter (-1)."""
    m, r = case["M"], min(case["requests"], case["M"])
    cut = torch.randperm(m - 1, generator=g)[:r - 1].sort().values + 1
    length = torch.diff(torch.cat([torch.zeros(1, dtype=torch.int64), cut, torch.tensor([m])]))
    a = torch.randint(0, case["adapters"], (r,), generator=g)
    if r >= 4:
        a = torch.where(torch.rand(r, generator=g) < 0.1, torch.full_like(a, -1), a)
    return a.repeat_interleave(length).to(torch.int32)


def _prepare_linear(case, seed):
    g, h = torch.Generator(DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
    m, n, k, na = case["M"], case["N"], case["K"], case["adapters"]

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std
    rows = _rows(case, h)
    s = dict(case=case, rows=rows.to(DEV))
    # NF4 codes of normal weights are spread nearly evenly over the 16 levels
    s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    s["absmax"] = 0.02 * (2.0 + torch.rand(k // 64, n, generator=g, device=DEV))
    s["x"] = randn(m, k).bfloat16()
    s["A"] = (torch.rand(na, R, k, generator=g, device=DEV) * 2 - 1) / math.sqrt(k)
    s["B"] = randn(na, n, R, std=0.01)
    if case.get("adapter") == "bf16":
        s["A"], s["B"] = s["A"].bfloat16(), s["B"].bfloat16()
    p = case.get("dropout", 0.0)
    s["scale"] = (torch.randint(1, 5, (na,), generator=g, device=DEV).float() * 0.5) / (1 - p)
    s["mask"] = None
    if p > 0:  # one keep bit for each element of x
        keep = torch.rand(m, k // 32, 32, generator=g, device=DEV) >= p
        w = (keep.to(torch.int64) << torch.arange(32, device=DEV)).sum(-1)
        s["mask"] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    if case["op"] == "bwd":
        s["dY"] = randn(m, n).bfloat16()
        s["U"] = _shrink(s, s["x"].float(), s["A"].float())  # what the forward kept
    if own:
        from weight_streaming_nf4_gb300 import ops
        s["W"] = ops.NF4Weight(s["codes"], s["absmax"], n, k)
        s["set"] = ops.LoraSet(s["A"], s["B"], s["scale"])
        s["plan"] = ops.lora_multi_plan(s["rows"], na)  # one for a batch: all its linears share it
        s["ws"] = torch.empty(ops.lora_multi_workspace_size(m, n, k, na), dtype=torch.uint8, device=DEV)
        if case["op"] == "fwd":
            s["y"] = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
            s["U"] = torch.empty(m, R, device=DEV)
        else:
            s["dX"] = torch.empty(m, k, dtype=torch.float32 if case["dx"] == "f32" else torch.bfloat16, device=DEV)
            s["dA"], s["dB"] = torch.empty_like(s["A"]), torch.empty_like(s["B"])
    return s


def _sizes(case, h):
    """Elements of each tensor and its group: A and B of every linear of every layer for each
    adapter (= group), and odd-sized tensors (norm gains, biases) shared out among the groups."""
    hid, kv, inter = STACKS[case["stack"]]
    shapes = [(hid, hid), (kv, hid), (kv, hid), (hid, hid), (inter, hid), (inter, hid), (hid, inter)]
    layer = [x * R for n, k in shapes for x in (k, n)]
    sizes, group = [], []
    for i in range(case["groups"]):
        odd = [int(2 ** (torch.rand(1, generator=h).item() * 17)) for _ in range(i, case["odd"], case["groups"])]
        sizes += layer * case["layers"] + odd
        group += [i] * (len(layer) * case["layers"] + len(odd))
    return sizes, group


def _prepare_adamw(case, seed):
    g, h = torch.Generator(DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
    shape = torch.Generator().manual_seed(17)  # sizes go by the case, values by the seed
    sizes, group = _sizes(case, shape)
    blocks = [-(-n // BLOCK) for n in sizes]
    nb, ng = sum(blocks), case["groups"]
    starts = torch.cumsum(torch.tensor([0] + blocks), 0)[:-1] * BLOCK
    of_tensor = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor(blocks))
    # every tensor starts a block; the elements behind a tensor's end hold zeros
    filled = torch.tensor(sizes)[of_tensor] - (torch.arange(nb) * BLOCK - starts[of_tensor])
    real = torch.arange(BLOCK, device=DEV) < filled.to(DEV)[:, None]

    def randn(std):
        return torch.randn(nb, BLOCK, generator=g, device=DEV).mul_(std).mul_(real)
    s = dict(case=case, step=case["step"], block_group=torch.tensor(group)[of_tensor].to(DEV))
    s["p"] = randn(0.02)
    s["g"] = randn(1e-3 * (1 + torch.rand(nb, 1, generator=g, device=DEV)))
    if case["grad"] == "bf16":
        s["g"] = s["g"].bfloat16()
    warm = 0.0 if case["step"] == 0 else 1.0
    m = randn(3e-4 * warm)
    v = (randn(1e-3 * warm).square_() + 1e-8 * warm).mul_(real)
    if case["bits"] == 8:
        s["m"], s["ms"] = _encode_m(m)
        s["v"], s["vs"] = _encode_r(v.sqrt_())
    else:
        s["m"], s["v"] = m, v
    del m, v
    rnd = torch.rand(ng, generator=h, dtype=torch.float64)
    norm = torch.zeros(ng, dtype=torch.float64, device=DEV).index_add_(
        0, s["block_group"], s["g"].double().square_().sum(1)).sqrt().cpu()
    s["lr"], s["beta1"], s["beta2"] = 1e-4 * (1 + rnd), 0.9 - 0.05 * (rnd > 0.5), 0.999 - 0.009 * (rnd > 0.7)
    s["eps"], s["wd"] = torch.full((ng,), 1e-8, dtype=torch.float64), 0.01 * (rnd < 0.8)
    s["max_norm"] = norm * (0.5 + rnd)  # some groups are clipped, some are not
    if own:
        from weight_streaming_nf4_gb300 import ops

        def views(t):
            flat, per = t.view(-1), t.numel() // nb
            first = (starts // BLOCK * per).tolist()
            return [flat[a:a + (n if per == BLOCK else b)] for a, n, b in zip(first, sizes, blocks)]
        eight = {} if case["bits"] == 32 else dict(exp_avg_scales=views(s["ms"]), exp_avg_sq_scales=views(s["vs"]))
        s["plan"] = ops.adamw_plan(views(s["p"]), views(s["g"]), views(s["m"]), views(s["v"]), groups=group, **eight)
        s["groups"] = ops.adamw_groups([dict(lr=a, beta1=b, beta2=c, eps=d, weight_decay=e, max_norm=f, step=case["step"])
                                        for a, b, c, d, e, f in zip(*(s[q].tolist() for q in ("lr", "beta1", "beta2", "eps", "wd", "max_norm")))])
        s["norms"] = torch.zeros(ng, device=DEV)
    return s


def prepare(case, seed):
    return _prepare_adamw(case, seed) if case["op"] == "adamw" else _prepare_linear(case, seed)


# ------------------------------------------------------------------------- plain forms
def _weight(s):
    """The NF4 weight as the framework defines it: level * absmax, rounded to bf16."""
    c = s["codes"].to(torch.int64)
    q = torch.stack([c >> 4, c & 15], -1).view(c.shape[0], -1)
    w = torch.tensor(LEVELS, device=DEV)[q].view(c.shape[0], -1, 64) * s["absmax"].t()[:, :, None]
    return w.bfloat16().float().view(c.shape[0], -1)


def _keep(s):
    w = s["mask"].to(torch.int64) & 0xFFFFFFFF
    return ((w[:, :, None] >> torch.arange(32, device=DEV)) & 1).view(w.shape[0], -1).float()


def _own_slot(s, t):
    """[M, R] -> [M, adapters * R] with row m's values in its adapter's slot, zeros elsewhere."""
    na = s["scale"].numel()
    hit = s["rows"][:, None] == torch.arange(na, device=DEV)
    return (hit[:, :, None] * t[:, None, :]).reshape(t.shape[0], na * R)


def _of_slot(s, t):
    """[M, adapters * R] -> [M, R]: each row's own slot, zeros for a row without an adapter."""
    na = s["scale"].numel()
    hit = s["rows"][:, None] == torch.arange(na, device=DEV)
    return torch.where(hit[:, :, None], t.view(-1, na, R), torch.zeros((), device=DEV)).sum(1)


def _row_scale(s):
    sc = torch.cat([s["scale"], torch.zeros(1, device=DEV)])
    return sc[s["rows"].to(torch.int64)][:, None]


def _shrink(s, x, a):
    if s["mask"] is not None:
        x = x * _keep(s)
    return _of_slot(s, x @ a.view(-1, a.shape[2]).t())


def _plain_fwd(s):
    x, a, b = s["x"].float(), s["A"].float(), s["B"].float()
    u = _shrink(s, x, a)
    y = x @ _weight(s).t()
    y += _own_slot(s, u * _row_scale(s)) @ b.transpose(1, 2).reshape(-1, b.shape[1])
    return dict(y=y.bfloat16(), U=u)


def _plain_bwd(s):
    x, dy = s["x"].float(), s["dY"].float()
    na, n = s["B"].shape[:2]
    k = x.shape[1]
    bcat = s["B"].transpose(1, 2).reshape(na * R, n)
    gs = _own_slot(s, _of_slot(s, dy @ bcat.t()) * _row_scale(s))
    lora = gs @ s["A"].view(na * R, k)
    if s["mask"] is not None:
        keep = _keep(s)
        x, lora = x * keep, lora * keep
    dx = dy @ _weight(s) + lora
    us = _own_slot(s, s["U"] * _row_scale(s))
    db = (dy.t() @ us).view(n, na, R).transpose(0, 1).contiguous()
    da = (gs.t() @ x).view(na, R, k)
    return dict(dX=dx if s["case"]["dx"] == "f32" else dx.bfloat16(), dA=da, dB=db)


def _encode_m(m):
    """Blocks of 256 first moments as e4m3 numbers and one fp32 scale each."""
    scale = m.abs().amax(1, keepdim=True) / M_TOP
    q = torch.where(scale > 0, m / scale.clamp(min=1e-45), torch.zeros((), device=m.device))
    return q.to(torch.float8_e4m3fn), scale


def _encode_r(r):
    """Blocks of 256 roots of second moments as codes of an unsigned number with 4 exponent and
    4 mantissa bits, (1 + (c & 15) / 16) 2^((c >> 4) - 15), code 0 = 0; a non-zero root never gets 0."""
    scale = r.amax(1, keepdim=True) / V_TOP
    q = torch.where(scale > 0, r / scale.clamp(min=1e-45), torch.zeros((), device=r.device))
    f, e = torch.frexp(q.clamp(V_LOW, V_TOP))
    f = torch.round(f * 32)  # 16 .. 32, ties to even
    e = e.to(torch.int32) + (f == 32)
    f = torch.where(f == 32, torch.full_like(f, 16), f)
    c = (e + 14) * 16 + f.to(torch.int32) - 16
    return torch.where(q > 0, c, torch.zeros_like(c)).to(torch.uint8), scale


def _decode_r(c, scale):
    c = c.to(torch.int32)
    r = torch.ldexp(1 + (c & 15) / 16, (c >> 4) - 15)
    return torch.where(c > 0, r, torch.zeros((), device=r.device)) * scale


def _states(s):
    """What the states stand for. Of 8 bits, in bf16: five significant bits at most, times a scale."""
    if s["case"]["bits"] == 32:
        return dict(m=s["m"], v=s["v"])
    return dict(m=(s["m"].float() * s["ms"]).bfloat16(), r=_decode_r(s["v"], s["vs"]).bfloat16(), m_scale=s["ms"], r_scale=s["vs"])


def _plain_adamw(s):
    c, grp = s["case"], s["block_group"]
    s["step"] += 1
    b1, b2 = s["beta1"], s["beta2"]
    hyper = torch.stack([b1, 1 - b1, b2, 1 - b2, 1 - s["lr"] * s["wd"], s["lr"] / (1 - b1 ** s["step"]),
                         1 / (1 - b2 ** s["step"]).sqrt(), s["eps"]]).to(DEV)
    g = s["g"].float()
    out = {}
    if c["clip"]:
        norm = torch.zeros(c["groups"], dtype=torch.float64, device=DEV).index_add_(0, grp, g.double().square().sum(1)).sqrt()
        out["norms"] = norm.float()
        g = g * (s["max_norm"].to(DEV) / (norm + 1e-6)).clamp(max=1.0).float()[grp][:, None]
    b1, nb1, b2, nb2, decay, lr, rb2, eps = hyper.float()[:, grp][:, :, None]
    m, v = (s["m"], s["v"]) if c["bits"] == 32 else (s["m"].float() * s["ms"], _decode_r(s["v"], s["vs"]).square())
    m = m * b1 + g * nb1
    v = v * b2 + g.square() * nb2
    s["p"] = s["p"] * decay - lr * (m / (v.sqrt() * rb2 + eps))
    if c["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["ms"] = _encode_m(m)
        s["v"], s["vs"] = _encode_r(v.sqrt())
    return dict(out, p=s["p"], **_states(s))


def _own(s):
    from weight_streaming_nf4_gb300 import ops
    c = s["case"]
    if c["op"] == "fwd":
        y, u = ops.lora_linear_fwd_multi(s["W"], s["x"], s["set"], s["plan"], mask=s["mask"], y=s["y"], U=s["U"], workspace=s["ws"])
        return dict(y=y, U=u)
    if c["op"] == "bwd":
        dx, da, db = ops.lora_linear_bwd_multi(s["W"], s["x"], s["set"], s["plan"], s["U"], s["dY"], mask=s["mask"],
                                               dX=s["dX"], dA=s["dA"], dB=s["dB"], workspace=s["ws"])
        return dict(dX=dx, dA=da, dB=db)
    ops.adamw_step(s["plan"], s["groups"], clip=c["clip"], norms=s["norms"] if c["clip"] else None)
    out = dict({"norms": s["norms"]} if c["clip"] else {}, p=s["p"])
    if c["bits"] == 32:
        return dict(out, m=s["m"], v=s["v"])
    return dict(out, m=ops.adamw_decode8(s["m"], s["ms"], False, dtype=torch.bfloat16), m_scale=s["ms"],
                r=ops.adamw_decode8(s["v"], s["vs"], True, dtype=torch.bfloat16), r_scale=s["vs"])


def run(state):
    if own:
        return _own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "adamw": _plain_adamw}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ work
def work(case):
    if case["op"] == "adamw":
        sizes, _ = _sizes(case, torch.Generator().manual_seed(17))
        n, g = sum(sizes), 4 if case["grad"] == "f32" else 2
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return dict(bytes=n * (8 + g + state), flops=n * 20)
    m, n, k = case["M"], case["N"], case["K"]
    present = min(case["adapters"], case["requests"], m)
    weight = n * k // 2 + n * k // 16
    if case["op"] == "fwd":
        per = 4 if case["adapter"] == "f32" else 2
        return dict(bytes=weight + 2 * m * (k + n) + 64 * m + present * R * (n + k) * per, flops=2 * m * n * k + 4 * m * R * (n + k))
    mask = m * k // 8 if case["dropout"] > 0 else 0
    return dict(bytes=weight + 2 * m * (k + n) + mask + 64 * m + present * R * (n + k) * 4 + case["adapters"] * R * (n + k) * 4
                + m * k * (4 if case["dx"] == "f32" else 2), flops=2 * m * n * k + 8 * m * R * (n + k))


# ------------------------------------------------------------------------------ exact
def _exact_weight(s):
    q = torch.empty(s["codes"].shape[0], 2 * s["codes"].shape[1], dtype=torch.int64, device=DEV)
    q[:, 0::2], q[:, 1::2] = torch.div(s["codes"], 16, rounding_mode="floor"), s["codes"] % 16
    levels = torch.tensor(LEVELS, dtype=torch.float32, device=DEV).double()
    w = levels[q] * s["absmax"].double().t().repeat_interleave(64, 1)
    return w.to(torch.bfloat16).double()


def _exact_linear(case, s):
    x, w = s["x"].double(), _exact_weight(s)
    xm = x
    if s["mask"] is not None:
        keep = torch.empty_like(x)
        for bit in range(32):
            keep[:, bit::32] = torch.bitwise_and(torch.bitwise_right_shift(s["mask"], bit), 1).double()
        xm = x * keep
    rows = s["rows"].tolist()
    of = {a: torch.tensor([i for i, b in enumerate(rows) if b == a], device=DEV) for a in set(rows) if a >= 0}
    if case["op"] == "fwd":
        y, u = x @ w.t(), torch.zeros(case["M"], R, dtype=torch.float64, device=DEV)
        for a, i in of.items():
            u[i] = xm[i] @ s["A"][a].double().t()
            y[i] += s["scale"][a].double() * (u[i] @ s["B"][a].double().t())
        return dict(y=y, U=u)
    dy, u = s["dY"].double(), s["U"].double()
    dx = dy @ w
    da = torch.zeros(s["A"].shape, dtype=torch.float64, device=DEV)
    db = torch.zeros(s["B"].shape, dtype=torch.float64, device=DEV)
    for a, i in of.items():
        g = s["scale"][a].double() * (dy[i] @ s["B"][a].double())
        part = g @ s["A"][a].double()
        dx[i] += part if s["mask"] is None else part * keep[i]
        da[a], db[a] = g.t() @ xm[i], s["scale"][a].double() * (dy[i].t() @ u[i])
    return dict(dX=dx, dA=da, dB=db)


def _exact_adamw(case, s):
    n, t = case["groups"], case["step"] + 1
    out = dict(p=s["p"].double())
    g = s["g"].double()
    if case["bits"] == 8:
        m = s["m"].double() * s["ms"].double()
        c = s["v"].double()
        r = (16 + c % 16) * 2.0 ** (torch.floor(c / 16) - 19) * s["vs"].double()
        v = torch.where(c == 0, torch.zeros_like(r), r) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    norms = torch.zeros(n, dtype=torch.float64, device=DEV)
    for i in range(n):
        at = s["block_group"] == i
        b1, b2, gi = s["beta1"][i].item(), s["beta2"][i].item(), g[at]
        norms[i] = torch.linalg.vector_norm(gi)
        if case["clip"]:
            gi = gi * min(1.0, s["max_norm"][i].item() / (norms[i].item() + 1e-6))
        m[at] = b1 * m[at] + (1 - b1) * gi
        v[at] = b2 * v[at] + (1 - b2) * gi * gi
        lr = s["lr"][i].item()
        step = m[at] / (1 - b1 ** t) / ((v[at] / (1 - b2 ** t)).sqrt() + s["eps"][i].item())
        out["p"][at] = out["p"][at] * (1 - lr * s["wd"][i].item()) - lr * step
    if case["clip"]:
        out["norms"] = norms
    if case["bits"] == 32:
        return dict(out, m=m, v=v)
    out["m_scale"] = m.abs().amax(1, keepdim=True) / M_TOP
    q = m / out["m_scale"].clamp(min=1e-300)
    unit = 2.0 ** (torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    out["m"] = torch.round(q / unit) * unit * out["m_scale"]
    r = v.sqrt()
    out["r_scale"] = r.amax(1, keepdim=True) / V_TOP
    q = r / out["r_scale"].clamp(min=1e-300)
    unit = 2.0 ** (torch.floor(torch.log2(q.clamp(min=V_LOW))) - 4)
    out["r"] = torch.where(q > 0, (torch.round(q / unit) * unit).clamp(V_LOW, V_TOP), q) * out["r_scale"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(case, s) if case["op"] == "adamw" else _exact_linear(case, s)
