"""Norm and rotary positions of query and key heads, forward and backward, against plain 64-bit forms.

Tolerances.  A result is rounded to bf16 once: 2^-8 of it.  Before that, in fp32 (a rounding is 2^-24): the sum of squares
adds 16 values in turn and four partial sums (20 roundings, 2^-19.6, halved by the root), 1/sqrt and two products are a few
roundings more; an angle is off by 2^-25 half turns (2^-23.3) and sine and cosine by 2^-23; two products and a sum follow.
Together below 2^-19 of |n_a| + |n_b| for each pair.  The backward doubles that chain: 2^-18.  A gradient of a gain sums
its terms (each off by 2^-19 of itself) in chains of fewer than 128 additions: 2^-16 of the sum of sizes."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import ops as o
    return o


def _tables(pos, freq, factor):
    angle = torch.tensor([[math.remainder(math.fmod(p * f, 2 * math.pi), 2 * math.pi) for f in freq] for p in pos.tolist()],
                         dtype=torch.float64, device=DEV)
    return factor * angle.cos()[:, None], factor * angle.sin()[:, None]


def _pairs(rot, il):
    i = torch.arange(rot // 2, device=DEV)
    return (2 * i, 2 * i + 1) if il else (i, i + rot // 2)


def _forward(x, gain, rope, hd):
    """y in the input's precision, and the size that its fp32 errors go by; rope = (cos, sin, rot, interleaved) or None."""
    x = x.reshape(x.shape[0], -1, hd)
    n = x if gain is None else x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * gain
    if rope is None:
        return n, n.abs()
    cos, sin, rot, il = rope
    a, b = _pairs(rot, il)
    y, size = n.clone(), n.abs().clone()
    y[..., a] = n[..., a] * cos - n[..., b] * sin
    y[..., b] = n[..., a] * sin + n[..., b] * cos
    f = (cos.square() + sin.square()).sqrt().amax()
    size[..., a] = size[..., b] = (n[..., a].abs() + n[..., b].abs()) * f
    return y, size


def _inputs(seed, M, nh, nkv, hd, kind="plain"):
    g = torch.Generator().manual_seed(seed)
    rows = [(torch.randn(M, h * hd, generator=g) * 3).bfloat16().to(DEV) for h in (nh, nkv, nh, nkv)]
    gains = [(1 + 0.3 * torch.randn(hd, generator=g)).to(DEV) for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (M,), generator=g, dtype=torch.int32)
    if kind == "far":  # the ends of the range
        pos[:4] = torch.tensor([(1 << 31) - 1, -(1 << 31), -1, 0], dtype=torch.int32)
    return rows, gains, pos.to(DEV)


CASES = [  # M, query heads, kv heads, head size, rotated, interleaved, norm of q, norm of k
    (1, 1, 1, 64, 64, False, True, True), (1, 40, 8, 128, 128, False, True, True), (2, 14, 2, 64, 32, True, False, False),
    (3, 5, 5, 128, 16, False, True, False), (7, 28, 4, 128, 64, True, False, True), (33, 3, 1, 64, 48, False, True, True),
    (61, 64, 8, 128, 112, True, True, True), (130, 9, 2, 64, 64, True, True, True), (517, 40, 8, 128, 128, False, True, True),
    (4099, 6, 2, 64, 64, False, True, True), (9001, 14, 2, 64, 64, True, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_forward_and_backward(ops, case):
    M, nh, nkv, hd, rot, il, nq, nk = case
    (q, k, dyq, dyk), (gq, gk), pos = _inputs(M, M, nh, nkv, hd, "far" if M >= 4 else "plain")
    gq, gk = gq if nq else None, gk if nk else None
    freq, factor = ops.rope_frequencies(rot, base=1e6, scaling="yarn", factor=4.0, original=32768)
    rope = ops.rope(rot, base=1e6, interleaved=il, scaling="yarn", scale=4.0, original=32768)
    assert rope.factor == factor
    cos, sin = _tables(pos, freq, factor)
    oq, ok = ops.qk_norm_rope_fwd(q, k, hd, rope, pos, q_gain=gq, k_gain=gk, eps=EPS)
    dq, dk, dgq, dgk = ops.qk_norm_rope_bwd(q, k, dyq, dyk, hd, rope, pos, q_gain=gq, k_gain=gk, eps=EPS)
    assert (dgq is None) == (gq is None) and (dgk is None) == (gk is None)
    for x, dy, gain, o, dx, dg in ((q, dyq, gq, oq, dq, dgq), (k, dyk, gk, ok, dk, dgk)):
        w = None if gain is None else gain.double().requires_grad_()
        xr = x.double().requires_grad_()
        y, size = _forward(xr, w, (cos, sin, rot, il), hd)
        got = o.double().view_as(y)
        assert (got - y).abs().le(2.0 ** -8 * y.abs() + 2.0 ** -19 * size).all()
        y.backward(dy.double().view_as(y))
        d, dsize = _forward(dy.double(), None, (cos, -sin, rot, il), hd)  # rotated back
        ref, got = xr.grad.view_as(y), dx.double().view_as(y)
        if gain is None:
            bound = dsize
        else:
            xh = x.double().view_as(y)
            r = (xh.square().mean(-1, keepdim=True) + EPS).rsqrt()
            u = xh * r
            bound = r * (dsize * w.abs() + u.abs() * (dsize * w.abs() * u.abs()).mean(-1, keepdim=True))
            total = (dsize * u.abs()).sum((0, 1))
            assert (dg.double() - w.grad).abs().le(2.0 ** -16 * total).all()
        assert (got - ref).abs().le(2.0 ** -8 * ref.abs() + 2.0 ** -18 * bound).all()


def test_the_64_bit_gradients_agree_with_differences(ops):
    """The reference's gradients that the kernels are held to, against central differences of the forward formula."""
    (q, _, dy, _), (g, _), pos = _inputs(5, 3, 2, 1, 64)
    cos, sin = _tables(pos, ops.rope_frequencies(32, base=1e4)[0], 1.25)
    rope = (cos, sin, 32, True)
    x, w, d = q.double().requires_grad_(), g.double().requires_grad_(), dy.double()

    def loss(x, w):
        return (_forward(x, w, rope, 64)[0].reshape(3, -1) * d).sum()
    loss(x, w).backward()
    for t, grad in ((x, x.grad), (w, w.grad)):
        flat = t.detach().clone()
        for i in range(0, flat.numel(), 37):
            h = 1e-5
            vals = []
            for s in (h, -h):
                z = flat.clone()
                z.view(-1)[i] += s
                vals.append(loss(z if t is x else x.detach(), z if t is w else w.detach()).item())
            assert abs((vals[0] - vals[1]) / (2 * h) - grad.reshape(-1)[i].item()) < 1e-5


def test_norm_alone_and_rotation_alone(ops):
    (q, k, dyq, dyk), (gq, gk), pos = _inputs(6, 37, 4, 2, 128)
    oq, ok = ops.qk_norm_rope_fwd(q, k, 128, q_gain=gq, k_gain=gk, eps=EPS)
    for x, o, g in ((q, oq, gq), (k, ok, gk)):
        y, size = _forward(x.double(), g.double(), None, 128)
        assert (o.double().view_as(y) - y).abs().le(2.0 ** -8 * y.abs() + 2.0 ** -19 * size).all()
    # position 0 turns nothing: the rotation alone is the identity there, bit for bit
    rope = ops.rope(64, interleaved=True)
    oq, ok = ops.qk_norm_rope_fwd(q, k, 128, rope, torch.zeros_like(pos))
    assert torch.equal(oq, q) and torch.equal(ok, k)
    dq, dk, a, b = ops.qk_norm_rope_bwd(q, k, dyq, dyk, 128, rope, torch.zeros_like(pos))
    assert torch.equal(dq, dyq) and torch.equal(dk, dyk) and a is None and b is None
    # elements behind the rotated ones pass as they are, whatever the rotated ones hold
    q[3, 0] = math.nan
    q[4, 127] = math.inf
    oq, _ = ops.qk_norm_rope_fwd(q, k, 128, rope, pos)
    assert torch.equal(oq.view(37, 4, 128)[:, :, 64:], q.view(37, 4, 128)[:, :, 64:])
    bad = ~oq.view(37, 4, 128)[:, :, :64].isfinite()
    assert bad.nonzero().tolist() == [[3, 0, 0], [3, 0, 1]]


def test_zero_and_non_finite_heads_stay_by_themselves(ops):
    (q, k, dyq, dyk), (gq, gk), pos = _inputs(7, 20, 6, 2, 64)
    rope = ops.rope(64)
    ref = ops.qk_norm_rope_fwd(q, k, 64, rope, pos, q_gain=gq, k_gain=gk, eps=EPS)[0].clone()
    dref = ops.qk_norm_rope_bwd(q, k, dyq, dyk, 64, rope, pos, q_gain=gq, k_gain=gk, eps=EPS, want_gains=False)[0].clone()
    q[2, 64:128] = 0
    q[5, 130] = math.nan
    q[9, 10] = math.inf
    hit = torch.zeros(20, 6, dtype=torch.bool, device=DEV)
    hit[2, 1] = hit[5, 2] = hit[9, 0] = True
    o = ops.qk_norm_rope_fwd(q, k, 64, rope, pos, q_gain=gq, k_gain=gk, eps=EPS)[0].view(20, 6, 64)
    d = ops.qk_norm_rope_bwd(q, k, dyq, dyk, 64, rope, pos, q_gain=gq, k_gain=gk, eps=EPS, want_gains=False)[0].view(20, 6, 64)
    assert torch.equal(o[~hit], ref.view(20, 6, 64)[~hit]) and torch.equal(d[~hit], dref.view(20, 6, 64)[~hit])
    assert (o[2, 1] == 0).all() and d[2, 1].isfinite().all()
    assert o[5, 2].isnan().all() and d[5, 2].isnan().all()
    assert o[9, 0, 10].isnan()


def test_strided_rows_in_place_and_what_lies_between(ops):
    M, nh, nkv, hd = 45, 10, 2, 64
    (q, k, dyq, dyk), (gq, gk), pos = _inputs(8, M, nh, nkv, hd)
    rope = ops.rope(48, interleaved=False)
    want = ops.qk_norm_rope_fwd(q, k, hd, rope, pos, q_gain=gq, k_gain=gk)
    wide = torch.full((M, 1024), 7.0, dtype=torch.bfloat16, device=DEV)  # one projection's rows: gap, q, gap, k
    sq, sk = wide[:, 8:8 + nh * hd], wide[:, 800:800 + nkv * hd]
    sq.copy_(q)
    sk.copy_(k)
    a, b = ops.qk_norm_rope_fwd(sq, sk, hd, rope, pos, q_gain=gq, k_gain=gk, q_out=sq, k_out=sk)
    assert a is sq and torch.equal(sq, want[0]) and torch.equal(sk, want[1])
    rest = torch.ones(1024, dtype=torch.bool, device=DEV)
    rest[8:8 + nh * hd] = rest[800:800 + nkv * hd] = False
    assert (wide[:, rest] == 7).all()
    dw = ops.qk_norm_rope_bwd(q, k, dyq, dyk, hd, rope, pos, q_gain=gq, k_gain=gk)
    sq.copy_(dyq)
    sk.copy_(dyk)
    got = ops.qk_norm_rope_bwd(q, k, sq, sk, hd, rope, pos, q_gain=gq, k_gain=gk, dq=sq, dk=sk)
    assert all(torch.equal(x, y) for x, y in zip(got, dw))
    x = q.clone()
    got = ops.qk_norm_rope_bwd(x, k, dyq, dyk, hd, rope, pos, q_gain=gq, k_gain=gk, dq=x)
    assert all(torch.equal(x, y) for x, y in zip(got, dw))


def test_accumulated_frozen_and_single_gains(ops):
    (q, k, dyq, dyk), (gq, gk), pos = _inputs(9, 301, 8, 2, 128)
    rope = ops.rope(128)
    _, _, a, b = ops.qk_norm_rope_bwd(q, k, dyq, dyk, 128, rope, pos, q_gain=gq, k_gain=gk)
    a2, b2 = torch.ones_like(a), torch.full_like(b, -2.0)
    ops.qk_norm_rope_bwd(q, k, dyq, dyk, 128, rope, pos, q_gain=gq, k_gain=gk, dq_gain=a2, dk_gain=b2, grad_accumulate=True)
    assert torch.equal(a2, 1 + a) and torch.equal(b2, b - 2)
    dq, dk, none, only = ops.qk_norm_rope_bwd(q, k, dyq, dyk, 128, rope, pos, k_gain=gk)
    assert none is None and torch.equal(only, b)
    frozen = ops.qk_norm_rope_bwd(q, k, dyq, dyk, 128, rope, pos, q_gain=gq, k_gain=gk, want_gains=False)
    full = ops.qk_norm_rope_bwd(q, k, dyq, dyk, 128, rope, pos, q_gain=gq, k_gain=gk)
    assert torch.equal(frozen[0], full[0]) and torch.equal(frozen[1], full[1]) and frozen[2] is None
    with pytest.raises(ValueError):
        ops.qk_norm_rope_bwd(q, k, dyq, dyk, 128, rope, pos, q_gain=gq, k_gain=gk, grad_accumulate=True)
    with pytest.raises(ValueError):
        ops.qk_norm_rope_fwd(q, k, 128, rope, pos.long())
    with pytest.raises(ValueError):
        ops.qk_norm_rope_fwd(q, k, 128, rope, pos[:-1])
    with pytest.raises(ValueError):
        ops.qk_norm_rope_fwd(q, k, 128, rope, pos, q_gain=gq.bfloat16())


def test_repeats_streams_and_replays(ops):
    (q, k, dyq, dyk), (gq, gk), pos = _inputs(10, 777, 12, 4, 64)
    rope = ops.rope(64, interleaved=True)
    out = [torch.empty_like(t) for t in (q, k, q, k)]
    dg = [torch.empty(64, device=DEV) for _ in range(2)]
    ws = torch.full((ops.qk_norm_rope_workspace_size(777, 12, 4, 64),), 255, dtype=torch.uint8, device=DEV)

    def call(stream=None):
        ops.qk_norm_rope_fwd(q, k, 64, rope, pos, q_gain=gq, k_gain=gk, q_out=out[0], k_out=out[1], stream=stream)
        ops.qk_norm_rope_bwd(q, k, dyq, dyk, 64, rope, pos, q_gain=gq, k_gain=gk, dq=out[2], dk=out[3], dq_gain=dg[0], dk_gain=dg[1],
                             workspace=ws, stream=stream)

    def take():
        torch.cuda.synchronize()
        return [t.clone() for t in out + dg]
    call()
    first = take()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    assert all(torch.equal(a, b) for a, b in zip(first, take()))
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    pos += 1000
    q.mul_(1.5)
    graph.replay()
    again = take()
    call()
    assert all(torch.equal(a, b) for a, b in zip(again, take()))
    assert not torch.equal(again[0], first[0])
