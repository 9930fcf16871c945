"""Norm and rotary positions of many rows, where a group has all heads of its tokens and, backward with gradients of the
gains, takes several tokens one after another; against plain 64-bit forms, with the bounds of test_gpu_rope.py.

A gradient of a gain sums terms that are each off by 2^-19 of themselves.  The chain of its additions: a thread's tokens
times the heads it has of each, the groups of a CTA one after another (256 threads of head_dim/16 make one), every 32nd CTA,
and 32 of those sums.  On 152 SMs or more there are 2 CTAs each at most, so no fewer than 304 share the tokens: L additions
are L 2^-24 of the sum of sizes."""
import pytest
import torch

from test_gpu_rope import DEV, EPS, _forward, _inputs, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import ops as o
    return o


CASES = [  # M, query heads, kv heads, head size, rotated, interleaved, norm of q, norm of k
    (30011, 3, 1, 128, 128, False, True, True), (30011, 2, 2, 128, 64, True, True, True), (60013, 2, 1, 64, 64, False, True, True),
    (60013, 1, 2, 64, 32, True, True, True), (19457, 3, 2, 64, 64, True, True, False), (9729, 5, 1, 128, 128, False, False, True),
    (12007, 12, 4, 128, 128, True, True, True), (40001, 1, 1, 64, 48, False, True, True)]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_many_rows(ops, case):
    M, nh, nkv, hd, rot, il, nq, nk = case
    (q, k, dyq, dyk), (gq, gk), pos = _inputs(M + nh, M, nh, nkv, hd, "far")
    gq, gk = gq if nq else None, gk if nk else None
    freq, factor = ops.rope_frequencies(rot, base=1e6)
    rope = ops.rope(rot, base=1e6, interleaved=il)
    cos, sin = _tables(pos, freq, factor)
    oq, ok = ops.qk_norm_rope_fwd(q, k, hd, rope, pos, q_gain=gq, k_gain=gk, eps=EPS)
    size = ops.qk_norm_rope_workspace_size(M, nh, nkv, hd)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device=DEV)
    dgq, dgk = (None if g is None else torch.full((hd + 8,), 7.0, device=DEV) for g in (gq, gk))
    given = dict(q_gain=gq, k_gain=gk, eps=EPS, dq_gain=None if dgq is None else dgq[4:-4], dk_gain=None if dgk is None else dgk[4:-4])
    dq, dk, a, b = ops.qk_norm_rope_bwd(q, k, dyq, dyk, hd, rope, pos, workspace=ws[32:32 + size], **given)
    assert (ws[:32] == 255).all() and (ws[32 + size:] == 255).all()
    first = [t.clone() for t in (dq, dk, a, b) if t is not None]
    dq, dk, a, b = ops.qk_norm_rope_bwd(q, k, dyq, dyk, hd, rope, pos, **given)
    assert all(torch.equal(x, y) for x, y in zip(first, [t for t in (dq, dk, a, b) if t is not None]))
    frozen = ops.qk_norm_rope_bwd(q, k, dyq, dyk, hd, rope, pos, q_gain=gq, k_gain=gk, eps=EPS, want_gains=False)
    assert torch.equal(frozen[0], dq) and torch.equal(frozen[1], dk)
    groups = 256 // (hd // 16)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ctas = 2 * sms
    for x, dy, gain, o, dx, dg, pad, heads in ((q, dyq, gq, oq, dq, a, dgq, nh), (k, dyk, gk, ok, dk, b, dgk, nkv)):
        w = None if gain is None else gain.double().requires_grad_()
        xr = x.double().requires_grad_()
        y, size = _forward(xr, w, (cos, sin, rot, il), hd)
        got = o.double().view_as(y)
        assert (got - y).abs().le(2.0 ** -8 * y.abs() + 2.0 ** -19 * size).all()
        y.backward(dy.double().view_as(y))
        d, dsize = _forward(dy.double(), None, (cos, -sin, rot, il), hd)  # rotated back
        ref, got = xr.grad.view_as(y), dx.double().view_as(y)
        bound = dsize
        if gain is not None:
            xh = x.double().view_as(y)
            r = (xh.square().mean(-1, keepdim=True) + EPS).rsqrt()
            u = xh * r
            bound = r * (dsize * w.abs() + u.abs() * (dsize * w.abs() * u.abs()).mean(-1, keepdim=True))
            chain = -(-M // (ctas * groups)) * heads + groups + -(-ctas // 32) + 32
            total = (dsize * u.abs()).sum((0, 1))
            assert (dg.double() - w.grad).abs().le((2.0 ** -19 + chain * 2.0 ** -24) * total).all()
            assert (pad[:4] == 7).all() and (pad[-4:] == 7).all()
            # and far closer than the terms' own size: no token is left out or counted twice
            assert (dg.double() - w.grad).norm() <= 1e-5 * w.grad.norm()
        assert (got - ref).abs().le(2.0 ** -8 * ref.abs() + 2.0 ** -18 * bound).all()


def test_gradients_of_gains_added_over_many_rows(ops):
    """What dq_gain and dk_gain hold is added to once, whatever the number of tokens a group takes."""
    M, hd = 30011, 128
    (q, k, dyq, dyk), (gq, gk), pos = _inputs(3, M, 1, 1, hd)
    rope = ops.rope(hd)
    _, _, a, b = ops.qk_norm_rope_bwd(q, k, dyq, dyk, hd, rope, pos, q_gain=gq, k_gain=gk)
    a2, b2 = torch.full_like(a, 3.0), torch.full_like(b, -1.0)
    ops.qk_norm_rope_bwd(q, k, dyq, dyk, hd, rope, pos, q_gain=gq, k_gain=gk, dq_gain=a2, dk_gain=b2, grad_accumulate=True)
    assert torch.equal(a2, 3.0 + a) and torch.equal(b2, b - 1.0)
