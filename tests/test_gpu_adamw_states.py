"""The states of ws_adamw_step: 8-bit codes over the whole range of fp32; the memory a plan keeps."""
import gc

import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_streaming_nf4_gb300 import ops as o
    return o


def root_values():
    """The 256 values of the root's code, in 64 bits."""
    c = np.arange(256)
    v = (1 + (c % 16) / 16) * 2.0 ** (c // 16 - 15)
    v[0] = 0
    return v


def test_codes_of_subnormal_blocks(ops):
    """Block maxima from the smallest fp32 number up: the scale is then a few units of 2^-149, rounded to one of them, and
    the largest quotient reaches 2.  A value's code is never 0 and never its neighbour's business.

    With the stored scale s (subnormal: any value), a code is the nearest of q = x / s <= 2: off by half a step, 2^-5 q,
    where q > 1.9375 too (2 - 1.9375 = 2^-5 2); a value below the smallest code gets that, (1 + 1/16) 2^-15 s; decoding
    rounds the product to a multiple of 2^-149, at most 2^-150 off."""
    tops = np.unique(np.concatenate([np.arange(1, 2050), 2 ** np.arange(1, 40), 3 * 2 ** np.arange(1, 40)]))
    bits = np.zeros((len(tops), 256), np.float64)
    for i, t in enumerate(tops):
        bits[i, 1::2] = np.maximum(1, np.floor(t * np.linspace(0.01, 1, 128)))   # (even places: zeros beside them)
    x = torch.from_numpy((bits * 2.0 ** -149).astype(np.float32))
    codes, scales = ops.adamw_encode8(x.view(-1).to(dev()), True)
    c, s = codes.cpu().numpy().reshape(bits.shape), scales.cpu().numpy().astype(np.float64)[:, None]
    assert ((c == 0) == (bits == 0)).all(), tops[((c == 0) != (bits == 0)).any(1)]
    want = bits * 2.0 ** -149
    got = ops.adamw_decode8(codes, scales, True).cpu().numpy().astype(np.float64).reshape(bits.shape)
    assert (np.abs(got - want) <= 2.0 ** -5 * want + (17 / 16) * 2.0 ** -15 * s + 2.0 ** -150).all()
    # first moments in such blocks: the nearest e4m3 number of x / s, the largest (448) beyond it
    codes, scales = ops.adamw_encode8((x * torch.where(torch.arange(256) % 4 == 1, -1.0, 1.0)).view(-1).to(dev()), False)
    s = scales.cpu().numpy().astype(np.float64)[:, None]
    q = np.divide(want, s, out=np.zeros_like(want), where=s > 0)
    c = codes.float().cpu().numpy().astype(np.float64).reshape(bits.shape)
    near = torch.from_numpy(np.minimum(q, 448.0)).float().to(torch.float8_e4m3fn).double().numpy()
    assert (np.abs(c) == near).all() and (np.signbit(c)[:, 1::4] | (c[:, 1::4] == 0)).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_plan_keeps_its_tensors(ops, bits):
    """A caller may clear or refill its lists, or give a tensor other storage: the plan's step still finds the memory
    that the plan was made for."""
    n = 1000
    z = lambda dt=F, k=n: [torch.zeros(k, dtype=dt, device=dev()) for _ in range(2)]
    p, g = z(), z()
    if bits == 32:
        m, v, kw = z(), z(), {}
    else:
        m, v = z(torch.uint8), z(torch.uint8)
        kw = dict(exp_avg_scales=z(k=4), exp_avg_sq_scales=z(k=4))
    lists = [p, g, m, v, *kw.values()]
    plan = ops.adamw_plan(p, g, m, v, **kw)
    where = [[t.data_ptr() for t in x] for x in lists]
    p[1].data = torch.ones(n, device=dev())     # other storage for the same tensor
    for x in lists:
        x.clear()
    gc.collect()
    assert [[t.data_ptr() for t in x] for x in plan.tensors if x is not None] == where
    # nobody else is given that memory while the plan lives
    taken = {q for x in where for q in x}
    fresh = [torch.empty(k, dtype=dt, device=dev()) for k, dt in ((n, F), (n, torch.uint8), (4, F)) for _ in range(64)]
    assert not taken & {t.data_ptr() for t in fresh}


def root_values():
    """The 256 values of the root's code."""
    c = np.arange(256)
    v = (1 + (c % 16) / 16) * 2.0 ** (c // 16 - 15.0)
    v[0] = 0
    return v.astype(np.float32)


class Definition:
    """8-bit states and a step without clipping, operation by operation in IEEE fp32."""

    def __init__(self, n, beta1, beta2):
        self.n, nb = n, -(-n // 256)
        self.m, self.v = np.zeros((nb, 256), np.float32), np.zeros((nb, 256), np.uint8)   # (m: the codes' values)
        self.ms, self.vs = np.zeros((nb, 1), np.float32), np.zeros((nb, 1), np.float32)
        f = np.float32
        self.c = f(beta1), f(1 - beta1), f(beta2), f(1 - beta2)

    def step(self, g):
        b1, nb1, b2, nb2 = self.c
        x = np.zeros(self.m.size, np.float32)
        x[:self.n] = g
        x = x.reshape(self.m.shape)
        r = root_values()[self.v] * self.vs
        m = (self.m * self.ms) * b1 + x * nb1
        root = np.sqrt((r * r) * b2 + (x * x) * nb2)
        self.ms = np.abs(m).max(1, keepdims=True) * np.float32(1 / 448)
        self.vs = root.max(1, keepdims=True) * np.float32(1 / 1.9375)
        q = np.divide(m, self.ms, out=np.zeros_like(m), where=self.ms > 0)
        self.m = torch.from_numpy(np.clip(q, -448, 448)).to(torch.float8_e4m3fn).float().numpy()
        q = np.divide(root, self.vs, out=np.zeros_like(root), where=self.vs > 0)
        f, e = np.frexp(np.clip(q, np.float32(17 / 16 * 2.0 ** -15), np.float32(1.9375)))
        code = (e + 14) * 16 + np.rint(f * 32).astype(np.int64) - 16      # f * 32 in [16, 32]; ties to even
        self.v = np.where(q > 0, code, 0).astype(np.uint8)
        assert m.dtype == root.dtype == self.m.dtype == self.vs.dtype == np.float32


@pytest.mark.parametrize("g_dtype", [F, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.999), (0.85, 0.95), (0.0, 0.5)])
def test_eight_bit_states_are_the_definition_s_bit_for_bit(ops, g_dtype, beta1, beta2):
    """Many steps from zero states, none of them brought back to the other's: every code and every scale is the one that
    the formula gives when each of its operations is rounded once to fp32."""
    rng = np.random.default_rng(5)
    sizes = [1, 255, 256, 300, 4096, 40001]
    spread = [np.exp(rng.normal(0, 2.0, n)).astype(np.float32) * 10.0 ** rng.uniform(-12, 3) for n in sizes]
    spread[3][:] = 0
    spread[4][::3] = 0
    p = [torch.zeros(n, device=dev()) for n in sizes]
    g = [torch.zeros(n, dtype=g_dtype, device=dev()) for n in sizes]
    m, v = ([torch.zeros(n, dtype=torch.uint8, device=dev()) for n in sizes] for _ in range(2))
    ms, vs = ([torch.zeros(-(-n // 256), device=dev()) for n in sizes] for _ in range(2))
    plan = ops.adamw_plan(p, g, m, v, exp_avg_scales=ms, exp_avg_sq_scales=vs)
    groups = ops.adamw_groups([dict(lr=1e-3, beta1=beta1, beta2=beta2)])
    want = [Definition(n, beta1, beta2) for n in sizes]
    for step in range(80):
        for i, n in enumerate(sizes):
            x = torch.from_numpy((rng.standard_normal(n) * spread[i] * (0.1 if step > 40 else 1.0)).astype(np.float32)).to(g_dtype)
            g[i].copy_(x)
            want[i].step(x.float().numpy())
        ops.adamw_step(plan, groups)
        for i, (n, w) in enumerate(zip(sizes, want)):
            assert np.array_equal(ms[i].cpu().numpy(), w.ms[:, 0]) and np.array_equal(vs[i].cpu().numpy(), w.vs[:, 0]), (step, n)
            assert np.array_equal(v[i].cpu().numpy(), w.v.reshape(-1)[:n]), (step, n)
            assert np.array_equal(m[i].view(torch.float8_e4m3fn).float().cpu().numpy(), w.m.reshape(-1)[:n]), (step, n)
            assert torch.isfinite(p[i]).all()


@pytest.mark.parametrize("g_dtype", [F, BF], ids=["f32", "bf16"])
def test_norms_are_the_correctly_rounded_ones(ops, g_dtype):
    """Sums of squares in two fp32 parts hold some 44 bits: the norm is off by its own rounding to fp32, half a step (2^-24),
    and less than a thousandth of that.  A plain fp32 sum, whose error is of the size of a step, fails this somewhere."""
    r = torch.Generator().manual_seed(1)
    sizes = [int(2 ** x) + 1 for x in torch.linspace(0, 20, 60).tolist()]
    g = [(torch.rand(n, generator=r) * 10.0 ** (i % 7 - 3)).to(g_dtype).to(dev()) for i, n in enumerate(sizes)]
    z = lambda: [torch.zeros(n, device=dev()) for n in sizes]
    plan = ops.adamw_plan(z(), g, z(), z(), groups=list(range(60)))
    norms = torch.zeros(60, device=dev())
    ops.adamw_step(plan, ops.adamw_groups([dict(lr=0.0)] * 60), norms=norms)
    want = torch.stack([x.double().square().sum().sqrt() for x in g])
    assert ((norms.double() - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -10) * want).all()
    plain = torch.stack([x.float().square().cumsum(0)[-1].sqrt() for x in g]).double()
    assert not ((plain - want).abs() <= 2.0 ** -24 * (1 + 2.0 ** -10) * want).all()


@pytest.mark.parametrize("clip", [False, True])
def test_moments_in_32_bits(ops, clip):
    """m: the clip factor, its product with g, a coefficient, its product and the sum, rounded once each: 5 2^-24 of the
    absolute terms.  v: twice the first two, the square, a coefficient, its product and the sum: 8 2^-24 (9 with what the
    bound leaves out, products of two errors)."""
    r = torch.Generator().manual_seed(2)
    n = 100003
    g, m, v = (torch.randn(n, generator=r).to(dev()) for _ in range(3))
    m, v = m * 0.1, v.square() * 0.01
    p = torch.zeros(n, device=dev())
    plan = ops.adamw_plan([p], [g], [m], [v])
    b1, b2 = 0.9, 0.999
    norm = float(g.double().norm())
    m0, v0, c = m.double(), v.double(), 0.37 * norm / (norm + 1e-6) if clip else 1.0
    ops.adamw_step(plan, ops.adamw_groups([dict(lr=1e-3, beta1=b1, beta2=b2, max_norm=0.37 * norm)]), clip=clip)
    x = g.double() * c
    assert ((m.double() - (b1 * m0 + (1 - b1) * x)).abs() <= 6 * 2.0 ** -24 * (b1 * m0.abs() + (1 - b1) * x.abs())).all()
    assert ((v.double() - (b2 * v0 + (1 - b2) * x * x)).abs() <= 9 * 2.0 ** -24 * (b2 * v0 + (1 - b2) * x * x)).all()


def test_a_tensor_of_more_than_2_31_elements(ops):
    """One step from zero 8-bit states and its decoding, checked at both ends and around element 2^31."""
    n, lr = 2 ** 31 + 777, 2.0 ** -7
    g = torch.empty(n, dtype=BF, device=dev()).normal_(generator=torch.Generator(device=dev()).manual_seed(3))
    p = torch.ones(n, dtype=BF, device=dev())
    m, v = (torch.zeros(n, dtype=torch.uint8, device=dev()) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), device=dev()) for _ in range(2))
    plan = ops.adamw_plan([p], [g], [m], [v], exp_avg_scales=[ms], exp_avg_sq_scales=[vs])
    norms = torch.zeros(1, device=dev())
    ops.adamw_step(plan, ops.adamw_groups([dict(lr=lr, weight_decay=0.0)]), norms=norms)
    dm = ops.adamw_decode8(m.view(torch.float8_e4m3fn), ms, False, dtype=BF)
    dr = ops.adamw_decode8(v, vs, True, dtype=BF)
    sq = sum(float(g[i:i + 2 ** 28].float().double().square().sum()) for i in range(0, n, 2 ** 28))
    assert abs(float(norms[0]) - sq ** 0.5) <= 2.0 ** -23 * sq ** 0.5
    for a in (0, 2 ** 31 - 2048, n - n % 256 - 2048):
        b = min(n, a + 4096)
        x = g[a:b].float().cpu().numpy()
        d = Definition(b - a, 0.9, 0.999)
        d.step(x)
        assert np.array_equal(ms[a // 256:-(-b // 256)].cpu().numpy(), d.ms[:, 0])
        assert np.array_equal(v[a:b].cpu().numpy(), d.v.reshape(-1)[:b - a])
        for got, want in ((dm, d.m * d.ms), (dr, root_values()[d.v] * d.vs)):
            assert torch.equal(got[a:b].cpu(), torch.from_numpy(want.reshape(-1)[:b - a]).to(BF))
        # from zero states the step is lr g / (|g| + eps), rounded to bf16 once (half a step: 2^-8 of the value)
        w = 1 - lr * x.astype(np.float64) / (np.abs(x) + 1e-8)
        assert (np.abs(p[a:b].double().cpu().numpy() - w) <= 2.0 ** -8 * np.abs(w)).all()
    # encoded from values: half a step of the code (2^-5 of the value), the smallest code, and the scale's rounding
    big = torch.zeros(n, device=dev())
    big[n - 3000:] = torch.rand(3000, generator=torch.Generator().manual_seed(4)).to(dev())
    codes, scales = ops.adamw_encode8(big, True)
    back = ops.adamw_decode8(codes, scales, True)
    assert ((back[n - 4000:] - big[n - 4000:]).abs() <= (2.0 ** -5 + 2.0 ** -20) * big[n - 4000:] + 2.0 ** -14).all()
    assert not back[:n - 4000].any()
