"""ws_adamw_step against the AdamW formula in 64 bits, one step at a time from
the very state the step found (so no error is carried along).

Tolerances: fp32 m and v have at most four roundings (2^-24 each of the sum of
the absolute terms) and coefficients rounded once: 2^-21 of it.  p: a change
whose factors are off by 2^-20 at most (roots, quotients, clip), plus half a
step of p and of its decay.  8-bit states: half a step of the code (e4m3 2^-4
of the value, the root's code 2^-5), or of the smallest step, beside a scale
off by 2^-22; a norm sums at most 16 + 13 terms in fp32: 2^-18.
"""
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
SIZES = [1, 3, 8, 255, 256, 257, 4095, 4096, 4097, 10007, 70000]


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_streaming_nf4_gb300 import ops as o
    return o


def guarded(x):
    """The tensor inside a larger buffer, 16-byte aligned, with marks behind it."""
    n, room = x.numel(), 64
    buf = torch.zeros(n + room, dtype=x.dtype, device=dev())
    buf.view(torch.uint8).fill_(0x5A)
    buf[:n] = x.to(dev())
    return buf[:n], buf


def root_table():
    c = torch.arange(256, dtype=torch.float64)
    v = (1 + (c % 16) / 16) * 2.0 ** (torch.floor(c / 16) - 15)
    v[0] = 0
    return v.to(dev())


class Run:
    def __init__(self, ops, p_dtype, g_dtype, bits, groups=3, seed=0, sizes=SIZES, warm=True):
        r = torch.Generator().manual_seed(seed)
        self.ops, self.bits, self.p_dtype = ops, bits, p_dtype
        self.group = [(i * 2) % groups for i in range(len(sizes))]
        mk = lambda n, s, dt=F: guarded((torch.randn(n, generator=r) * s).to(dt))
        self.p, pb = zip(*[mk(n, 0.1, p_dtype) for n in sizes])
        self.g, gb = zip(*[mk(n, 10.0 ** -(i % 5), g_dtype) for i, n in enumerate(sizes)])
        m = [torch.randn(n, generator=r) * 1e-2 * warm for n in sizes]
        v = [(torch.randn(n, generator=r) * 1e-2) ** 2 * warm for n in sizes]
        self.guards = [*pb, *gb]
        if bits == 32:
            self.m, mb = zip(*[guarded(x) for x in m])
            self.v, vb = zip(*[guarded(x) for x in v])
            self.ms = self.vs = None
            self.guards += [*mb, *vb]
        else:
            em = [ops.adamw_encode8(x.to(dev()), False) for x in m]
            ev = [ops.adamw_encode8(x.sqrt().to(dev()), True) for x in v]
            self.m, mb = zip(*[guarded(a.view(torch.uint8)) for a, _ in em])
            self.v, vb = zip(*[guarded(a) for a, _ in ev])
            self.ms, msb = zip(*[guarded(b) for _, b in em])
            self.vs, vsb = zip(*[guarded(b) for _, b in ev])
            self.guards += [*mb, *vb, *msb, *vsb]
        self.sizes = sizes
        self.hyper = [dict(lr=1e-3 * (i + 1), beta1=0.9 - 0.1 * i, beta2=0.999 - 0.01 * i, eps=1e-8,
                           weight_decay=0.1 * i, max_norm=[0.5, 1e9, 0.0][i % 3], step=[0, 7, 999][i % 3])
                      for i in range(groups)]
        self.groups = ops.adamw_groups(self.hyper)
        kw = {} if bits == 32 else dict(exp_avg_scales=self.ms, exp_avg_sq_scales=self.vs)
        self.plan = ops.adamw_plan(self.p, self.g, self.m, self.v, groups=self.group, n_groups=groups, **kw)
        self.ends = [b[-64:].view(torch.uint8).clone() for b in self.guards]

    def values(self):
        """(m, root of v) of every tensor in 64 bits."""
        if self.bits == 32:
            return [(m.double(), v.double().sqrt()) for m, v in zip(self.m, self.v)]
        t = root_table()
        blow = lambda s, n: s.double().repeat_interleave(256)[:n]
        return [(m.view(torch.float8_e4m3fn).double() * blow(ms, n), t[v.long()] * blow(vs, n))
                for m, v, ms, vs, n in zip(self.m, self.v, self.ms, self.vs, self.sizes)]

    def state(self):
        return [t.clone() for x in (self.p, self.m, self.v, self.ms or (), self.vs or ()) for t in x] + [self.groups.clone()]

    def step_and_check(self, clip):
        before = [(p.double(), g.double(), *s) for p, g, s in zip(self.p, self.g, self.values())]
        norms = torch.zeros(len(self.hyper), device=dev())
        self.ops.adamw_step(self.plan, self.groups, norms=norms, clip=clip)
        now = self.values()
        for h, hy in enumerate(self.hyper):
            of = [i for i, q in enumerate(self.group) if q == h]
            norm = float(torch.cat([before[i][1] for i in of]).norm()) if of else 0.0
            assert abs(float(norms[h]) - norm) <= 2.0 ** -18 * norm
            c = min(1.0, hy["max_norm"] / (norm + 1e-6)) if clip and hy["max_norm"] > 0 else 1.0
            hy["step"] += 1
            t, b1, b2 = hy["step"], hy["beta1"], hy["beta2"]
            assert float(self.groups[h, 6]) == t
            for i in of:
                p0, g, m0, r0 = before[i]
                g = g * c
                m, v = b1 * m0 + (1 - b1) * g, b2 * r0 ** 2 + (1 - b2) * g ** 2
                den = (v / (1 - b2 ** t)).sqrt() + hy["eps"]
                upd = hy["lr"] / (1 - b1 ** t) * m / den
                p = p0 * (1 - hy["lr"] * hy["weight_decay"]) - upd
                # the terms of m may cancel: their errors count against the terms
                mabs = b1 * m0.abs() + (1 - b1) * g.abs()
                uabs = hy["lr"] / (1 - b1 ** t) * mabs / den
                half = 2.0 ** -8 if self.p_dtype == BF else 2.0 ** -24
                self.near(self.p[i], p, half * p.abs() + 2.0 ** -17 * uabs + 2.0 ** -23 * p0.abs() + 1e-30, "p", i)
                gm, gr = now[i]
                if self.bits == 32:
                    self.near(gm, m, 2.0 ** -17 * mabs + 1e-37, "m", i)
                    self.near(gr ** 2, v, 2.0 ** -17 * v + 1e-37, "v", i)
                else:
                    n = self.sizes[i]
                    for got, want, abs_, top, rel, least, sc in (
                            (gm, m, mabs, 448.0, 2.0 ** -4, 2.0 ** -10, self.ms[i]),
                            (gr, v.sqrt(), v.sqrt(), 1.9375, 2.0 ** -5, (1 + 1 / 16) * 2.0 ** -15, self.vs[i])):
                        pad = torch.zeros(-(-n // 256) * 256, dtype=torch.float64, device=dev())
                        pad[:n] = want.abs()
                        big = pad.view(-1, 256).amax(1)
                        big_abs = torch.zeros_like(pad)
                        big_abs[:n] = abs_
                        slack = 2.0 ** -17 * big_abs.view(-1, 256).amax(1)
                        self.near(sc, big / top, (slack + 2.0 ** -22 * big) / top + 1e-37, "scale", i)
                        s = sc.double().repeat_interleave(256)[:n]
                        self.near(got, want, rel * want.abs() + least * s + slack.repeat_interleave(256)[:n] + 1e-37, "8 bits", i)
                        if top < 2:
                            assert ((got > 0) | (want == 0)).all()   # a denominator never vanishes
        for b, e in zip(self.guards, self.ends):
            assert torch.equal(b[-64:].view(torch.uint8), e)         # what lies behind a tensor stays

    @staticmethod
    def near(got, want, tol, what, i):
        bad = (got.double() - want).abs() > tol
        assert not bad.any(), (what, i, int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


@pytest.mark.parametrize("clip", [False, True], ids=["plain", "clip"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype,g_dtype", [(F, F), (F, BF), (BF, F), (BF, BF)], ids=["ff", "fb", "bf", "bb"])
def test_step(ops, p_dtype, g_dtype, bits, clip):
    r = Run(ops, p_dtype, g_dtype, bits)
    for _ in range(3):
        r.step_and_check(clip)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero_states(ops, bits):
    r = Run(ops, F, F, bits, warm=False, groups=1, sizes=[256, 5, 1000])
    r.g[0].zero_()   # no gradient, no state: only the weight decay moves it
    r.step_and_check(True)
    assert all((x == 0).all() for x in r.values()[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_group_without_a_finite_norm_takes_no_step(ops, bits):
    for bad in (float("inf"), float("nan"), 3e38):   # 3e38 squared overflows fp32: not a norm either
        r = Run(ops, F, F, bits)
        i = r.group.index(1)
        r.g[i][0] = bad
        s0 = r.state()
        norms = torch.zeros(3, device=dev())
        ops.adamw_step(r.plan, r.groups, norms=norms, clip=True)
        s1 = r.state()
        n = len(r.sizes)
        for k in range(len(s0) - 1):
            same = torch.equal(s0[k].view(torch.uint8), s1[k].view(torch.uint8))
            if r.group[k % n] == 1:
                assert same, k
            elif k < n:
                assert not same, k   # every parameter of the other groups moves
        assert (s1[-1][:, 6] - s0[-1][:, 6]).tolist() == [1.0, 0.0, 1.0]
        assert not torch.isfinite(norms[1]) and torch.isfinite(norms[[0, 2]]).all()


def test_without_clipping_a_bad_gradient_stays_in_its_block(ops):
    r = Run(ops, F, F, 8, groups=1, sizes=[1000, 600])
    r.g[0][300] = float("nan")
    ops.adamw_step(r.plan, r.groups)
    m, v = r.values()[0]
    for x in (m, v):
        assert torch.isnan(x[256:512]).all() and torch.isfinite(x[:256]).all() and torch.isfinite(x[512:]).all()
    assert torch.isfinite(r.p[0]).sum() == 999 and torch.isfinite(r.p[1]).all()


def test_a_group_without_tensors_and_a_shared_gradient(ops):
    g = torch.randn(500, device=dev())
    z = lambda: [torch.zeros(500, device=dev()) for _ in range(2)]
    p = z()
    plan = ops.adamw_plan(p, [g, g], z(), z(), groups=[0, 2], n_groups=3)
    groups = ops.adamw_groups([dict(lr=1e-3), dict(lr=1e-3), dict(lr=1e-3)])
    norms = torch.full((3,), -1.0, device=dev())
    ops.adamw_step(plan, groups, norms=norms, clip=True)
    assert torch.equal(p[0], p[1]) and (p[0] != 0).all()
    assert float(norms[1]) == 0.0 and float(norms[0]) == float(norms[2]) > 0


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_is_the_eager_one(ops, bits):
    a, b = Run(ops, F, F, bits, seed=4), Run(ops, F, F, bits, seed=4)
    st = torch.cuda.Stream()
    norms = torch.zeros(3, device=dev())
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        ops.adamw_step(a.plan, a.groups, norms=norms, clip=True, stream=st)
    for k in range(3):
        for r in (a, b):
            r.groups[:, 0] *= 0.5     # a schedule: the groups may be rewritten between replays
            for g in r.g:
                g.mul_(-0.7)
        torch.cuda.synchronize()
        graph.replay()
        ops.adamw_step(b.plan, b.groups, clip=True)
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_codes(ops):
    """All codes decode to the documented values, and encode back to themselves."""
    codes = torch.arange(256, dtype=torch.uint8, device=dev())
    one = torch.ones(1, device=dev())
    assert torch.equal(ops.adamw_decode8(codes, one, True).double(), root_table())
    got = ops.adamw_decode8(codes.view(torch.float8_e4m3fn), one, False)
    assert torch.equal(got.nan_to_num(7.0), codes.view(torch.float8_e4m3fn).float().nan_to_num(7.0))
    c, s = ops.adamw_encode8(root_table().float(), True)
    assert float(s) == 1.0 and torch.equal(c, codes)
    v = got.nan_to_num(448.0)
    c, s = ops.adamw_encode8(v, False)
    assert float(s) == 1.0 and torch.equal(c.float(), v)
    # ties go to even, small roots to code 1, everything to zero in a zero block
    x = torch.tensor([1.9375, 1 + 1 / 32, 1 + 3 / 32, 1e-7, 0.0], device=dev())
    c, _ = ops.adamw_encode8(x, True)
    assert c.tolist() == [255, 240, 242, 1, 0]
    c, s = ops.adamw_encode8(torch.zeros(300, device=dev()), True)
    assert (c == 0).all() and (s == 0).all()


@pytest.mark.parametrize("root", [False, True])
@pytest.mark.parametrize("n", [1, 7, 256, 300, 5000])
def test_encode_decode(ops, n, root):
    x = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dev()) * torch.logspace(-3, 2, n, device=dev())
    x = x.abs() if root else x
    c, s = ops.adamw_encode8(x, root)
    y = ops.adamw_decode8(c, s, root).double()
    sc = s.double().repeat_interleave(256)[:n]
    rel, least = (2.0 ** -5, 2.0 ** -14) if root else (2.0 ** -4, 2.0 ** -10)
    assert ((y - x.double()).abs() <= (rel + 2.0 ** -22) * x.double().abs() + least * sc).all()
    b = ops.adamw_decode8(c, s, root, dtype=BF)
    assert torch.equal(b, y.float().bfloat16())


def test_refusals(ops):
    z = lambda n=64, dt=F: torch.zeros(n, dtype=dt, device=dev())
    ok = dict(params=[z()], grads=[z()], exp_avg=[z()], exp_avg_sq=[z()])
    plan = ops.adamw_plan(**ok)
    for bad in (dict(params=[z(65)]), dict(params=[z(dt=torch.float16)]), dict(exp_avg=[z(dt=BF)]), dict(grads=[z(), z()]),
                dict(params=[torch.zeros(8, 16, device=dev())[:, ::2]]), dict(exp_avg_scales=[z(1)]),
                dict(exp_avg_scales=[z(1)], exp_avg_sq_scales=[z(1)])):
        with pytest.raises(ValueError):
            ops.adamw_plan(**{**ok, **bad})
    with pytest.raises(ops.WsError):
        ops.adamw_plan([z()], [z()], [z(65)[1:]], [z()])     # misaligned
    p = z()
    with pytest.raises(ops.WsError):
        ops.adamw_plan([p, p], [z(), z()], [z(), z()], [z(), z()])   # one parameter twice
    g = ops.adamw_groups([dict(lr=1e-3)])
    with pytest.raises(ValueError):
        ops.adamw_step(plan, torch.cat([g, g]))
    with pytest.raises(ValueError):
        ops.adamw_step(plan, g, norms=torch.zeros(2, device=dev()))
    with pytest.raises(ops.WsError):
        ops.adamw_step(plan, g, workspace=torch.zeros(16, dtype=torch.uint8, device=dev()))
