"""The linear with the adapters of many requests (ws_lora_linear_fwd_multi /
_bwd_multi) against its formulas in 64 bits.

Tolerances, elementwise, with S(.) the same sums over absolute values:
- products of bf16 values are exact in fp32; a tensor-core sum over K terms is
  rounded at most once per 16 terms and once per warp, CTA or split that joins,
  each by 2^-23 of a partial sum (truncation included), so by at most
  acc(K) = (K / 16 + 80) 2^-23 of S;
- an fp32 factor enters the skinny and gradient products as two bf16 parts: off
  by at most 2^-16 of the term (2^-8 twice);
- the adapter term of y and dX: 16 fp32 products and sums, or bf16 parts of both
  factors: at most 2^-14 of S;
- a bf16 result adds half a step, 2^-8 of its value.
"""
import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu
LEVELS = [-1.0, -0.6962, -0.5251, -0.3949, -0.2844, -0.1848, -0.0911, 0.0,
          0.0796, 0.1609, 0.2461, 0.3379, 0.4407, 0.5626, 0.7230, 1.0]


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_streaming_nf4_gb300 import ops as o
    return o


def rows_of(kind, M, n, g):
    if kind == "one":
        return torch.full((M,), n - 1, dtype=torch.int32)
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if kind == "distinct":
        return (torch.arange(M, dtype=torch.int32) * 7) % n
    if kind == "runs":      # sorted requests
        return (torch.arange(M) * n // M).to(torch.int32)
    r = torch.randint(-1, n, (M,), generator=g, dtype=torch.int32)
    if kind == "wild":      # ids outside the set mean "no adapter"
        r[::3] = torch.tensor([n, 2 ** 31 - 1, -2 ** 31, -5, n + 1], dtype=torch.int32).repeat(M)[:len(r[::3])]
    return r


class Case:
    def __init__(self, ops, M, N, K, n, kind="random", dtype=torch.float32, mask=False, seed=0, pool=0, alloc=dev):
        g = torch.Generator().manual_seed(seed)
        d = alloc()
        self.M, self.N, self.K, self.n = M, N, K, n
        self.rows = rows_of(kind, M, n, g)
        self.codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).to(d)
        self.absmax = (0.02 * (2 + torch.rand(K // 64, N, generator=g))).to(d)
        self.x = torch.randn(M, K, generator=g).bfloat16().to(d)
        self.dY = torch.randn(M, N, generator=g).bfloat16().to(d)
        # adapters as slices of a pool: a stride with room (multiples of 8 elements) between them
        A = torch.full((n, 16 * K + pool), 9e9).to(d)
        B = torch.full((n, 16 * N + pool), 9e9).to(d)
        self.A, self.B = A[:, :16 * K].view(n, 16, K), B[:, :16 * N].view(n, N, 16)
        self.A.copy_((torch.rand(n, 16, K, generator=g) * 2 - 1) / K ** 0.5)
        self.B.copy_(torch.randn(n, N, 16, generator=g) * 0.05)
        if dtype == torch.bfloat16:
            self.A, self.B = self.A.bfloat16(), self.B.bfloat16()
        self.scale = (0.5 + torch.rand(n, generator=g)).to(d)
        self.mask = None
        if mask:
            self.mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (M, K // 32), generator=g, dtype=torch.int32).to(d)
        self.W = ops.NF4Weight(self.codes, self.absmax, N, K)
        self.set = ops.LoraSet(self.A, self.B, self.scale)
        self.plan = ops.lora_multi_plan(self.rows.to(d), n)

    # ---- 64-bit formulas
    def weight(self):
        q = torch.stack([self.codes >> 4, self.codes & 15], -1).view(self.N, self.K).long()
        w = torch.tensor(LEVELS, device=q.device)[q].view(self.N, -1, 64) * self.absmax.t()[:, :, None]
        return w.bfloat16().double().view(self.N, self.K)

    def keep(self):
        if self.mask is None:
            return torch.ones(self.M, self.K, dtype=torch.float64, device=self.x.device)
        b = (self.mask.long()[:, :, None] >> torch.arange(32, device=self.x.device)) & 1
        return b.view(self.M, self.K).double()

    def own(self):
        """(adapter of each row clamped to the set, 1 where the row has one)."""
        r = self.rows.to(self.x.device).long()
        has = (r >= 0) & (r < self.n)
        return torch.where(has, r, torch.zeros_like(r)), has.double()[:, None]

    def forward(self):
        a, has = self.own()
        xm, A, B = self.x.double() * self.keep(), self.A.double(), self.B.double()
        s = self.scale.double()[a][:, None]
        U = torch.bmm(A[a], xm[:, :, None])[:, :, 0] * has
        SU = torch.bmm(A[a].abs(), xm.abs()[:, :, None])[:, :, 0] * has
        w = self.weight()
        lora = torch.bmm(B[a], U[:, :, None])[:, :, 0] * s
        Slora = torch.bmm(B[a].abs(), SU[:, :, None])[:, :, 0] * s
        y = self.x.double() @ w.t() + lora
        return dict(U=U, SU=SU, y=y, Sy=self.x.double().abs() @ w.abs().t(), Slora=Slora)

    def backward(self, U):
        a, has = self.own()
        dY, keep, A, B = self.dY.double(), self.keep(), self.A.double(), self.B.double()
        xm, s = self.x.double() * keep, self.scale.double()[a][:, None]
        G = torch.bmm(dY[:, None, :], B[a])[:, 0] * has
        SG = torch.bmm(dY.abs()[:, None, :], B[a].abs())[:, 0] * has
        w = self.weight()
        dX = dY @ w + torch.bmm(G[:, None, :], A[a])[:, 0] * s * keep
        Slora = torch.bmm(SG[:, None, :], A[a].abs())[:, 0] * s * keep
        hot = torch.nn.functional.one_hot(a, self.n).double() * has
        dA = torch.einsum("mn,mj,mk->njk", hot * s, G, xm)
        SdA = torch.einsum("mn,mj,mk->njk", hot * s, SG, xm.abs())
        dB = torch.einsum("mn,mc,mj->ncj", hot * s, dY, U.double())
        SdB = torch.einsum("mn,mc,mj->ncj", hot * s, dY.abs(), U.double().abs())
        return dict(dX=dX, SdX=dY.abs() @ w.abs(), Slora=Slora, dA=dA, SdA=SdA, dB=dB, SdB=SdB)


def acc(k):
    return (k / 16 + 80) * 2.0 ** -23


def close(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    bad = (got - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / tol.clamp(min=1e-300)).max()))


def check_forward(c, y, U):
    r = c.forward()
    split = 0 if c.A.dtype == torch.bfloat16 else 2.0 ** -16
    close(U, r["U"], (split + acc(c.K)) * r["SU"], "U")
    close(y, r["y"], 2.0 ** -8 * r["y"].abs() + acc(c.K) * r["Sy"] + 2.0 ** -14 * r["Slora"] + 1e-30, "y")


def check_backward(c, U, dX, dA, dB):
    r = c.backward(U)
    half = 2.0 ** -8 if dX.dtype == torch.bfloat16 else 2.0 ** -23
    close(dX, r["dX"], half * r["dX"].abs() + acc(c.N) * r["SdX"] + 2.0 ** -14 * r["Slora"] + 1e-30, "dX")
    # G's own error (split of B, its sum), then the split of G and the sum over rows
    close(dA, r["dA"], (2 * 2.0 ** -16 + acc(c.N) + acc(c.M)) * r["SdA"], "dA")
    close(dB, r["dB"], (2.0 ** -16 + acc(c.M)) * r["SdB"], "dB")


SHAPES = [
    # M, N, K, adapters, rows, mask
    (1, 64, 64, 1, "one", False),
    (1, 192, 1088, 5, "random", True),
    (2, 128, 64, 2, "distinct", False),
    (7, 320, 448, 3, "none", True),
    (8, 256, 2048, 16, "distinct", False),
    (16, 896, 896, 4, "wild", True),
    (17, 64, 896, 64, "distinct", True),
    (33, 1024, 192, 2, "runs", False),
    (64, 576, 640, 9, "random", True),
    (65, 128, 4864, 1, "one", True),
    (129, 448, 512, 40, "wild", False),
    (200, 64, 64, 3, "runs", True),
    (257, 512, 384, 7, "random", True),
    (300, 1088, 320, 300, "distinct", False),
    (513, 192, 576, 2, "runs", True),
    (1100, 320, 256, 1, "random", False),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_forward(ops, shape, dtype):
    M, N, K, n, kind, mask = shape
    c = Case(ops, M, N, K, n, kind, dtype, mask, seed=M + N, pool=24 if dtype == torch.float32 else 0)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=dev())
    U = torch.full((M, 16), float("nan"), device=dev())
    ws = torch.full((ops.lora_multi_workspace_size(M, N, K, n),), 255, dtype=torch.uint8, device=dev())
    ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask, y=y, U=U, workspace=ws)
    check_forward(c, y, U)
    y2, U2 = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)
    assert torch.equal(y, y2) and torch.equal(U, U2)
    assert ops.device_error() == 0


BIG = [
    # weights large enough for the tensor-core kernel of few rows and for tiles cut between CTAs
    (17, 9728, 2112, 5, "random", False),
    (33, 4864, 4864, 33, "distinct", True),
    (64, 8192, 2880, 6, "wild", False),
    (48, 5184, 5120, 48, "distinct", False),
    (1, 5120, 5120, 2, "one", True),
    (16, 2112, 9728, 3, "random", True),
    (520, 2560, 896, 9, "runs", True),
    (520, 2560, 896, 30, "random", True),
]


@pytest.mark.parametrize("shape", BIG, ids=["-".join(map(str, s)) for s in BIG])
def test_forward_of_large_weights(ops, shape):
    M, N, K, n, kind, mask = shape
    c = Case(ops, M, N, K, n, kind, torch.float32, mask, seed=M)
    ws = torch.full((ops.lora_multi_workspace_size(M, N, K, n),), 255, dtype=torch.uint8, device=dev())
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=dev())
    U = torch.full((M, 16), float("nan"), device=dev())
    for _ in range(3):   # the same workspace again: what a call leaves in it does not matter
        y.fill_(float("nan"))
        ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask, y=y, U=U, workspace=ws)
        check_forward(c, y, U)
    assert ops.device_error() == 0


BIG_ROWS = [
    # rows without an adapter, one row past the narrow form, a tile of 64 outputs at the end, ends inside a step
    (20, 5184, 5184, 3, "none", False),
    (32, 9792, 2880, 32, "distinct", True),
    (33, 5184, 5120, 7, "wild", False),
    (64, 19456, 1088, 64, "distinct", False),
    (50, 4928, 8256, 1, "one", True),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", BIG_ROWS, ids=["-".join(map(str, s)) for s in BIG_ROWS])
def test_forward_of_large_weights_in_both_types(ops, shape, dtype):
    M, N, K, n, kind, mask = shape
    c = Case(ops, M, N, K, n, kind, dtype, mask, seed=M + K, pool=24)
    ws = torch.full((ops.lora_multi_workspace_size(M, N, K, n),), 255, dtype=torch.uint8, device=dev())
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=dev())
    U = torch.full((M, 16), float("nan"), device=dev())
    for _ in range(2):
        y.fill_(float("nan"))
        ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask, y=y, U=U, workspace=ws)
        check_forward(c, y, U)
    assert ops.device_error() == 0


def test_a_diverged_adapter_stays_alone_beside_large_weights(ops):
    """Infinite and NaN factors of one adapter reach its own rows only."""
    c = Case(ops, 40, 5184, 5120, 5, "distinct", seed=8)
    want, _ = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan)
    c.A[2].fill_(float("inf")), c.B[2].fill_(float("nan"))
    y, U = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan)
    own = (c.rows == 2).to(dev())
    assert own.any() and not torch.isfinite(y[own]).any()
    assert torch.equal(y[~own], want[~own])


@pytest.mark.parametrize("dx32", [True, False], ids=["dx32", "dx16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
def test_backward(ops, shape, dx32):
    M, N, K, n, kind, mask = shape
    c = Case(ops, M, N, K, n, kind, torch.float32, mask, seed=M + K, pool=16)
    U = c.forward()["U"].float()
    dX = torch.full((M, K), float("nan"), dtype=torch.float32 if dx32 else torch.bfloat16, device=dev())
    dA, dB = c.set.empty_grads()
    gap_a = torch.as_strided(dA, (n - 1, 16), (dA.stride(0), 1), 16 * K) if n > 1 else None
    dA.fill_(float("nan")), dB.fill_(float("nan"))
    if n > 1:
        gap_a.fill_(5.0)
    ws = torch.full((ops.lora_multi_workspace_size(M, N, K, n),), 255, dtype=torch.uint8, device=dev())
    ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX=dX, dA=dA, dB=dB, workspace=ws)
    check_backward(c, U, dX, dA, dB)
    if n > 1:
        assert (gap_a == 5.0).all()   # what lies between two adapters of a pool stays
    r2 = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=dx32)
    assert torch.equal(dX, r2[0]) and torch.equal(dA, r2[1]) and torch.equal(dB, r2[2])
    assert ops.device_error() == 0


@pytest.mark.parametrize("M,n,kind", [(1, 1, "one"), (70, 3, "random"), (1025, 5, "wild"), (2500, 4096, "distinct"),
                                      (3000, 2, "runs"), (64, 7, "none")])
def test_plan_sorts_rows_by_adapter(ops, M, n, kind):
    rows = rows_of(kind, M, n, torch.Generator().manual_seed(M))
    p = ops.lora_multi_plan(rows.to(dev()), n).data.cpu().numpy()
    up = lambda x: -(-x // 4) * 4
    r = rows.numpy().astype(np.int64)
    r = np.where((r >= 0) & (r < n), r, n)
    o_perm, o_off, o_tile = 4 + up(M), 4 + 2 * up(M), 4 + 2 * up(M) + up(n + 1)
    assert np.array_equal(p[4:4 + M], np.where(r == n, -1, r))
    order = np.argsort(r, kind="stable")
    assert np.array_equal(p[o_perm:o_perm + M], order)
    assert np.array_equal(p[o_off:o_off + n + 1], np.searchsorted(r[order], np.arange(n + 1)))
    tiles = p[o_tile:o_tile + 4 * p[0]].reshape(-1, 4)
    want = [[a if a < n else -1, s, min(64, e - s), 0] for a in range(n + 1)
            for b, e in [(np.searchsorted(r[order], a), np.searchsorted(r[order], a, side="right"))]
            for s in range(b, e, 64)]
    assert tiles.tolist() == want


def test_accumulation(ops):
    c = Case(ops, 90, 192, 320, 4, "runs", mask=True, seed=3)
    rows = c.rows.clone()
    rows[rows == 2] = -1     # adapter 2 has no row: its gradients only stay or become zero
    c.rows, c.plan = rows, ops.lora_multi_plan(rows.to(dev()), 4)
    U = c.forward()["U"].float()
    dX, dA, dB = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=True)
    assert (dA[2] == 0).all() and (dB[2] == 0).all()
    oX, oA, oB = (torch.randn_like(t) for t in (dX, dA, dB))
    aX, aA, aB = oX.clone(), oA.clone(), oB.clone()
    ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX=aX, dA=aA, dB=aB, accumulate=True,
                              grad_accumulate=True)
    assert torch.equal(aA, oA + dA) and torch.equal(aB, oB + dB)     # one fp32 add each
    assert ((aX - (oX + dX)).abs() <= 2.0 ** -21 * (oX.abs() + dX.abs())).all()
    assert ops.device_error() == 0


BIG_FEW = [
    # gradients of few rows: weights whose tiles are cut between CTAs, ends inside a step or a tile
    (1, 5120, 5120, 2, "one", True),
    (2, 9728, 2112, 2, "distinct", False),
    (16, 2112, 9728, 3, "random", True),
    (31, 5184, 4928, 31, "wild", True),
    (32, 4864, 8192, 5, "distinct", False),
    (33, 2112, 4864, 5, "random", True),
    (33, 9728, 8256, 40, "wild", True),
    (64, 8256, 9728, 64, "distinct", False),
]


@pytest.mark.parametrize("dx32", [True, False], ids=["dx32", "dx16"])
@pytest.mark.parametrize("shape", BIG_FEW, ids=["-".join(map(str, s)) for s in BIG_FEW])
def test_backward_of_large_weights(ops, shape, dx32):
    M, N, K, n, kind, mask = shape
    c = Case(ops, M, N, K, n, kind, torch.float32, mask, seed=N)
    U = c.forward()["U"].float()
    ws = torch.full((ops.lora_multi_workspace_size(M, N, K, n),), 255, dtype=torch.uint8, device=dev())
    dX = torch.full((M, K), float("nan"), dtype=torch.float32 if dx32 else torch.bfloat16, device=dev())
    dA, dB = c.set.empty_grads()
    for _ in range(3):   # the same workspace again
        dX.fill_(float("nan"))
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX=dX, dA=dA, dB=dB, workspace=ws)
        check_backward(c, U, dX, dA, dB)
    assert ops.device_error() == 0


@pytest.mark.parametrize("M,n", [(1, 1), (5, 40), (32, 3)])
def test_accumulation_of_few_rows(ops, M, n):
    c = Case(ops, M, 320, 192, n, "random", mask=True, seed=M)
    U = c.forward()["U"].float()
    dX, dA, dB = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=True)
    oX, oA, oB = (torch.randn_like(t) for t in (dX, dA, dB))
    aX, aA, aB = oX.clone(), oA.clone(), oB.clone()
    ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX=aX, dA=aA, dB=aB, accumulate=True,
                              grad_accumulate=True)
    assert torch.equal(aX, oX + dX) and torch.equal(aA, oA + dA) and torch.equal(aB, oB + dB)   # one fp32 add each


@pytest.mark.parametrize("M", [70, 300])
def test_accumulation_with_more_adapters_than_slots(ops, M):
    c = Case(ops, M, 192, 320, 30, "random", mask=True, seed=M)
    U = c.forward()["U"].float()
    dX, dA, dB = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=True)
    oX, oA, oB = (torch.randn_like(t) for t in (dX, dA, dB))
    aX, aA, aB = oX.clone(), oA.clone(), oB.clone()
    ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX=aX, dA=aA, dB=aB, accumulate=True,
                              grad_accumulate=True)
    # one fp32 add each (adapters without a row: 0 added, or left)
    assert torch.equal(aX, oX + dX) and torch.equal(aA, oA + dA) and torch.equal(aB, oB + dB)


def test_two_streams_at_once(ops):
    """Calls that overlap, each with its own workspace and plan, do not meet."""
    cs = [Case(ops, M, 2112, 1088, 12, "random", mask=True, seed=M) for M in (5, 40, 90, 300)]
    want = [ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask) for c in cs]
    grads = [ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, w[1], c.dY, mask=c.mask) for c, w in zip(cs, want)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = []
        for c, s, w in zip(cs, st, want):
            f = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask, stream=s)
            got.append((f, ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, f[1], c.dY, mask=c.mask, stream=s)))
        torch.cuda.synchronize()
        for (f, b), w, g in zip(got, want, grads):
            assert all(torch.equal(p, q) for p, q in zip((*f, *b), (*w, *g)))
    assert ops.device_error() == 0


def test_two_streams_beside_large_weights(ops):
    """The same, where tiles are cut between CTAs that wait for one another's sums."""
    cs = [Case(ops, M, N, K, 6, "random", seed=M) for M, N, K in ((40, 5184, 5120), (20, 9728, 4928), (64, 8256, 9728))]
    want = [ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan) for c in cs]
    grads = [ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, w[1], c.dY) for c, w in zip(cs, want)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = []
        for c, s in zip(cs, st):
            f = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, stream=s)
            got.append((*f, *ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, f[1], c.dY, stream=s)))
        torch.cuda.synchronize()
        for g, f, b in zip(got, want, grads):
            assert all(torch.equal(p, q) for p, q in zip(g, (*f, *b)))
    assert ops.device_error() == 0


def test_gradients_against_differences(ops):
    """sum(y . dY) as a function of A, B and x, in 64 bits, differenced."""
    c = Case(ops, 37, 128, 128, 3, "random", mask=True, seed=5)
    c.A, c.B = c.A.clone(), c.B.clone()
    U = c.forward()["U"].float()
    dX, dA, dB = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=True)
    r = c.backward(U)
    a, _ = c.own()
    A0, B0, x0 = c.A.double(), c.B.double(), c.x.double()
    w, keep, s = c.weight(), c.keep(), c.scale.double()[a][:, None]
    has = c.own()[1]

    def loss(A, B, x):
        u = torch.bmm(A[a], (x * keep)[:, :, None])[:, :, 0] * has
        return ((x @ w.t() + torch.bmm(B[a], u[:, :, None])[:, :, 0] * s) * c.dY.double()).sum()
    g = torch.Generator().manual_seed(1)
    for name, got, base, S in (("A", dA, A0, r["SdA"]), ("B", dB, B0, r["SdB"]), ("x", dX, x0, r["SdX"] + r["Slora"])):
        for _ in range(12):
            i = tuple(int(torch.randint(0, k, (1,), generator=g)) for k in base.shape)
            h = 0.5   # the loss is linear in each factor: the difference has no step error
            args = {"A": A0, "B": B0, "x": x0}
            up, lo = base.clone(), base.clone()
            up[i] += h
            lo[i] -= h
            num = (loss(**{**args, name: up}) - loss(**{**args, name: lo})) / (2 * h)
            assert abs(float(got[i]) - float(num)) <= 2.0 ** -13 * float(S[i]) + 1e-9 * abs(float(loss(A0, B0, x0))), (name, i)


def test_masks_are_those_of_the_single_adapter_linear(ops):
    """One adapter for all rows, the framework's dropout bits: the single-adapter linear's results."""
    M, N, K = 130, 256, 512
    c = Case(ops, M, N, K, 1, "one", seed=9)
    key = ops.dropout_key(seed=3, step=2, layer=1, linear=4, p=0.1)
    scale = torch.tensor([32.0 / 16 / 0.9], device=dev())
    A, B = c.A[0].contiguous(), c.B[0].contiguous()
    y, U, mask = ops.lora_linear_fwd(c.W, c.x, A, B, key)
    m = ops.dropout_mask(key, M, K)
    assert torch.equal(m, mask)
    s = ops.LoraSet(c.A, c.B, scale)
    y2, U2 = ops.lora_linear_fwd_multi(c.W, c.x, s, c.plan, mask=m)
    assert torch.allclose(U, U2, rtol=0, atol=2.0 ** -14 * float(U.abs().max()))
    assert ((y.float() - y2.float()).abs() <= 2.0 ** -6 * y.float().abs() + 1e-3).all()
    dX, dA, dB = ops.lora_linear_bwd(c.W, c.x, A, B, key, U, mask, c.dY, dX_f32=True)
    dX2, dA2, dB2 = ops.lora_linear_bwd_multi(c.W, c.x, s, c.plan, U, c.dY, mask=m, dX_f32=True)
    for p, q in ((dX, dX2), (dA, dA2[0]), (dB, dB2[0])):
        assert float((p - q).norm()) <= 1e-4 * float(p.norm())


@pytest.mark.parametrize("M", [3, 60, 200, 400])
@pytest.mark.parametrize("n", [3, 40])
def test_a_diverged_adapter_stays_alone(ops, M, n):
    """NaN and infinities in one adapter (and in a dropped element of x) reach no row of another."""
    N, K = 128, 192
    c = Case(ops, M, N, K, n, "distinct", mask=True, seed=M)
    good = Case(ops, M, N, K, n, "distinct", mask=True, seed=M)
    c.B[1, 5, 3], c.B[1, 70, :] = float("nan"), float("inf")
    c.A[1, 2, 9] = float("-inf")
    r = c.rows.to(dev()).long()
    bad = r == 1
    y0, U0 = ops.lora_linear_fwd_multi(good.W, good.x, good.set, good.plan, mask=good.mask)
    y1, U1 = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)
    assert torch.equal(y0[~bad], y1[~bad]) and torch.equal(U0[~bad], U1[~bad])
    assert not torch.isfinite(y1[bad][:, 5]).any() and not torch.isfinite(y1[bad][:, 70]).any()
    U = good.forward()["U"].float()
    g0 = ops.lora_linear_bwd_multi(good.W, good.x, good.set, good.plan, U, good.dY, mask=good.mask, dX_f32=True)
    g1 = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=True)
    others = torch.arange(n, device=dev()) != 1
    assert torch.equal(g0[0][~bad], g1[0][~bad])
    assert torch.equal(g0[1][others], g1[1][others]) and torch.equal(g0[2], g1[2])
    assert torch.isnan(g1[1][1]).any() == bad.any()
    # only B's diverged rows: A and U are finite, so only these columns of y are not
    c2 = Case(ops, M, N, K, n, "distinct", mask=True, seed=M)
    c2.B[1, 5, 3] = float("nan")
    y2, _ = ops.lora_linear_fwd_multi(c2.W, c2.x, c2.set, c2.plan, mask=c2.mask)
    keep = torch.ones(N, dtype=torch.bool, device=dev())
    keep[5] = False
    assert torch.equal(y2[:, keep], y0[:, keep]) and torch.isnan(y2[bad][:, 5]).all() and torch.equal(y2[~bad], y0[~bad])
    # a dropped element of x: the adapter does not see it, the frozen base does
    c3 = Case(ops, M, N, K, n, "distinct", mask=True, seed=M)
    c3.mask[0, 1] &= ~4
    U3a = ops.lora_linear_fwd_multi(c3.W, c3.x, c3.set, c3.plan, mask=c3.mask)[1]
    c3.x[0, 34] = float("nan")
    y3, U3 = ops.lora_linear_fwd_multi(c3.W, c3.x, c3.set, c3.plan, mask=c3.mask)
    assert torch.equal(U3, U3a) and torch.isfinite(y3[1:]).all()
    assert ops.device_error() == 0


@pytest.mark.parametrize("M", [5, 40, 150, 600])
def test_another_stream_and_a_captured_call(ops, M):
    """plan, forward and backward on a side stream, captured once and replayed with other rows and inputs."""
    c = Case(ops, M, 192, 256, 6, "random", mask=True, seed=M)
    st = torch.cuda.Stream()
    rows = c.rows.to(dev())
    bufs = dict(y=torch.empty(M, 192, dtype=torch.bfloat16, device=dev()), U=torch.empty(M, 16, device=dev()))
    dX = torch.empty(M, 256, device=dev())
    dA, dB = c.set.empty_grads()
    ws = torch.empty(ops.lora_multi_workspace_size(M, 192, 256, 6), dtype=torch.uint8, device=dev())

    def go():
        ops.lora_multi_plan(rows, 6, plan=c.plan, stream=st)
        ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask, workspace=ws, stream=st, **bufs)
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, bufs["U"], c.dY, mask=c.mask, dX=dX, dA=dA, dB=dB,
                                  workspace=ws, stream=st)
    st.wait_stream(torch.cuda.current_stream())
    go()
    st.synchronize()
    check_forward(c, bufs["y"], bufs["U"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        go()
    for seed in (1, 2):
        other = Case(ops, M, 192, 256, 6, "wild", mask=True, seed=M + seed)
        rows.copy_(other.rows.to(dev()))
        c.rows = other.rows
        c.x.copy_(other.x), c.dY.copy_(other.dY), c.mask.copy_(other.mask)
        for t in (*bufs.values(), dX, dA, dB):
            t.fill_(float("nan"))
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            g.replay()
        st.synchronize()
        check_forward(c, bufs["y"], bufs["U"])
        check_backward(c, bufs["U"], dX, dA, dB)
    assert ops.device_error() == 0


def test_memory_of_the_call_s_stream(ops):
    """Gradients made by a call on another stream come from that stream's memory, not from what the
    current one has just given back."""
    c = Case(ops, 9, 128, 256, 3)
    U = torch.zeros(9, 16, device=dev())
    st = torch.cuda.Stream()
    old = [torch.empty(3, 16, 256, device=dev()), torch.empty(3, 128, 16, device=dev())]
    ptrs = {t.data_ptr() for t in old}
    del old
    torch.cuda.synchronize()
    _, dA, dB = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, stream=st)
    torch.cuda.synchronize()
    assert not ptrs & {dA.data_ptr(), dB.data_ptr()}


def test_more_outputs_than_a_grid_s_second_axis(ops):
    """2^23 + 64 output rows: 65537 tiles of the weight; checked at both ends and at the 65535th tile."""
    M, N, K = 2, 2 ** 23 + 64, 64
    g = torch.Generator(device=dev()).manual_seed(4)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=dev())
    absmax = 0.02 * (2 + torch.rand(1, N, generator=g, device=dev()))
    x = torch.randn(M, K, generator=g, device=dev()).bfloat16()
    A = torch.randn(1, 16, K, generator=g, device=dev()) / 8
    B = torch.randn(1, N, 16, generator=g, device=dev()) / 8
    W, aset = ops.NF4Weight(codes, absmax, N, K), ops.LoraSet(A, B, torch.ones(1, device=dev()))
    plan = ops.lora_multi_plan(torch.zeros(M, dtype=torch.int32, device=dev()), 1)
    y, U = ops.lora_linear_fwd_multi(W, x, aset, plan)
    close(U, x.double() @ A[0].double().t(), acc(K) * (x.double().abs() @ A[0].double().abs().t()), "U")
    for a in (0, 65535 * 128 - 64, N - 128):
        q = torch.stack([codes[a:a + 128] >> 4, codes[a:a + 128] & 15], -1).view(128, K).long()
        w = (torch.tensor(LEVELS, device=dev())[q] * absmax[0, a:a + 128, None]).bfloat16().double()
        b, S = B[0, a:a + 128].double(), x.double().abs() @ w.abs().t()
        want = x.double() @ w.t() + U.double() @ b.t()
        close(y[:, a:a + 128], want, 2.0 ** -8 * want.abs() + acc(K) * S + 2.0 ** -14 * (U.double().abs() @ b.abs().t()), "y")
    assert ops.device_error() == 0


def test_a_plan_of_another_device_is_refused(ops):
    c = Case(ops, 9, 128, 128, 3)
    elsewhere = ops.LoraPlan(torch.empty_like(c.plan.data, device="cpu"), 9, 3)
    with pytest.raises(ValueError, match="device"):
        ops.lora_linear_fwd_multi(c.W, c.x, c.set, elsewhere)
    with pytest.raises(ValueError, match="device"):
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, elsewhere, torch.zeros(9, 16, device=dev()), c.dY)
    with pytest.raises(ValueError, match="device"):
        ops.lora_multi_plan(c.rows.to(dev()), 3, plan=elsewhere)


def test_refusals(ops):
    c = Case(ops, 9, 128, 128, 3)
    f = lambda **k: ops.lora_linear_fwd_multi(k.pop("W", c.W), k.pop("x", c.x), k.pop("s", c.set), k.pop("p", c.plan), **k)
    other = Case(ops, 10, 128, 192, 2)
    for bad in (dict(x=c.x.float()), dict(x=c.x[:4]), dict(p=other.plan), dict(s=other.set), dict(W=other.W),
                dict(x=c.x.t().contiguous().t()), dict(y=torch.empty(9, 128, device=dev())),
                dict(U=torch.empty(9, 8, device=dev())), dict(mask=torch.zeros(9, 8, dtype=torch.int32, device=dev())),
                dict(x=c.x.cpu()), dict(W=ops.Bf16Weight(c.x, 128, 128))):
        with pytest.raises(ValueError):
            f(**bad)
    with pytest.raises(ops.WsError):
        f(workspace=torch.empty(16, dtype=torch.uint8, device=dev()))
    b16 = Case(ops, 9, 128, 128, 3, dtype=torch.bfloat16)
    U = torch.zeros(9, 16, device=dev())
    with pytest.raises(ops.WsError):      # bf16 adapters are not trained
        ops.lora_linear_bwd_multi(b16.W, b16.x, b16.set, b16.plan, U, b16.dY)
    with pytest.raises(ValueError):
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, accumulate=True)
    with pytest.raises(ops.WsError):      # adding needs an fp32 dX
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, accumulate=True,
                                  dX=torch.zeros(9, 128, dtype=torch.bfloat16, device=dev()))
    with pytest.raises(ValueError):
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, dA=torch.zeros(3, 16, 64, device=dev()))
    with pytest.raises(ValueError):
        ops.lora_multi_plan(torch.zeros(9, dtype=torch.int64, device=dev()), 3)
    assert ops.device_error() == 0
