"""The many-adapter linear over its whole range: long sums, many rows and adapters, offsets past
32 bits, against the formulas in 64 bits (Case, check_forward and check_backward are those of test_gpu_lora_multi)."""
import pytest
import torch

from gpu_util import dev
from test_gpu_lora_multi import Case, check_backward, check_forward, ops  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_set_keeps_its_tensors(ops):  # noqa: F811
    """A tensor that is given other storage afterwards: the set still reads the memory that it was made for."""
    c = Case(ops, 20, 128, 192, 3, seed=2)
    A, B, s = c.A.clone(), c.B.clone(), c.scale.clone()
    aset = ops.LoraSet(A, B, s)
    want = ops.lora_linear_fwd_multi(c.W, c.x, aset, c.plan)[0]
    taken = {t.data_ptr() for t in (A, B, s)}
    for t in (A, B, s):
        t.data = torch.full_like(t, float("nan"))
    fresh = [torch.full(t.shape, float("nan"), device=dev()) for t in (A, B, s) for _ in range(16)]
    assert not taken & {t.data_ptr() for t in fresh}
    assert torch.equal(ops.lora_linear_fwd_multi(c.W, c.x, aset, c.plan)[0], want)


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("M", [20000, 65536, 262144 + 5])
def test_gradients_of_an_adapter_with_many_rows(ops, M, mask):  # noqa: F811
    """dA and dB of one adapter whose terms all have one sign.

    A warp adds up a sixty-fourth of the rows, 16 at a time: n = M / 64 sums.  The 16 rows' own sum is off by at most
    2^-20 of itself (a few truncations at 2^-23), and each of the n additions rounds to nearest, 2^-24 of the sum so far,
    in no fixed direction: by Hoeffding's inequality 8 sqrt(n) 2^-24 of the whole holds but for one element in 10^13, and
    the root mean square over all elements is below sqrt(n) 2^-24.  (Sums that cut off instead of rounding drift by
    about 0.2 n 2^-23 for each addition.)  dA's G adds its own error, 2^-20: a sum of 128 terms in fp32 from three bf16
    parts, which hold all 24 bits."""
    N = K = 128
    g = torch.Generator(device=dev()).manual_seed(M)
    pos = lambda *s: torch.rand(*s, generator=g, device=dev()) + 0.25
    x, dY, U = pos(M, K).bfloat16(), pos(M, N).bfloat16(), pos(M, 16)
    A, B, scale = pos(1, 16, K), pos(1, N, 16), torch.full((1,), 0.75, device=dev())
    W = ops.NF4Weight(torch.zeros(N, K // 2, dtype=torch.uint8, device=dev()), torch.ones(K // 64, N, device=dev()), N, K)
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (M, K // 32), generator=g, dtype=torch.int32, device=dev()) if mask else None
    plan = ops.lora_multi_plan(torch.zeros(M, dtype=torch.int32, device=dev()), 1)
    _, dA, dB = ops.lora_linear_bwd_multi(W, x, ops.LoraSet(A, B, scale), plan, U, dY, mask=bits)
    xm = x.double()
    if mask:
        xm *= ((bits.long()[:, :, None] >> torch.arange(32, device=dev())) & 1).view(M, K)
    G = dY.double() @ B[0].double()
    step, n = 2.0 ** -20, M / 64
    for what, got, want, own in (("dB", dB[0], 0.75 * (dY.double().t() @ U.double()), step),
                                 ("dA", dA[0], 0.75 * (G.t() @ xm), 2 * step)):
        off = (got.double() - want) / want
        assert float(off.abs().max()) <= 8 * n ** 0.5 * 2.0 ** -24 + own, (what, float(off.abs().max()))
        assert float(off.square().mean().sqrt()) <= n ** 0.5 * 2.0 ** -24 + own, (what, float(off.square().mean().sqrt()))
    assert ops.device_error() == 0


@pytest.mark.parametrize("M", [1, 40, 100, 300])
def test_gradients_of_an_adapter_without_rows_are_zero_whatever_its_scale(ops, M):  # noqa: F811
    c = Case(ops, M, 128, 192, 4, "none", seed=M)
    c.rows = torch.zeros(M, dtype=torch.int32)
    c.plan = ops.lora_multi_plan(c.rows.to(dev()), 4)
    c.scale[1], c.scale[2], c.scale[3] = float("nan"), float("inf"), float("-inf")
    U = c.forward()["U"].float()
    _, dA, dB = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY)
    assert torch.isfinite(dA[0]).all() and (dA[0] != 0).any()
    for d in (dA, dB):
        assert (d[1:] == 0).all() and not torch.signbit(d[1:]).any()
    # added into what is there: those stay as they are, bit for bit
    oA, oB = torch.randn_like(dA), torch.randn_like(dB)
    aA, aB = oA.clone(), oB.clone()
    ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, dA=aA, dB=aB, grad_accumulate=True)
    assert torch.equal(aA[1:], oA[1:]) and torch.equal(aB[1:], oB[1:])


def test_graphs_captured_far_apart_share_nothing(ops):  # noqa: F811
    """Graphs of calls whose tiles are cut between CTAs, captured thousands of calls apart and replayed at once, each with
    its own workspace: no flag of one is another's, however many calls of any kind were made in between."""
    M, N, K, n = 300, 2112, 1088, 6
    cs = [Case(ops, M, N, K, n, "random", mask=True, seed=s) for s in range(5)]
    want, made = [], []
    for c in cs:
        f = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)
        want.append((*f, *ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, f[1], c.dY, mask=c.mask)))
    ws = torch.empty(ops.lora_multi_workspace_size(M, N, K, n), dtype=torch.uint8, device=dev())
    out = dict(y=torch.empty_like(want[0][0]), U=torch.empty_like(want[0][1]), workspace=ws)

    def capture(c, w):
        st, got = torch.cuda.Stream(), [torch.empty_like(t) for t in w]
        own = torch.empty_like(ws)
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask, y=got[0], U=got[1], workspace=own, stream=st)
            ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, got[1], c.dY, mask=c.mask, dX=got[2], dA=got[3], dB=got[4],
                                      workspace=own, stream=st)
        made.append((g, st, got, own))
    capture(cs[0], want[0])
    for c, w in zip(cs[1:], want[1:]):
        for _ in range(3450):
            ops.lora_linear_fwd_multi(cs[0].W, cs[0].x, cs[0].set, cs[0].plan, mask=cs[0].mask, **out)
        capture(c, w)
    torch.cuda.synchronize()
    for _ in range(40):
        for _, _, got, _ in made:
            for t in got:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st, _, _ in made:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, got, _), w in zip(made, want):
            assert all(torch.equal(p, q) for p, q in zip(got, w))
    assert ops.device_error() == 0


@pytest.mark.parametrize("M,n,kind", [(100, 8, "all"), (100, 9, "all"), (129, 3, "all"), (256, 40, "one tile of 8"),
                                      (1300, 40, "one tile of 8"), (1300, 40, "one tile of 9"), (700, 5, "none"),
                                      (513, 4096, "one each")])
def test_slots_of_a_plan(ops, M, n, kind):  # noqa: F811
    """The plan's second half: each row's slot and each tile row's adapters in order of their first row; the most slots of
    any tile row, or -1 where one has more than eight."""
    tile = 128 if M <= 128 else 256 if M <= 256 else 512
    rows = torch.full((M,), 7 % n, dtype=torch.int32)
    if kind == "all":
        rows = (torch.arange(M, dtype=torch.int32) * 5) % n
    elif kind.startswith("one tile"):
        k, a = int(kind[-1]), (M - 1) // tile * tile        # (the last tile row; the others hold adapter 7)
        rows[a:] = torch.arange(M - a, dtype=torch.int32) % k * 3 + 10
        rows[a + 1] = -1
    elif kind == "none":
        rows[:] = n
    else:
        rows[:] = torch.arange(M, dtype=torch.int32) // tile * 17
    p = ops.lora_multi_plan(rows.to(dev()), n).data.cpu()
    up = lambda x: -(-x // 4) * 4
    tiles = M // 64 + min(n + 1, M)
    o_slot = 4 + 2 * up(M) + up(n + 1) + 4 * tiles
    o_list = o_slot + up(M)
    most, many = 0, False
    for t in range(-(-M // tile)):
        seen = []
        for i in range(t * tile, min(M, (t + 1) * tile)):
            a = int(rows[i])
            if 0 <= a < n and a not in seen:
                seen.append(a)
        if len(seen) > 8:
            many = True      # the batch takes the other form: slots are not read
            continue
        most = max(most, len(seen))
        assert p[o_list + 8 * t:o_list + 8 * t + 8].tolist() == seen + [-1] * (8 - len(seen))
        want = [seen.index(int(a)) if int(a) in seen else -1 for a in rows[t * tile:min(M, (t + 1) * tile)]]
        assert p[o_slot + t * tile:o_slot + t * tile + len(want)].tolist() == want
    assert int(p[1]) == (-1 if many else most) and many == (kind == "one tile of 9" or (kind, n) == ("all", 9))


def rms(x):
    return float(x.double().square().mean().sqrt())


def two_parts(t):
    """A value as the sum of two bf16 numbers: what two parts would keep of it."""
    hi = t.bfloat16().float()
    return hi + (t - hi).bfloat16().float()


@pytest.mark.parametrize("M,N,K", [(40, 1024, 4096), (200, 4096, 4096), (700, 1024, 2048)])
def test_fp32_factors_enter_with_all_their_bits(ops, M, N, K):  # noqa: F811
    """Root mean square errors of U, dA and dB relative to the values'.

    U: a 64-deep step is 12 tensor-core sums, small parts first, so that the last four (the high part's, 16 products each)
    cut off up to 2^-23 of the step's sum each, and those before them 2^-8 of that; the steps' sums are random in sign and
    add up in fp32 (2^-24 each, in at most 8 rounds that see the whole): 2^-21 + 2^-23 of the root mean square.  G is made
    the same way.  dA, dB: a 16-row step cuts off 2^-23 of itself and the additions round by 2^-24 of sums that grow like
    the square root of their number: 2^-22 in all, for dA beside G's error.  A factor of two bf16 parts would be off by
    2^-18 at most in each product, about 2^-19.3 root mean square: more than each bound, which is asserted."""
    c = Case(ops, M, N, K, 3, "random", mask=True, seed=N)
    y, U = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)
    r = c.forward()
    U64 = r["U"].float()
    _, dA, dB = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U64, c.dY, mask=c.mask)
    b = c.backward(U64)
    one, total = 2.0 ** -21 + 2.0 ** -23, 2.0 ** -22
    assert rms(U - r["U"]) <= one * rms(r["U"]), rms(U - r["U"]) / rms(r["U"])
    assert rms(dB - b["dB"]) <= total * rms(b["dB"]), rms(dB - b["dB"]) / rms(b["dB"])
    assert rms(dA - b["dA"]) <= (one + total) * rms(b["dA"]), rms(dA - b["dA"]) / rms(b["dA"])
    # two parts fail each of them
    A, B = c.A, c.B
    c.A, c.B = two_parts(A), two_parts(B)
    assert rms(c.forward()["U"] - r["U"]) > one * rms(r["U"])
    assert rms(c.backward(U64)["dA"] - b["dA"]) > (one + total) * rms(b["dA"])
    c.A, c.B = A, B
    assert rms(c.backward(two_parts(U64))["dB"] - b["dB"]) > total * rms(b["dB"])


def test_the_most_adapters(ops):  # noqa: F811
    """4096 adapters: a few with rows, the gradients of all others zero; every row another adapter, too."""
    for M, kind in ((300, "random"), (4096, "distinct"), (50, "random")):
        c = Case(ops, M, 64, 128, 4096, kind, mask=True, seed=M)
        y, U = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)
        a, has = c.own()
        xm = c.x.double() * c.keep()
        U64 = torch.einsum("mjk,mk->mj", c.A[a].double(), xm) * has
        assert ((U - U64).abs() <= 2.0 ** -18 * torch.einsum("mjk,mk->mj", c.A[a].double().abs(), xm.abs()) + 1e-30).all()
        check_forward(c, y, U)
        _, dA, dB = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask)
        have = torch.zeros(4096, dtype=torch.bool, device=dev())
        have[a[has[:, 0] > 0]] = True
        assert (dA[~have] == 0).all() and (dB[~have] == 0).all() and (dB[have] != 0).flatten(1).any(1).all()
        hot = torch.zeros(4096, M, dtype=torch.float64, device=dev())
        hot[a, torch.arange(M, device=dev())] = has[:, 0]
        su = c.scale.double()[a][:, None] * U.double()
        want = torch.stack([hot @ (su[:, j:j + 1] * c.dY.double()) for j in range(16)], -1)
        S = torch.stack([hot @ (su[:, j:j + 1] * c.dY.double()).abs() for j in range(16)], -1)
        assert ((dB - want).abs() <= 2.0 ** -18 * S + 1e-30).all()
    assert ops.device_error() == 0


@pytest.mark.parametrize("n", [3, 24])
def test_offsets_past_32_bits(ops, n):  # noqa: F811
    """2^20 rows of 4160 outputs: y and dX hold more than 2^32 elements, the mask 2^32 bits; checked on rows from all over
    and the last ones, with adapters in slots and with more than slots."""
    M, K = 1 << 20, 64
    N = 4160
    g = torch.Generator(device=dev()).manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev())
    rows = torch.randint(-1, n, (M,), generator=g, device=dev(), dtype=torch.int32)
    plan = ops.lora_multi_plan(rows, n)
    at = torch.cat([torch.randint(0, M, (500,), generator=g, device=dev()), torch.arange(M - 40, M, device=dev())])
    a = rows[at].long().clamp(min=0)
    has = (rows[at] >= 0).double()[:, None]
    lev = torch.tensor([-1.0, -0.6962, -0.5251, -0.3949, -0.2844, -0.1848, -0.0911, 0.0,
                        0.0796, 0.1609, 0.2461, 0.3379, 0.4407, 0.5626, 0.7230, 1.0], device=dev())

    def weight(codes, absmax):
        q = torch.stack([codes >> 4, codes & 15], -1).view(codes.shape[0], -1).long()
        return (lev[q].view(codes.shape[0], -1, 64) * absmax.t()[:, :, None]).bfloat16().double().view(codes.shape[0], -1)
    scale = torch.rand(n, generator=g, device=dev()) + 0.5
    s = scale.double()[a][:, None] * has
    # forward: [M, 64] -> [M, 4160]
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev(), dtype=torch.uint8)
    absmax = torch.rand(K // 64, N, generator=g, device=dev()) + 0.5
    x, A, B = rnd(M, K).bfloat16(), rnd(n, 16, K) / 8, rnd(n, N, 16)
    y, U = ops.lora_linear_fwd_multi(ops.NF4Weight(codes, absmax, N, K), x, ops.LoraSet(A, B, scale), plan)
    xd, w = x[at].double(), weight(codes, absmax)
    u = torch.einsum("mjk,mk->mj", A.double()[a], xd) * has
    want = xd @ w.t() + s * torch.einsum("mnj,mj->mn", B.double()[a], u)
    S = xd.abs() @ w.abs().t() + s * torch.einsum("mnj,mj->mn", B.double()[a].abs(), torch.einsum("mjk,mk->mj", A.double()[a].abs(), xd.abs()))
    # a bf16 result, and sums of 64 + 16 products with factors of 16 bits or more
    assert ((y[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * S).all()
    assert ((U[at].double() - u).abs() <= 2.0 ** -18 * torch.einsum("mjk,mk->mj", A.double()[a].abs(), xd.abs()) + 1e-30).all()
    del y
    # backward: dY [M, 64], x and the mask [M, 4160] -> dX [M, 4160]
    N, K = K, N
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=dev(), dtype=torch.uint8)
    absmax = torch.rand(K // 64, N, generator=g, device=dev()) + 0.5
    dY, A, B = rnd(M, N).bfloat16(), rnd(n, 16, K), rnd(n, N, 16) / 8
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev())
    for i in range(0, M, 1 << 16):
        x[i:i + (1 << 16)] = rnd(1 << 16, K)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (M, K // 32), generator=g, dtype=torch.int32, device=dev())
    U = rnd(M, 16)
    dX, dA, dB = ops.lora_linear_bwd_multi(ops.NF4Weight(codes, absmax, N, K), x, ops.LoraSet(A, B, scale), plan, U, dY, mask=mask)
    dd, w = dY[at].double(), weight(codes, absmax)
    keep = ((mask[at].long()[:, :, None] >> torch.arange(32, device=dev())) & 1).view(len(at), K).double()
    G = torch.einsum("mn,mnj->mj", dd, B.double()[a])
    SG = torch.einsum("mn,mnj->mj", dd.abs(), B.double()[a].abs())
    want = dd @ w + keep * s * torch.einsum("mj,mjk->mk", G, A.double()[a])
    S = dd.abs() @ w.abs() + s * torch.einsum("mj,mjk->mk", SG, A.double()[a].abs())
    assert ((dX[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * S).all()
    # gradients: all rows, in 64 bits, some at a time
    wA, SA, wB, SB = (torch.zeros(k, dtype=torch.float64, device=dev()) for k in ((n, 16, K), (n, 16, K), (n, N, 16), (n, N, 16)))
    for i in range(0, M, 1 << 16):
        r, d = rows[i:i + (1 << 16)], dY[i:i + (1 << 16)].double()
        xm = x[i:i + (1 << 16)].double() * ((mask[i:i + (1 << 16)].long()[:, :, None] >> torch.arange(32, device=dev())) & 1).view(-1, K)
        for h in range(n):
            o = (r == h).nonzero()[:, 0]
            sc = float(scale[h])
            Gh = d[o] @ B[h].double()
            wA[h] += sc * (Gh.t() @ xm[o])
            SA[h] += sc * (d[o].abs() @ B[h].double().abs()).t() @ xm[o].abs()
            wB[h] += sc * (d[o].t() @ U[i:i + (1 << 16)][o].double())
            SB[h] += sc * (d[o].abs().t() @ U[i:i + (1 << 16)][o].double().abs())
    # (2^20 / n rows of random sign: the sums stay far below S, and with them the roundings)
    assert ((dA - wA).abs() <= 2.0 ** -18 * SA).all() and ((dB - wB).abs() <= 2.0 ** -18 * SB).all()
    assert ops.device_error() == 0


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("M", [100, 250, 600])
def test_the_adapter_term_of_an_fp32_gradient(ops, M, mask):  # noqa: F811
    """dX of a weight of zeros with one product an element: scale (dY B) A.

    The GEMM takes both factors of the term as two bf16 parts.  The first is off by half a step, at most 2^-8 of the value;
    what remains lies in binades below 2^-8 of the value's, where half a step is 2^-17 of it.  All four products of the
    parts are taken, so the term is off by 2^-16 (the roundings of scale A and G and the cut sums of four add less than
    2^-20).  Without the product of the two second parts it would be off by up to 2^-16 more."""
    N, K, n = 64, 4096, 3
    g = torch.Generator(device=dev()).manual_seed(M)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev())
    A, B = torch.zeros(n, 16, K, device=dev()), torch.zeros(n, N, 16, device=dev())
    A[:, 3], B[:, 7, 3] = rnd(n, K), rnd(n)
    dY = torch.zeros(M, N, dtype=torch.bfloat16, device=dev())
    dY[:, 7] = rnd(M)
    scale = torch.rand(n, generator=g, device=dev()) + 0.5
    W = ops.NF4Weight(torch.zeros(N, K // 2, dtype=torch.uint8, device=dev()), torch.zeros(K // 64, N, device=dev()), N, K)
    rows = torch.randint(0, n, (M,), generator=g, device=dev(), dtype=torch.int32)
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (M, K // 32), generator=g, dtype=torch.int32, device=dev()) if mask else None
    x = rnd(M, K).bfloat16()
    dX, _, _ = ops.lora_linear_bwd_multi(W, x, ops.LoraSet(A, B, scale), ops.lora_multi_plan(rows, n), rnd(M, 16), dY,
                                         mask=bits, dX_f32=True)
    a = rows.long()
    want = (scale[a].double() * dY[:, 7].double() * B[a, 7, 3].double())[:, None] * A[a, 3].double()
    if mask:
        want *= ((bits.long()[:, :, None] >> torch.arange(32, device=dev())) & 1).view(M, K)
    assert ((dX.double() - want).abs() <= (2.0 ** -16 + 2.0 ** -20) * want.abs()).all(), float(((dX.double() - want).abs() / want.abs().clamp(min=1e-30)).max())
    assert ops.device_error() == 0


SUMS = [
    # M, N, K, adapters: few rows (pieces of several parts), one CTA, pairs of 128-wide tiles, and of 256-wide ones
    (5, 16384, 2048, 3), (32, 5120, 5120, 3), (33, 8192, 9728, 3), (64, 27648, 5120, 3), (40, 8192, 256, 3),
    (100, 8192, 512, 3), (200, 8192, 512, 20), (300, 8192, 512, 3), (512, 5120, 5120, 8),
    (520, 4160, 9792, 5), (520, 8192, 4864, 20), (1100, 27648, 2112, 3), (300, 1216, 19456, 8),
]


@pytest.mark.parametrize("M,N,K,n", SUMS, ids=["-".join(map(str, s)) for s in SUMS])
def test_an_fp32_gradient_s_long_sums_round(ops, M, N, K, n):  # noqa: F811
    """Root mean square error of an fp32 dX relative to its values'.

    The tensor cores cut off, at each of the L = 72 products of 16 after which the sum moves on, less than 2^-23 of the sum
    so far, half of it on average, in units that are 0.72 (1 / (2 ln 2)) of that: 0.36 2^-23 of a sum that grows like the
    square root of its length, all in one direction while the sum keeps its sign: 0.36 (2 / 3) L 2^-23 = 2.1e-6 at most.
    The additions that follow round by 2^-24 of what they hold, in no fixed direction, N / 1152 of them: 2^-24 sqrt(N /
    1152).  The adapter term, which is a hundredth of dX here, adds 2^-16 of itself at most: 2^-22.  (Sums left to the
    accumulator as a whole were 4.9e-6 off at N = 5120, and 1.3e-5 at 27648.)"""
    c = Case(ops, M, N, K, n, "random", mask=True, seed=M + 1)
    c.A.mul_(0.2)
    U = torch.zeros(M, 16, device=dev())
    go = lambda **kw: ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, **kw)
    dX = go(dX_f32=True)[0]
    a, has = c.own()
    G = torch.stack([c.dY[i].double() @ c.B[a[i]].double() for i in range(M)]) * has * c.scale.double()[a][:, None]
    want = c.dY.double() @ c.weight()
    for h in range(n):
        o = (a == h).nonzero()[:, 0]
        want[o] += c.keep()[o] * (G[o] @ c.A[h].double())
    tol = 0.36 * (2 / 3) * 72 * 2.0 ** -23 + 2.0 ** -24 * (N / 1152) ** 0.5 + 2.0 ** -22
    off = float((dX.double() - want).norm() / want.norm())
    assert off <= tol, (off, tol)
    assert torch.equal(dX, go(dX_f32=True)[0])
    old = torch.randn_like(dX)
    add = old.clone()
    go(dX=add, accumulate=True)
    assert torch.equal(add, old + dX)
    # the same in bf16, whose sums need no such care: one rounding, of a value off by no more than 2e-5 of the largest
    d16 = go()[0].double()
    assert ((d16 - want).abs() <= 2.0 ** -8 * want.abs() + 2e-5 * want.abs().max()).all()
    assert ops.device_error() == 0


@pytest.mark.parametrize("M,N,K,n", [(1, 5120, 5120, 2), (16, 448, 640, 20), (40, 9728, 2112, 3), (64, 8256, 9728, 9), (90, 448, 640, 9),
                                     (200, 9728, 8256, 3), (300, 2112, 1088, 12), (520, 4160, 9792, 5), (700, 9792, 4160, 10)])
def test_a_workspace_of_the_stated_size_is_enough(ops, M, N, K, n):  # noqa: F811
    """Nothing is written behind it, and nothing of y, U, dX and the gradients goes elsewhere than in them."""
    c = Case(ops, M, N, K, n, "random", mask=True, seed=M)
    size, room = ops.lora_multi_workspace_size(M, N, K, n), 1 << 20
    kept = []

    def guarded(shape, dtype):
        k = 1
        for d in shape:
            k *= d
        buf = torch.empty(k + room, dtype=dtype, device=dev())
        buf.view(torch.uint8).fill_(0xA5)
        kept.append((buf, k))
        return buf[:k].view(shape)
    ws = guarded((size,), torch.uint8)
    y, U = guarded((M, N), torch.bfloat16), guarded((M, 16), torch.float32)
    dA, dB = guarded((n, 16, K), torch.float32), guarded((n, N, 16), torch.float32)
    f = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask, y=y, U=U, workspace=ws)
    for dtype in (torch.float32, torch.bfloat16):
        dX = guarded((M, K), dtype)
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX=dX, dA=dA, dB=dB, workspace=ws)
        want = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=dtype == torch.float32)
        assert all(torch.equal(p, q) for p, q in zip((dX, dA, dB), want))
    assert all(torch.equal(p, q) for p, q in zip(f, ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)))
    for buf, k in kept:
        assert (buf[k:].view(torch.uint8) == 0xA5).all()
    assert ops.device_error() == 0
