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
