"""The many-adapter linear on the 256-column tiles of its GEMM, which weights of this size and more than 128 rows (forward)
or 256 (backward) get: one CTA and pairs, tiles cut between them or ranges that leave steps out at a tile's end, adapters
in slots, a slot for each of eight, and more than slots; against the formulas in 64 bits."""
import pytest
import torch

from gpu_util import dev
from test_gpu_lora_multi import Case, check_backward, check_forward, ops  # noqa: F401

pytestmark = pytest.mark.gpu
F, BF = torch.float32, torch.bfloat16


def fresh(c, ops):  # noqa: F811
    """Outputs and workspace full of NaN."""
    ws = torch.full((ops.lora_multi_workspace_size(c.M, c.N, c.K, c.n),), 255, dtype=torch.uint8, device=dev())
    return torch.full((c.M, c.N), float("nan"), dtype=BF, device=dev()), torch.full((c.M, 16), float("nan"), device=dev()), ws


FORWARD = [
    # M, N, K, adapters, rows, adapter type, mask
    (200, 9728, 8256, 5, "random", F, True),        # one CTA, cut tiles
    (129, 9728, 8256, 8, "distinct", BF, False),
    (256, 9792, 8256, 30, "random", F, True),       # more than slots
    (200, 38976, 2112, 1, "one", BF, True),         # a tile or more for every SM
    (250, 38976, 2112, 8, "random", F, False),
    (520, 4864, 4160, 5, "random", F, True),        # pairs, cut tiles
    (520, 9792, 2112, 8, "distinct", BF, True),     # pairs, a tile or more each
    (520, 9792, 2112, 9, "distinct", F, False),     # one adapter more than slots
    (520, 9792, 2112, 6, "none", F, True),
    (1100, 9728, 8256, 8, "random", F, False),
    (1100, 9728, 8256, 40, "wild", BF, True),
]


@pytest.mark.parametrize("M,N,K,n,kind,dtype,mask", FORWARD, ids=["-".join(map(str, s[:5])) for s in FORWARD])
def test_forward(ops, M, N, K, n, kind, dtype, mask):  # noqa: F811
    c = Case(ops, M, N, K, n, kind, dtype, mask, seed=M + n, pool=24 if dtype == F else 0)
    y, U, ws = fresh(c, ops)
    for _ in range(2):   # the same workspace again
        y.fill_(float("nan"))
        ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask, y=y, U=U, workspace=ws)
        check_forward(c, y, U)
    assert ops.device_error() == 0


BACKWARD = [
    # M, N, K, adapters, rows, dX fp32, mask
    (520, 4160, 4864, 5, "random", True, True),     # cut tiles
    (520, 2112, 9792, 8, "distinct", False, True),  # a tile or more for every pair
    (520, 2112, 9792, 8, "random", True, False),
    (520, 2112, 9792, 9, "distinct", True, True),   # one adapter more than slots
    (300, 4160, 9728, 1, "one", True, True),
    (1100, 8256, 9728, 8, "random", True, True),
    (1100, 4160, 9792, 40, "wild", False, False),
]


@pytest.mark.parametrize("M,N,K,n,kind,f32,mask", BACKWARD, ids=["-".join(map(str, s[:5])) for s in BACKWARD])
def test_backward(ops, M, N, K, n, kind, f32, mask):  # noqa: F811
    c = Case(ops, M, N, K, n, kind, F, mask, seed=M + n, pool=16)
    U = c.forward()["U"].float()
    _, _, ws = fresh(c, ops)
    dX = torch.full((M, K), float("nan"), dtype=F if f32 else BF, device=dev())
    dA, dB = c.set.empty_grads()
    for _ in range(2):
        for t in (dX, dA, dB):
            t.fill_(float("nan"))
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX=dX, dA=dA, dB=dB, workspace=ws)
        check_backward(c, U, dX, dA, dB)
    if f32:   # added into what is there: one fp32 addition each
        oX, oA, oB = (torch.randn_like(t) for t in (dX, dA, dB))
        aX, (aA, aB) = oX.clone(), c.set.empty_grads()
        aA.copy_(oA), aB.copy_(oB)
        ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX=aX, dA=aA, dB=aB, workspace=ws,
                                  accumulate=True, grad_accumulate=True)
        assert torch.equal(aX, oX + dX) and torch.equal(aA, oA + dA) and torch.equal(aB, oB + dB)
    assert ops.device_error() == 0


@pytest.mark.parametrize("M,N,K,n", [(200, 9728, 8256, 8), (520, 9792, 2112, 5), (520, 4864, 4160, 20)])
def test_a_diverged_adapter_stays_alone(ops, M, N, K, n):  # noqa: F811
    """NaN and infinities in the factors of one adapter reach its own rows only, and there the formula's columns."""
    c = Case(ops, M, N, K, n, "random", mask=True, seed=M)
    own = (c.rows == 1).to(dev())
    U = c.forward()["U"].float()
    y0, _ = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)
    g0 = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=True)
    c.B[1, 5, 3], c.B[1, N - 1, :] = float("nan"), float("inf")
    y1, _ = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)
    cols = torch.ones(N, dtype=torch.bool, device=dev())
    cols[5] = cols[N - 1] = False
    assert torch.equal(y1[~own], y0[~own]) and torch.equal(y1[:, cols], y0[:, cols])
    assert not torch.isfinite(y1[own][:, ~cols]).any()
    c.B[1, 5, 3], c.B[1, N - 1, :] = 0.5, 0.5
    c.A[1, 2, 70] = float("-inf")
    g1 = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=True)
    kept = own & ((c.mask[:, 2] >> 6) & 1).bool()   # rows of the adapter that keep element 70
    assert not torch.isfinite(g1[0][kept][:, 70]).any() and torch.isfinite(g1[0][~kept]).all()
    assert torch.equal(g1[0][~own], g0[0][~own])
    assert ops.device_error() == 0
