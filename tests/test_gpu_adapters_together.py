"""Adapters trained side by side and then served: forward, backward, clipping and
AdamW of three adapters on one frozen NF4 weight, each step checked against the
formulas in 64 bits from the state the step found; then the trained adapters
answer single rows and a mixed batch."""
import pytest
import torch

from gpu_util import dev
from test_gpu_lora_multi import Case, check_backward, check_forward, ops  # noqa: F401

pytestmark = pytest.mark.gpu


class Pool:
    """Three adapters' A and B in one array each, as a training program keeps them."""

    def __init__(self, ops, c, bits):
        self.A, self.B = c.A, c.B
        self.dA, self.dB = torch.zeros_like(c.A), torch.zeros_like(c.B)
        tensors = [t for x in (c.A, c.B) for t in x]
        grads = [t for x in (self.dA, self.dB) for t in x]
        if bits == 32:
            self.m, self.v = ([torch.zeros_like(t) for t in tensors] for _ in range(2))
            kw = {}
        else:
            self.m, self.v = ([torch.zeros(t.numel(), dtype=torch.uint8, device=dev()) for t in tensors] for _ in range(2))
            sc = lambda: [torch.zeros(-(-t.numel() // 256), device=dev()) for t in tensors]
            kw = dict(exp_avg_scales=sc(), exp_avg_sq_scales=sc())
        n = c.A.shape[0]
        self.lr = [1e-3 * (i + 1) for i in range(n)]
        self.groups = ops.adamw_groups([dict(lr=l, weight_decay=0.05, max_norm=0.3) for l in self.lr])
        self.plan = ops.adamw_plan(tensors, grads, self.m, self.v, groups=list(range(n)) * 2, **kw)


@pytest.mark.parametrize("bits", [32, 8])
def test_train_then_serve(ops, bits):  # noqa: F811
    M, N, K, n = 150, 192, 256, 3
    c = Case(ops, M, N, K, n, "random", mask=True, seed=21)
    pool = Pool(ops, c, bits)
    target = torch.randn(M, N, generator=torch.Generator().manual_seed(2)).to(dev())
    norms = torch.zeros(n, device=dev())
    for step in range(1, 4):
        y, U = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan, mask=c.mask)
        check_forward(c, y, U)
        c.dY = ((y.float() - target) / M).bfloat16()
        dX, _, _ = ops.lora_linear_bwd_multi(c.W, c.x, c.set, c.plan, U, c.dY, mask=c.mask, dX_f32=True,
                                             dA=pool.dA, dB=pool.dB)
        check_backward(c, U, dX, pool.dA, pool.dB)
        before = c.A.double().clone(), c.B.double().clone()
        ops.adamw_step(pool.plan, pool.groups, norms=norms, clip=True)
        assert pool.groups[:, 6].tolist() == [step] * n
        for i in range(n):
            g = torch.cat([pool.dA[i].reshape(-1), pool.dB[i].reshape(-1)]).double()
            assert abs(float(norms[i]) - float(g.norm())) <= 2.0 ** -18 * float(g.norm())
            clip = min(1.0, 0.3 / (float(g.norm()) + 1e-6))
            for p0, p1, gr in ((before[0][i], c.A[i], pool.dA[i]), (before[1][i], c.B[i], pool.dB[i])):
                moved = p1.double() - p0 * (1 - pool.lr[i] * 0.05)
                assert torch.isfinite(moved).all()
                if step == 1:   # from zero states the step is lr g / (|g| + eps)
                    gc = gr.double() * clip
                    want = -pool.lr[i] * gc / (gc.abs() + 1e-8)
                    assert ((moved - want).abs() <= 2.0 ** -17 * pool.lr[i] + 2.0 ** -22 * p0.abs()).all()
    # served: each row alone, and eight of them in another order with none between, as in the batch
    y, U = ops.lora_linear_fwd_multi(c.W, c.x, c.set, c.plan)
    served = Case(ops, M, N, K, n, "random", seed=21)
    served.A, served.B, served.set = c.A, c.B, c.set
    check_forward(served, y, U)
    for rows in ([3], [149], [5, 0, 77, 40, 41, 8, 100, 9]):
        r = torch.tensor(rows)
        ids = c.rows[r].clone()
        if len(rows) > 1:
            ids[2] = -1
        p = ops.lora_multi_plan(ids.to(dev()), n)
        y1, _ = ops.lora_linear_fwd_multi(c.W, c.x[r.to(dev())].contiguous(), c.set, p)
        one = Case(ops, M, N, K, n, "random", seed=21)
        one.M, one.rows, one.x = len(rows), ids, c.x[r.to(dev())]
        one.A, one.B, one.set = c.A, c.B, c.set
        ref = one.forward()
        tol = 2.0 ** -8 * ref["y"].abs() + (K / 16 + 80) * 2.0 ** -23 * ref["Sy"] + 2.0 ** -14 * ref["Slora"]
        assert ((y1.double() - ref["y"]).abs() <= tol + 1e-30).all()
    assert ops.device_error() == 0
