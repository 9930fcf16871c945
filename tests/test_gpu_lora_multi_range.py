"""The many-adapter linear over its whole range: each form of its kernels, long sums, many rows and adapters, offsets past
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
