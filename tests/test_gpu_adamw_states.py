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
