"""The operators between the projections and the next layer, run as they are used: training (projections of several
adapters, norm and rotation, the causal core, and back), and serving from the 8-bit cache (prompts in chunks, single
tokens, proposed tokens taken back), each step against 64-bit forms of the definition."""
import math

import pytest
import torch

from test_gpu_kv import PAGE, Model, attention, empty_cache, ints, starts

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, NH, NKV, HD, EPS = 512, 6, 2, 64, 1e-6


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import ops as o
    return o


def _layer(ops, seed, n_adapters):
    """Frozen NF4 projections q, k, v with adapters each, and the gains."""
    g = torch.Generator().manual_seed(seed)
    out = {}
    for name, n in (("q", NH * HD), ("k", NKV * HD), ("v", NKV * HD)):
        w = (torch.randn(n, H, generator=g) * 0.05).bfloat16().to(DEV)
        A = (torch.rand(n_adapters, 16, H, generator=g) * 2 - 1).to(DEV) / math.sqrt(H)
        B = torch.randn(n_adapters, n, 16, generator=g).to(DEV) * 0.05
        out[name] = (ops.NF4Weight(*ops.quantize_nf4(w), n, H), ops.LoraSet(A, B, torch.full((n_adapters,), 2.0, device=DEV)))
    out["gq"], out["gk"] = ((1 + 0.2 * torch.randn(HD, generator=g)).to(DEV) for _ in range(2))
    return out


def _project(ops, layer, x, plan):
    return [ops.lora_linear_fwd_multi(layer[n][0], x, layer[n][1], plan) for n in "qkv"]


def _turned(x, gain, pos, freq, hd=HD):
    """Norm and rotation (half layout, the whole head) in 64 bits."""
    x = x.reshape(x.shape[0], -1, hd)
    n = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * gain
    a = pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=DEV)
    c, s, r = a.cos()[:, None], a.sin()[:, None], hd // 2
    return torch.cat([n[..., :r] * c - n[..., r:] * s, n[..., :r] * s + n[..., r:] * c], -1)


def _core(q, k, v, n_seq):
    """Causal attention of n_seq sequences, [M, heads, hd] each, in 64 bits."""
    M = q.shape[0]
    S, G = M // n_seq, q.shape[1] // k.shape[1]
    q, k, v = (t.view(n_seq, S, -1, HD).transpose(1, 2) for t in (q, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)))
    s = (q @ k.transpose(2, 3) / math.sqrt(HD)).masked_fill(torch.ones(S, S, device=DEV).triu(1).bool(), -math.inf)
    return (torch.softmax(s, -1) @ v).transpose(1, 2).reshape(M, -1)


def test_training_forward_and_backward(ops):
    """x -> q, k, v of three adapters -> norm and rotation -> attention, and the gradients down to the adapters' own."""
    n_seq, S = 3, 130
    M = n_seq * S
    layer = _layer(ops, 1, 3)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(M, H, generator=g).bfloat16().to(DEV)
    plan = ops.lora_multi_plan(torch.arange(n_seq, dtype=torch.int32).repeat_interleave(S).to(DEV), 3)
    freq, _ = ops.rope_frequencies(HD, base=1e4)
    rope, pos = ops.rope(HD, base=1e4), torch.arange(S, dtype=torch.int32).repeat(n_seq).to(DEV)
    (q, Uq), (k, Uk), (v, Uv) = _project(ops, layer, x, plan)
    qr, kr = ops.qk_norm_rope_fwd(q, k, HD, rope, pos, q_gain=layer["gq"], k_gain=layer["gk"], eps=EPS)
    o, o32, lse = ops.attention_fwd(qr, kr, v, n_seq, HD)
    dO = torch.randn(M, NH * HD, generator=g).bfloat16().to(DEV)
    dqr, dkr, dv = ops.attention_bwd(qr, kr, v, o32, lse, dO, n_seq, HD)
    dq, dk, dgq, dgk = ops.qk_norm_rope_bwd(q, k, dqr, dkr, HD, rope, pos, q_gain=layer["gq"], k_gain=layer["gk"], eps=EPS)
    back = [ops.lora_linear_bwd_multi(layer[n][0], x, layer[n][1], plan, U, d) for n, U, d in (("q", Uq, dq), ("k", Uk, dk), ("v", Uv, dv))]
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    # 64 bits from the projections' outputs on; the rotated rows and their gradients are rounded to bf16 on the way, each
    # 2^-8 / sqrt(3) of a value at most in the mean: four of them stay below 1e-2
    leaf = [t.double().requires_grad_() for t in (q, k, v, layer["gq"], layer["gk"])]
    ref = _core(_turned(leaf[0], leaf[3], pos, freq), _turned(leaf[1], leaf[4], pos, freq), leaf[2].view(M, NKV, HD), n_seq)
    ref.backward(dO.double())
    for got, want in [(o, ref.detach())] + list(zip((dq, dk, dv, dgq, dgk), (t.grad for t in leaf))):
        assert (got.double().view_as(want) - want).norm() <= 1e-2 * want.norm()
    # the adapters' gradients from those rows: dB of one adapter
    for (dX, dA, dB), U, d, n in zip(back, (Uq, Uk, Uv), (dq, dk, dv), "qkv"):
        for a in range(3):
            rows = slice(a * S, (a + 1) * S)
            want = 2.0 * d[rows].double().t() @ U[rows].double()
            assert (dB[a].double() - want).norm() <= 2e-3 * want.norm()


def test_serving_from_the_cache(ops):
    """Two layers' caches under one plan a step.  Sequences join, grow in chunks and single tokens, share a prompt's full
    pages, and take proposed tokens back; every step's attention is checked, and the cache at the end."""
    layers = [_layer(ops, 10 + i, 2) for i in range(2)]
    n_pages, n_seq = 24, 4
    caches = [empty_cache(ops, n_pages, NKV, HD) for _ in layers]
    models = [Model(c) for c in caches]
    freq, _ = ops.rope_frequencies(HD, base=1e4)
    rope = ops.rope(HD, base=1e4)
    g = torch.Generator().manual_seed(5)
    past, table, free = [0] * n_seq, [[-1] * 6 for _ in range(n_seq)], list(range(n_pages))[::-1]
    adapter = [0, 1, -1, 1]
    steps = [  # new rows of each sequence, and how many tokens are taken back after it
        ([150, 0, 9, 0], None), ([1, 130, 1, 0], None), ([1, 1, 40, 0], None), ([4, 4, 4, 0], [3, 0, 2, 0]),
        ("fork", None), ([1, 1, 1, 1], None), ([2, 70, 1, 30], [1, 0, 0, 0]), ([1, 1, 1, 1], None)]
    for new, back in steps:
        if new == "fork":  # sequence 3 goes on from sequence 0's full pages
            past[3] = past[0] // PAGE * PAGE
            table[3][:past[0] // PAGE] = table[0][:past[0] // PAGE]
            continue
        for i, n in enumerate(new):
            for p in range(-(-(past[i] + n) // PAGE)):
                if table[i][p] < 0:
                    table[i][p] = free.pop()
        T = sum(new)
        row_adapter = torch.tensor([adapter[i] for i, n in enumerate(new) for _ in range(n)], dtype=torch.int32, device=DEV)
        pos = torch.tensor([past[i] + j for i, n in enumerate(new) for j in range(n)], dtype=torch.int32, device=DEV)
        lora = ops.lora_multi_plan(row_adapter, 2)
        plan = ops.kv_plan(ints(past), ints(starts(new)), ints(table), T, max(new), NH, NKV, HD)
        x = torch.randn(T, H, generator=g).bfloat16().to(DEV)
        for layer, cache, model in zip(layers, caches, models):
            (q, _), (k, _), (v, _) = _project(ops, layer, x, lora)
            raw = q.clone(), k.clone()
            ops.qk_norm_rope_fwd(q, k, HD, rope, pos, q_gain=layer["gq"], k_gain=layer["gk"], eps=EPS, q_out=q, k_out=k)
            for t, r, gain in ((q, raw[0], layer["gq"]), (k, raw[1], layer["gk"])):
                want = _turned(r.double(), gain.double(), pos, freq).reshape(T, -1)
                assert (t.double() - want).norm() <= 2e-3 * want.norm()
            ops.kv_append(cache, plan, k, v)
            o, lse = ops.attention_kv(q, cache, plan, want_lse=True)
            torch.cuda.synchronize()
            assert ops.device_error() == 0
            model.append(past, new, table, k, v)
            for ro, tol, rl, ltol, r0 in attention(model, past, new, table, q, NH // NKV, HD, HD ** -0.5):
                n = ro.shape[0]
                assert (o[r0:r0 + n].double().view(n, NH, HD) - ro).abs().le(tol).all()
                assert (lse.t()[r0:r0 + n].double() - rl).abs().le(ltol).all()
        past = [p + n - b for p, n, b in zip(past, new, back or [0] * n_seq)]
    for cache, model in zip(caches, models):
        model.check(cache)


def test_a_cache_filled_at_once_or_token_by_token(ops):
    """The same rows in one call, in chunks and one by one: the same scales, and the same codes but for roundings of values
    that were subnormal when their page's scale grew."""
    g = torch.Generator().manual_seed(9)
    T = 200
    k, v = ((torch.randn(T, NKV * HD, generator=g) * torch.rand(T, 1, generator=g) * 8).bfloat16().to(DEV) for _ in range(2))
    table = ints([[3, 0, 2, 1]])
    got = []
    for sizes in ([200], [64, 64, 72], [1] * 200, [63, 2, 100, 35]):
        cache = empty_cache(ops, 4, NKV, HD)
        at = 0
        for n in sizes:
            plan = ops.kv_plan(ints([at]), ints([0, n]), table, n, n, NH, NKV, HD)
            ops.kv_append(cache, plan, k[at:at + n], v[at:at + n])
            at += n
        s = cache.scale.double()
        # the last page's places behind the 200 tokens hold what they held
        values = [(cache.k.double() * s[:, :, 0, None, None])[[3, 0, 2, 1]].transpose(1, 2).reshape(256, NKV, HD)[:T],
                  (cache.v.double().transpose(2, 3) * s[:, :, 1, None, None])[[3, 0, 2, 1]].transpose(1, 2).reshape(256, NKV, HD)[:T]]
        got.append((cache.scale.clone(), values))
    for scale, values in got[1:]:
        assert torch.equal(scale, got[0][0])
        for i, (a, b) in enumerate(zip(values, got[0][1])):
            unit = 2.0 ** -9 * scale[:, :, i].double()[[3, 0, 2, 1]].repeat_interleave(PAGE, 0)[:T, :, None]  # a subnormal step
            assert ((a - b).abs() <= unit).all() and (a != b).double().mean() < 0.02
