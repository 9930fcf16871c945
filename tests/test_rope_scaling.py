"""Frequencies for longer contexts, from the definitions with other arithmetic and against numbers worked out apart, and the
refusals of calls that leave out or misname the stretch (host only)."""
import math
from decimal import Decimal, getcontext

import pytest

getcontext().prec = 40
PI = Decimal("3.141592653589793238462643383279502884197")


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import build
    build.build()
    from weight_streaming_nf4_gb300 import ops as o
    return o


def yarn(rot, base, s, original, fast, slow):
    """Frequencies by the definition of "by parts" interpolation (Peng et al., 2023), in 40 digits: pair i turns
    base^(-2 i / rot) radians a position, so often within `original` positions; between the pairs (as whole numbers, outwards)
    that turn `fast` and `slow` times, a ramp leads from the frequency itself to an s-th of it."""
    b, half = Decimal(base), rot // 2

    def pair(turns):  # original base^(-2 i / rot) = 2 pi turns
        return (Decimal(original) / (2 * PI * Decimal(turns))).ln() / b.ln() * rot / 2
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    out = []
    for i in range(half):
        f = (-Decimal(2 * i) / rot * b.ln()).exp()
        r = Decimal(0) if i <= lo else Decimal(1) if i >= hi else Decimal(i - lo) / (hi - lo)
        out.append(f * (1 - r) + f * r / Decimal(s))
    return [float(x) for x in out]


CASES = [(128, 1e6, 4.0, 32768, 32.0, 1.0), (64, 1e4, 4.0, 2048, 32.0, 1.0), (128, 1e4, 16.0, 4096, 32.0, 1.0), (128, 5e5, 8.0, 8192, 4.0, 1.0),
         (16, 1e4, 2.0, 1024, 64.0, 2.0), (96, 1e6, 40.0, 4096, 32.0, 1.0), (128, 1e7, 1.0, 262144, 32.0, 1.0)]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_yarn(ops, case):
    rot, base, s, original, fast, slow = case
    got, amplitude = ops.rope_frequencies(rot, base=base, scaling="yarn", scale=s, original=original, beta_fast=fast, beta_slow=slow)
    want = yarn(*case)
    # a power (its argument at most 2 ln base < 33 long, rounded) and a few operations in 64 bits
    assert all(abs(a - b) <= 2.0 ** -46 * b for a, b in zip(got, want)) and len(got) == rot // 2
    assert abs(amplitude - float(Decimal(s).ln() / 10 + 1)) <= 2.0 ** -50
    r = ops.rope(rot, base=base, scaling="yarn", scale=s, original=original, beta_fast=fast, beta_slow=slow, device="cpu")
    assert r.factor == amplitude and r.turns.tolist() == ops.rope(rot, inv_freq=got, device="cpu").turns.tolist()


def test_yarn_s_ramp_by_hand(ops):
    """64 elements, base 10^4, 2048 positions: pair i turns 2048 10^(-i/8) / 2 pi times, 32 times for i = 8.065 and once for
    i = 20.107, so the ramp leads from pair 8 to pair 21."""
    f, _ = ops.rope_frequencies(64, base=1e4, scaling="yarn", scale=4.0, original=2048)
    for i, share in ((0, 1.0), (8, 1.0), (9, 1 - 0.75 / 13), (14, 1 - 0.75 * 6 / 13), (20, 1 - 0.75 * 12 / 13), (21, 0.25), (31, 0.25)):
        assert math.isclose(f[i], 10.0 ** (-i / 8) * share, rel_tol=1e-13)


def test_linear_and_ntk(ops):
    for s in (1.0, 2.0, 8.0, 3.5):
        f, a = ops.rope_frequencies(128, base=1e4, scaling="linear", scale=s)
        assert a == 1.0 and all(math.isclose(x, float(Decimal(10) ** (-Decimal(i) / 16) / Decimal(s)), rel_tol=1e-13) for i, x in enumerate(f))
        f, a = ops.rope_frequencies(128, base=1e4, scaling="ntk", scale=s)
        # base' = base s^(rot / (rot - 2)): pair i turns s^(-i / 63) times as fast
        assert a == 1.0 and all(math.isclose(x, 10.0 ** (-i / 16) * s ** (-i / 63), rel_tol=1e-13) for i, x in enumerate(f))


def test_the_stretch_has_one_name_and_is_not_left_out(ops):
    assert ops.rope_frequencies(64, scaling="linear", scale=4.0) == ops.rope_frequencies(64, scaling="linear", factor=4.0)
    assert ops.rope(64, scaling="yarn", scale=4.0, original=2048, attention_factor=1.25, device="cpu").factor == 1.25
    assert ops.rope(64, attention_factor=1.25, device="cpu").factor == 1.25
    for given in (dict(factor=1.5), dict(attention_factor=1.5)):
        assert ops.rope(16, inv_freq=[1.0] * 8, device="cpu", **given).factor == 1.5
    for bad in (dict(scaling="linear"), dict(scaling="ntk"), dict(scaling="yarn", original=2048),    # no stretch
                dict(scaling="linear", factor=8.0), dict(scaling="yarn", factor=4.0, original=2048),  # not its name in rope()
                dict(factor=8.0), dict(scale=4.0),                                                    # of nothing
                dict(scaling="linear", scale=4.0, factor=1.0), dict(inv_freq=[1.0] * 32, scale=4.0),
                dict(inv_freq=[1.0] * 32, factor=2.0, attention_factor=2.0), dict(inv_freq=[1.0] * 32, original=2048),
                dict(scaling="linear", scale=0.5), dict(scaling="linear", scale=math.nan), dict(attention_factor=math.inf)):
        with pytest.raises(ValueError):
            ops.rope(64, device="cpu", **bad)
    for bad in (dict(scaling="linear"), dict(scaling="yarn", original=2048), dict(scale=4.0), dict(factor=4.0),
                dict(scaling="linear", scale=4.0, factor=4.0)):
        with pytest.raises(ValueError):
            ops.rope_frequencies(64, **bad)
