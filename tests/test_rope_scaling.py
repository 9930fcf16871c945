"""Rotary positions for longer contexts: refusals of calls that leave out or misname the stretch (host only)."""
import math

import pytest


@pytest.fixture(scope="module")
def ops():
    from weight_streaming_nf4_gb300 import build
    build.build()
    from weight_streaming_nf4_gb300 import ops as o
    return o


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
