"""Every wait on a barrier in the kernels' sources gives up by the clock, and in every lane that goes on the phase was seen
complete (the sources are read as text: no wait is made to run out here)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_streaming_nf4_gb300", "csrc")


def functions(text):
    """(name, body) of the device functions: WS_DEVINL ... name(...) {...} at the beginning of a line."""
    for m in re.finditer(r"^WS_DEVINL [\w:<>\*& ]*?(\w+)\(", text, re.M):
        at = text.index("{", m.end())
        depth = 0
        for i in range(at, len(text)):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            if depth == 0:
                yield m.group(1), text[at:i + 1]
                break


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


@pytest.mark.parametrize("name", sources())
def test_waits_are_bounded_by_the_clock(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    inside = 0
    for fn, body in functions(text):
        n = body.count("mbar_try_wait(")
        if n and re.search(r"\b(for|while)\b", body):
            # the clock against the limit, in the function itself or through the limit that it keeps
            assert "kWaitLimitNs" in body or "limit.over(" in body, (name, fn)
        inside += n
    for m in re.finditer(r"struct WaitLimit \{(.*?)\n\};", text, re.S):
        assert "globaltimer()" in m.group(1) and "kWaitLimitNs" in m.group(1)
    # no loop of a kernel's own around the bare poll
    assert text.count("mbar_try_wait(") - inside - text.count("bool mbar_try_wait(") == 0
    # a vote orders no memory: one lane's success is not the others'
    assert not re.search(r"__any_sync\([^;]*mbar_try_wait", text)
