"""Waits of converged warps, read from the sources without a GPU.  A bounded wait
polls and gives up lane by lane.  Where the whole warp waits, its lanes have to
agree on the result before the next instruction that takes all 32 of them: a
lane that gave up alone would leave the others waiting for it without a limit."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rmsnorm_linear_projection_gb300", "csrc")


def waits(text):
    """(line, what the warp does with the result) of each mbar_wait and flag_wait call."""
    text = re.sub(r"//[^\n]*", "", text)
    text = re.sub(r"\bfor \([^;{}]*;[^;{}]*;", lambda m: m.group().replace(";", ","), text)  # a loop's head ends no statement
    for m in re.finditer(r"\b(?:mbar_wait|flag_wait)\(", text):
        # the statement that holds the call, and the two behind it
        start = max(text.rfind(c, 0, m.start()) for c in ";{}") + 1
        end = m.end()
        for _ in range(3):
            end = text.index(";", end) + 1
        yield text.count("\n", 0, m.start()) + 1, text[:start], text[start:end]


def one_lane(before):
    """Whether the innermost open blocks are a single lane's."""
    depth = 0
    for m in re.finditer(r"[{}]", before[::-1]):
        depth += 1 if m.group() == "{" else -1
        if depth > 0:
            at = len(before) - 1 - m.start()
            head = before[max(before.rfind(c, 0, at) for c in ";{}") + 1:at]
            if re.search(r"if \((?:lane == 0|elect_one\(\))\)", head):
                return True
            depth = 0
    return False


@pytest.mark.parametrize("name", ["grouped.cu"])
def test_lanes_agree_on_every_wait(name):
    found = list(waits(open(os.path.join(CSRC, name)).read()))
    assert len(found) >= 10
    alone = [line for line, before, behind in found if "__all_sync" not in behind and not one_lane(before)]
    assert not alone, f"{name}: waits whose result differs from lane to lane, lines {alone}"
