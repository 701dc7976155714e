"""The bounded waits of warps that stay together are decided by the whole warp (read from the sources: the answer differs
between lanes only when a time limit expires while the barrier flips, which no test brings about)."""

import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "exact_tiled_attention_41_b200", "csrc")


def waits(name):
    """Every wait that answers lane by lane, as (line index, text), and all lines without their comments."""
    src = open(os.path.join(CSRC, name)).read()
    lines = re.sub(r"//[^\n]*", "", src).split("\n")
    return [(n, line) for n, line in enumerate(lines) if re.search(r"\bmbar_wait\(", line)], lines


def one_lane(lines, n):
    """The wait lies inside a block that only lane 0 (or thread 0) enters."""
    depth = 0
    for line in reversed(lines[:n]):
        for ch in reversed(line):
            depth += (ch == "}") - (ch == "{")
            if depth < 0 and ch == "{":
                if re.search(r"if \((WARP \|\| )?(lane|threadIdx\.x) == 0\)", line):
                    return "WARP" not in line
                depth = 0
    return False


def voted(lines, n):
    """The answer goes through a vote of the warp before anything depends on it."""
    text = " ".join(lines[n:n + 5])
    if "__all_sync(0xffffffffu, mbar_wait(" in lines[n]:
        return True
    m = re.search(r"\b(got|ok) = ", lines[n])
    return bool(m) and re.search(r"__all_sync\(0xffffffffu, %s\)" % m.group(1), text) is not None


@pytest.mark.parametrize("name", ["fwd.cu", "bwd.cu", "bwd256.cu", "bwd_dq.cu", "decode.cu"])
def test_waits_of_whole_warps_are_voted(name):
    found, lines = waits(name)
    assert found
    alone = [f"{name}:{n + 1}: {line.strip()}" for n, line in found if not one_lane(lines, n) and not voted(lines, n)]
    assert not alone, "\n".join(alone)


def test_the_unit_feed_votes_for_whole_warps():
    src = open(os.path.join(CSRC, "sm100.cuh")).read()
    body = src[src.index("bool feed_get("):]
    assert "whole_warp ? mbar_wait_warp(" in body[:body.index("\n}\n")]
    body = src[src.index("bool mbar_wait_warp("):]
    assert "__all_sync(0xffffffffu, mbar_wait(bar, parity, w))" in body[:body.index("\n}\n")]


@pytest.mark.parametrize("name", ["fwd.cu", "bwd.cu", "bwd256.cu", "bwd_dq.cu", "sm100.cuh"])
def test_no_wait_without_a_limit_between_warps_that_may_give_up(name):
    # a warp that has given up does not come to a hardware barrier, and the others would stay there for good; the barriers
    # of the whole block (__syncthreads) stand where every role arrives, whatever became of it
    src = open(os.path.join(CSRC, name)).read()
    assert not re.search(r"bar\.sync|barrier\.sync|named_bar", re.sub(r"//[^\n]*", "", src))
