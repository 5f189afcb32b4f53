"""Waits that give up, read from the kernels' sources.  A wait's time limit is each lane's own.
A warp whose lanes go on together (named barriers count whole warps, tensor-memory loads and
cluster barriers are warp-wide) has to give up as one: mbar_wait_warp.  Only the one lane of a
role that has no others may use mbar_wait, and its warp meets again before a cluster barrier.
A timeout cannot be made on purpose here without copies in flight, so this is checked as text.
"""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "long_context_hs2_b200", "csrc")


def blocks(text):
    """(position, headers of the enclosing braces) of every word of the text."""
    stack, start = [], 0
    for m in re.finditer(r"[{};]|\w+(?=\s*\()", text):
        if m.group() == "{":
            stack.append(text[start:m.start()])
        elif m.group() == "}":
            stack.pop()
        elif m.group() != ";":
            yield m.group(), m.start(), list(stack)
            continue
        start = m.end()


@pytest.mark.parametrize("name", ["fp8_gemm.cuh", "bridge_gemm.cuh", "bridge_small.cuh"])
def test_warps_give_up_as_one(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    waits = 0
    for word, at, around in blocks(text):
        line = text.count("\n", 0, at) + 1
        alone = any("lane == 0" in h for h in around)
        if word in ("mbar_wait", "mbar_wait_warp"):
            waits += 1
            assert alone == (word == "mbar_wait"), "%s:%d" % (name, line)
        if word == "cluster_wait_acquire":
            before = text[:at].rstrip().rsplit(";", 2)[-2].split("}")[-1].strip()
            assert before in ("__syncwarp()", "cluster_arrive_release()"), "%s:%d" % (name, line)
    assert waits > 0
