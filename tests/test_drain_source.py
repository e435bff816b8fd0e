"""Source checks of how TMA producers end (no GPU).

A producer's last loads may still be on their way when its loop ends.  Normally its
consumers wait for them, but consumers that gave up after an error elsewhere in the
grid do not, and a load must not land in the shared memory of a CTA that has gone.
So every producer waits for its rings behind its loop, with or without an error:
a statement at the loop's own depth, under no condition but a pair's even and odd CTA.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_tensor_core_02_gb300",
                    "csrc")
# file -> barriers that its producers arm for their loads, in the order of the source
RINGS = {
    "gemm_kernel.cuh": ["full", "full8"],
    "gemm2sm_kernel.cuh": ["full"],
    "conv_halo_kernel.cuh": ["full", "hfull"],
    "few_tokens.cu": ["full"],
    "i8_tokens.cu": ["full"],
    "grouped_pair.cu": ["fix", "full"],
}


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def enclosing(text, at):
    """Heads of the blocks that position `at` lies in, innermost first."""
    heads, depth = [], 0
    for i in range(at - 1, -1, -1):
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth == 0:
                start = max(text.rfind(c, 0, i) for c in ";{}")
                heads.append(" ".join(text[start + 1:i].split()))
            else:
                depth -= 1
    return heads


def test_every_file_with_producers_is_listed():
    found = {n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")) and "mbar_arrive_expect_tx(&" in source(n)}
    assert found == set(RINGS)


@pytest.mark.parametrize("name", sorted(RINGS))
def test_producers_wait_for_their_loads(name):
    text = source(name)
    armed = {m.group(1) for m in re.finditer(r"mbar_arrive_expect_tx\(&(\w+)\[", text)}
    assert armed == set(RINGS[name])
    calls = list(re.finditer(r"\bdrain_ring(?:_lanes)?\(\s*(\w+)\s*,", text))
    calls = [c for c in calls if c.group(1) in armed]
    assert [c.group(1) for c in calls] == RINGS[name]
    for c in calls:
        # the block it lies in is the producer's (or the pair's even CTA's), no loop and no error path
        heads = enclosing(text, c.start())
        if "leader" in heads[0]:
            heads = heads[1:]
        assert re.search(r"\(lane == 0\)|^if \(warp == 0\)$", heads[0]), heads[0]
        before = text[:c.start()].rstrip()
        assert not before.endswith(")") or before.endswith("if (leader)"), before[-40:]
    assert not re.search(r"if \(!ok[^{;]*\{?\s*(for[^{;]*;[^{;]*;[^{)]*\)\s*)?(if[^;{]*)?drain_", text)


@pytest.mark.parametrize("name", ["gemm2sm_kernel.cuh", "conv_halo_kernel.cuh", "grouped_pair.cu"])
def test_odd_ctas_of_pairs(name):
    """Their loads complete on the even CTA's barriers."""
    assert len(re.findall(r"else\s*\{?\s*drain_odd_cta\(wc\);", source(name))) == 1


def test_a_stage_to_be_cleared_is_not_waited_for_on_full():
    """Its `full` completes by the clearing warps, in a phase that the producer did not arm."""
    text = source("grouped_pair.cu")
    clear = text[text.index("if (clear) {"):]
    assert "armed &= ~(1u << stage);" in clear[:clear.index("}")]
