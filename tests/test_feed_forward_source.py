"""Source checks of the gated and fp8 kernels (no GPU): they wait for the previous grid before
they first reach global memory, and their TMA producers wait for their last loads."""
import re

import pytest

from test_drain_source import enclosing, source
from test_pdl_source import _kernel_body, _pdl_launched_kernels, _sources

KERNELS = {"f8_plain_kernel": "f8_plain.cu", "f8_pair_kernel": "f8_pair.cu", "f8_tokens_kernel": "f8_tokens.cu",
           "f8_rows_kernel": "f8_quantize.cu", "f8_tiles_kernel": "f8_quantize.cu"}
GLOBAL = ["tma_load", "__ldg(", "build_group_table<", "mbar_wait(", "mbar_wait_warp(", "wait_warp_at(", ".load(", "four_scales("]
PRODUCERS = ["f8_pair.cu", "f8_tokens.cu"]


def test_every_kernel_is_listed():
    found = {(k, n) for n, text in _sources().items() if n.startswith("f8_")
             for k in re.findall(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", text)}
    assert found == set(KERNELS.items())


def test_launched_with_the_attribute():
    srcs = _sources()
    names = _pdl_launched_kernels(srcs)
    assert {"f8_plain_kernel", "f8_pair_kernel", "f8_tokens_kernel", "kernel"} <= names
    assert set(re.findall(r"launch_one\((\w+)<", srcs["f8_quantize.cu"])) == {"f8_rows_kernel", "f8_tiles_kernel"}


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_waits_before_global_access(kernel):
    body = _kernel_body(re.sub(r"//[^\n]*", "", _sources()[KERNELS[kernel]]), kernel)
    assert body is not None and body.count("grid_dependency_wait()") == 1
    body = re.sub(r"auto (\w+) = \[&\][^{]*\{.*?\n  \};", "", body, flags=re.S)  # bodies of lambdas run where they are called
    first = [x for x in (body.find(tok) for tok in GLOBAL) if x >= 0]
    assert first and body.index("grid_dependency_wait()") < min(first)
    assert body.index("grid_dependency_wait()") < body.index("grid_dependents_launch()")


@pytest.mark.parametrize("name", PRODUCERS)
def test_producers_wait_for_their_loads(name):
    text = source(name)
    assert set(re.findall(r"mbar_arrive_expect_tx\((\w+) \+ \w+,", text)) == {"full"}
    calls = list(re.finditer(r"\bdrain_ring(?:_lanes)?\(\s*full\s*,", text))
    assert len(calls) == 1
    heads = enclosing(text, calls[0].start())
    assert re.search(r"\(lane == 0\)|^if \(warp == 0\)$", heads[0]), heads[0]  # the producer's block: no loop, no error path
    before = text[:calls[0].start()].rstrip()
    assert not before.endswith(")") or before.endswith("if (leader)")
    assert not re.search(r"if \(!ok[^{;]*\{?\s*(for[^{;]*;[^{;]*;[^{)]*\)\s*)?(if[^;{]*)?drain_", text)


def test_every_producer_file_is_listed():
    names = {n for n in _sources() if "mbar_arrive_expect_tx(full + " in source(n)}
    assert names == set(PRODUCERS)
    assert len(re.findall(r"else\s*\{?\s*drain_odd_cta\(wc\);", source("f8_pair.cu"))) == 1


def test_registers_that_warpgroups_ask_for_fit_the_launch():
    text = source("f8_pair.cu")
    regs = {k: int(v) for k, v in re.findall(r"(kRegs\w+) = (\d+)", text)}
    warps = int(re.search(r"kEpiWarpCount = (\d+)", text).group(1))
    first = int(re.search(r"kEpiWarp0 = (\d+)", text).group(1))
    threads = 32 * (first + warps)
    assert regs["kRegsFew"] * 32 * first + regs["kRegsMany"] * 32 * warps <= regs["kRegsLaunch"] * threads <= 65536
    assert all(r % 8 == 0 for r in regs.values()) and "numRegs != kRegsLaunch" in text
