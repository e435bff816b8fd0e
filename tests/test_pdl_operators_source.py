"""Source checks for programmatic dependent launch of the grouped and int8 operators
(no GPU): each of their kernels is launched with the attribute and waits for the
previous grid before it first reads or writes global memory."""
import re

import pytest

from test_pdl_source import _kernel_body, _pdl_launched_kernels, _sources

# calls that reach global memory; build_group_table reads the offsets, the load_*
# and prefetch_w lambdas of i8_rows_kernel its operands
GLOBAL = ["tma_load", "__ldg(", "__ldcs(", "build_group_table<", "mbar_wait(", "mbar_wait_warp(", "mbar_wait_cluster(",
          "widen_load<", "src[", "load_w(c", "load_x(c", "prefetch_w(c"]
KERNELS = {
    "few_tokens_kernel": "few_tokens.cu", "grouped_pair_kernel": "grouped_pair.cu", "grouped_plain_kernel": "grouped_plain.cu",
    "i8_rows_kernel": "i8_rows.cu", "i8_tokens_kernel": "i8_tokens.cu", "quantize_rows_kernel": "quantize.cu",
    "quantize_any_kernel": "quantize.cu", "widen_i8_kernel": "repack.cu",
}


def without_comments(text):
    return re.sub(r"//[^\n]*", "", text)


def test_launched_with_the_attribute():
    srcs = _sources()
    names = _pdl_launched_kernels(srcs)
    direct = set(KERNELS) - {"quantize_rows_kernel", "quantize_any_kernel"}  # those through launch_one
    assert direct <= names, direct - names
    assert "kernel" in names
    launched = set(re.findall(r"launch_one\((\w+)<", srcs["quantize.cu"]))
    assert launched == {"quantize_rows_kernel", "quantize_any_kernel"}


def test_every_kernel_of_these_files_is_listed():
    srcs = _sources()
    for name in set(KERNELS.values()) - {"repack.cu"}:
        found = set(re.findall(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", srcs[name]))
        assert found == {k for k, f in KERNELS.items() if f == name}


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_waits_before_global_access(kernel):
    body = _kernel_body(without_comments(_sources()[KERNELS[kernel]]), kernel)
    assert body is not None and body.count("grid_dependency_wait()") == 1
    # bodies of lambdas run where they are called
    body = re.sub(r"auto (\w+) = \[&\][^{]*\{.*?\n  \};", "", body, flags=re.S)
    first = [x for x in (body.find(tok) for tok in GLOBAL) if x >= 0]
    assert first and body.index("grid_dependency_wait()") < min(first)
    assert body.index("grid_dependency_wait()") < body.index("grid_dependents_launch()")
