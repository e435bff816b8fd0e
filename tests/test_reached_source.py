"""Source checks that nothing of the int8 operators' host side is without use (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_tensor_core_02_gb300",
                    "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_every_block_of_tokens_is_one_the_host_picks():
    text = source("i8_tokens.cu")
    launch = text[text.index("cudaError_t launch_i8_tokens("):]
    cases = {int(m) for m in re.findall(r"case (\d+):", launch)}
    host = source("operators.cu")
    block = re.search(r"const int block = ([^;]*);\s*double few_us", host).group(1)
    # the kernel runs from 17 tokens on
    assert re.search(r"const bool few = M > 16 &&", host)
    assert all(int(m) > 16 for m in re.findall(r"M <= (\d+)", block)), block
    assert cases == {int(m) for m in re.findall(r"[?:] (\d+)", block)}


def test_every_field_of_the_environment_is_read():
    fields = re.search(r"struct HostEnv \{(.*?)\};", source("host.cuh"), re.S).group(1)
    names = re.findall(r"(\w+);", fields)
    readers = "".join(source(n) for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")) and n != "gemm.cu")
    assert names and all(f"env.{n}" in readers for n in names), names
