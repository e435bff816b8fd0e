"""The torch wrappers on a stream of the caller's: the memory they take for
results and scratch belongs to no work that is still to run on another stream."""
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from operators_util import generator

pytestmark = pytest.mark.gpu
DELAY = 200_000_000  # clocks: about a tenth of a second


def normal(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=generator(seed), device="cuda").to(dtype)


def calls():
    """name -> (call(stream), bytes of each block that the call takes)"""
    M, N, K = 1100, 4100, 1111
    a, b = normal(1, M, 1024), normal(2, 1024, 2048)
    w = normal(3, 2, 1024, 2048)
    offsets = torch.tensor([0, 500, M], dtype=torch.int32, device="cuda")
    x = normal(4, M, K)
    dy = normal(5, M, 2048)
    qx, sx = ttc.quantize_rows(x)
    qw, sw = ttc.quantize_rows(normal(6, N, K))
    need = ttc.ttc_gemm_i8_scaled_workspace_size(M, N, K, qx.data_ptr(), qx.stride(0), qw.data_ptr(), qw.stride(0), 0, N,
                                                 ttc.DTYPE["bf16"])
    assert need > 0
    return {
        "gemm": (lambda s: (ttc.gemm(a, b, stream=s),), [M * 2048 * 2]),
        "gemm_grouped": (lambda s: (ttc.gemm_grouped(a, w, offsets, stream=s),), [M * 2048 * 2]),
        "gemm_grouped_wgrad": (lambda s: (ttc.gemm_grouped_wgrad(a, dy, offsets, stream=s),), [2 * 1024 * 2048 * 4]),
        "quantize_rows": (lambda s: ttc.quantize_rows(x, stream=s), [M * 1120, M * 4]),
        "gemm_i8_scaled": (lambda s: (ttc.gemm_i8_scaled(qx, sx, qw, sw, stream=s),), [M * N * 2, need]),
    }


NAMES = ["gemm", "gemm_grouped", "gemm_grouped_wgrad", "quantize_rows", "gemm_i8_scaled"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_with_work_on_the_current_stream(name):
    call, blocks = calls()[name]
    s = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    copies = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in blocks]
    tenants = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in blocks]
    torch.cuda.synchronize()
    # the current stream reads the blocks late and writes them again after that
    torch.cuda._sleep(DELAY)
    for t, c in zip(tenants, copies):
        c.copy_(t)
        t.fill_(9)
    tenants.clear()
    del t
    got = call(s.cuda_stream)
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", NAMES)
def test_results_read_on_the_current_stream(name):
    """A result is dropped while the current stream has yet to read it; the next call
    on the other stream may not have its memory."""
    call, _ = calls()[name]
    s = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    kept = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = call(s.cuda_stream)
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    for k, g in zip(kept, got):
        k.copy_(g)
    del got, g
    with torch.cuda.stream(s):
        scratch = [torch.full_like(w, 3) for w in want]  # what the other stream does next
    torch.cuda.synchronize()
    assert len(scratch) == len(want)
    for k, w in zip(kept, want):
        assert torch.equal(k, w)


def test_the_default_stream_by_its_address():
    """Address 0 is the default stream, whatever stream is current."""
    a, b = normal(7, 64, 96), normal(8, 96, 128)
    want = ttc.gemm(a, b)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = ttc.gemm(a, b, stream=0)
        q, scale = ttc.quantize_rows(a, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(scale, a.float().abs().amax(dim=1) / 127)


@pytest.mark.parametrize("name", NAMES)
def test_an_external_stream_that_is_current(name):
    call, _ = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call(s.cuda_stream)
    s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
