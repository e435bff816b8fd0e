"""The grouped and int8 operators on the kernel for plain loads with operands that
TMA could read, and a stalled pipeline: every wait ends, the call reports the
timeout, and the next call's result is right."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from operators_util import check, clamp_offsets, ok, stream, to64

pytestmark = pytest.mark.gpu


@pytest.fixture
def knob():
    names = []

    def set_knob(name, value):
        assert ttc.ttc_set_knob(name, value) == 0
        names.append(name)

    yield set_knob
    for name in names:
        ttc.ttc_set_knob(name, 0)


def normal(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def problem(rows, groups, K, N, seed=0):
    cuts = np.sort(np.random.default_rng(seed).integers(0, rows + 1, groups - 1))
    offsets = [0, *map(int, cuts), rows]
    return (normal((rows, K), seed + 1), normal((groups, K, N), seed + 2), normal((rows, N), seed + 3), offsets,
            torch.tensor(offsets, dtype=torch.int32, device="cuda"))


def verify_grouped(a, b, offsets, dev):
    got = ttc.gemm_grouped(a, b, dev)
    ok(0)
    for g, (lo, hi) in enumerate(clamp_offsets(offsets, a.shape[0])):
        A, B = to64(a)[lo:hi], to64(b)[g]
        check(to64(got)[lo:hi], A @ B, np.abs(A) @ np.abs(B), a.shape[1], "bf16")


def verify_wgrad(a, dy, offsets, dev, out_dtype):
    got = ttc.gemm_grouped_wgrad(a, dy, dev, out_dtype=out_dtype)
    ok(0)
    for g, (lo, hi) in enumerate(clamp_offsets(offsets, a.shape[0])):
        A, B = to64(a)[lo:hi], to64(dy)[lo:hi]
        check(to64(got)[g], A.T @ B, np.abs(A).T @ np.abs(B), max(hi - lo, 1), "f32" if out_dtype == torch.float32 else "bf16")


def verify_i8(M, N, K, workspace=True):
    g = torch.Generator(device="cuda").manual_seed(M)
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ones = lambda n: torch.ones(n, device="cuda")
    ws = None if workspace else torch.empty(1, dtype=torch.uint8, device="cuda")
    got = ttc.gemm_i8_scaled(a, ones(M), b, ones(N), out_dtype=torch.float32, workspace=ws)
    ok(0)
    want = (a.cpu().double() @ b.cpu().double().T).float()  # the exact sum, rounded once
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("rows,groups,K,N", [(300, 3, 256, 264), (40, 8, 512, 136), (900, 2, 72, 520)])
def test_plain_loads_of_aligned_operands(knob, rows, groups, K, N):
    a, b, dy, offsets, dev = problem(rows, groups, K, N)
    knob("force_generic_load", 1)
    verify_grouped(a, b, offsets, dev)
    verify_grouped(a, b.transpose(1, 2).contiguous().transpose(1, 2), offsets, dev)
    for out in (torch.float32, torch.bfloat16):
        verify_wgrad(a, dy, offsets, dev, out)


@pytest.mark.parametrize("M", [40, 300, 520])
def test_int8_on_plain_loads(knob, M):
    knob("force_generic_load", 1)
    verify_i8(M, 264, 528)


# (mean rows a group) few tokens, CTA pairs, plain loads
@pytest.mark.parametrize("rows,groups,K,N,plain", [(32, 4, 256, 256, False), (1200, 2, 256, 512, False),
                                                   (1200, 2, 256, 512, True)])
def test_a_stalled_grouped_product_times_out(knob, rows, groups, K, N, plain):
    a, b, dy, offsets, dev = problem(rows, groups, K, N, seed=9)
    if plain:
        knob("force_generic_load", 1)
    knob("timeout_ns", 20_000_000)
    knob("inject_stall", 1)
    out = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    grad = torch.empty((groups, K, N), device="cuda")
    ttc.gemm_grouped(a, b, dev, out)
    assert ttc.STATUS[ttc.ttc_get_device_error(stream())] == "TTC_ERR_TIMEOUT"
    ttc.gemm_grouped_wgrad(a, dy, dev, out=grad)
    assert ttc.STATUS[ttc.ttc_get_device_error(stream())] == "TTC_ERR_TIMEOUT"
    knob("inject_stall", 0)
    knob("timeout_ns", 0)
    verify_grouped(a, b, offsets, dev)
    verify_wgrad(a, dy, offsets, dev, torch.float32)


@pytest.mark.parametrize("M,N,K", [(20, 256, 1024), (64, 512, 512), (1024, 4096, 512)])
def test_a_stalled_int8_product_times_out(knob, M, N, K):
    knob("timeout_ns", 20_000_000)
    knob("inject_stall", 1)
    a, b = torch.ones((M, K), dtype=torch.int8, device="cuda"), torch.ones((N, K), dtype=torch.int8, device="cuda")
    ttc.gemm_i8_scaled(a, torch.ones(M, device="cuda"), b, torch.ones(N, device="cuda"))
    assert ttc.STATUS[ttc.ttc_get_device_error(stream())] == "TTC_ERR_TIMEOUT"
    knob("inject_stall", 0)
    knob("timeout_ns", 0)
    verify_i8(M, N, K)
