"""Operands and results whose offsets pass 2^31 elements: the last rows, groups and
tiles against 64-bit forms (and the first, which an offset cut to 32 bits would hit)."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from operators_util import check, ok, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def normal(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ints(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("K", [64, 63])  # CTA pairs, plain loads
def test_grouped_result_beyond_2_31(K):
    M, N, offsets = 530_000, 4104, [0, 5, 529_000, 530_000]
    assert M * N > 1 << 31
    a, b = normal((M, K), 1), normal((3, N, K), 2).transpose(1, 2)
    got = ttc.gemm_grouped(a, b, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    ok(0)
    for g, rows in ((0, slice(0, 5)), (1, slice(5, 70)), (1, slice(523_000, 523_300)), (2, slice(529_700, 530_000))):
        A, B = to64(a[rows]), to64(b[g])
        check(to64(got[rows]), A @ B, np.abs(A) @ np.abs(B), K, "bf16")


@pytest.mark.parametrize("rows", [2, 300])  # few tokens, CTA pairs
def test_grouped_weights_beyond_2_31(rows):
    groups, N, K = 40, 14336, 4096
    assert groups * N * K > 1 << 31
    b = torch.empty((groups, N, K), dtype=torch.bfloat16, device="cuda")
    for g in range(groups):
        b[g].copy_(normal((N, K), g))
    a = normal((groups * rows, K), 99)
    offsets = torch.arange(0, groups * rows + 1, rows, dtype=torch.int32, device="cuda")
    got = ttc.gemm_grouped(a, b.transpose(1, 2), offsets)
    ok(0)
    for g in (0, 3, 38, 39):
        part = slice(g * rows, g * rows + 2)
        A, B = to64(a[part]), to64(b[g]).T
        check(to64(got[part]), A @ B, np.abs(A) @ np.abs(B), K, "bf16")


def test_gradients_beyond_2_31():
    groups, N, K, rows = 130, 4096, 4104, 5
    assert groups * N * K > 1 << 31
    a, b = normal((groups * rows, K), 3), normal((groups * rows, N), 4)
    offsets = torch.arange(0, groups * rows + 1, rows, dtype=torch.int32, device="cuda")
    out = torch.full((groups, K, N), 0.5, device="cuda")
    ttc.gemm_grouped_wgrad(a, b, offsets, c=out, out=out, beta=1.0)
    ok(0)
    for g in (0, 2, 127, 129):
        A, B = to64(a[g * rows:(g + 1) * rows]), to64(b[g * rows:(g + 1) * rows])
        for part in (slice(0, 40), slice(K - 40, K)):
            check(to64(out[g, part]), A[:, part].T @ B + 0.5, np.abs(A[:, part]).T @ np.abs(B) + 0.5, rows, "f32")


@pytest.mark.parametrize("workspace", [True, False])
def test_int8_result_beyond_2_31(workspace):
    M, N, K = 530_000, 4104, 128
    assert M * N > 1 << 31
    a, b = ints((M, K), 5), ints((N, K), 6)
    ws = None if workspace else torch.empty(1, dtype=torch.uint8, device="cuda")
    got = ttc.gemm_i8_scaled(a, torch.ones(M, device="cuda"), b, torch.ones(N, device="cuda"), workspace=ws,
                             out_dtype=torch.float16 if workspace else torch.float32)
    ok(0)
    for rows in (slice(0, 300), slice(523_200, 523_300), slice(529_800, 530_000)):
        want = (a[rows].cpu().double() @ b.cpu().double().T).float().to(got.dtype)  # exact, rounded once
        assert torch.equal(got[rows].cpu(), want)


def test_quantized_rows_beyond_2_31():
    rows, cols = 1_060_000, 2056
    assert rows * cols > 1 << 31
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 53_000):
        x[i:i + 53_000].copy_(normal((53_000, cols), i))
    q, scale = ttc.quantize_rows(x)
    ok(0)
    for part in (slice(0, 64), slice(rows - 64, rows)):
        v = to64(x[part])
        s = np.float32(np.abs(v).max(axis=1) / 127.0)
        assert (to64(scale[part]) == s).all()
        # within half a step, and two roundings of a quotient of at most 127
        assert (np.abs(to64(q[part]) * s[:, None].astype(np.float64) - v) <= 0.5 * s[:, None] * (1 + 2.0 ** -15)).all()
