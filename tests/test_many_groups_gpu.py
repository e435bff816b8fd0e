"""Grouped products of so many groups that the CTA pairs' table holds every fourth
group only (forward from 192 groups, with too many rows for the few-token kernel),
or none of the offsets (gradient of weights from 384)."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from operators_util import check, clamp_offsets, ok, to64

pytestmark = pytest.mark.gpu


def problem(groups, mean, K, N, seed, dtype=torch.bfloat16):
    """Uneven groups, a tenth of them empty, one as long as several tiles."""
    rng = np.random.default_rng(seed)
    rows = rng.integers(0, 2 * mean, groups) * (rng.random(groups) > 0.1)
    rows[groups // 3] = 600
    ends = np.concatenate([[0], np.cumsum(rows)]).tolist()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(dtype)
    return (normal(ends[-1], K), normal(groups, K, N), normal(ends[-1], N), ends,
            torch.tensor(ends, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("groups", [190, 191, 192, 193, 257, 1024])
def test_forward(groups):
    K, N = 64, 264
    a, b, _, ends, offsets = problem(groups, 110, K, N, groups)
    assert ends[-1] > 81 * groups  # not few tokens
    got = to64(ttc.gemm_grouped(a, b, offsets))
    ok(0)
    A, B = to64(a), to64(b)
    for g, (lo, hi) in enumerate(clamp_offsets(ends, ends[-1])):
        check(got[lo:hi], A[lo:hi] @ B[g], np.abs(A[lo:hi]) @ np.abs(B[g]), K, "bf16")


@pytest.mark.parametrize("groups", [382, 383, 384, 385, 1024])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_gradient(groups, out):
    K, N = 72, 40
    a, _, dy, ends, offsets = problem(groups, 12, K, N, groups + 1)
    got = to64(ttc.gemm_grouped_wgrad(a, dy, offsets, out_dtype=out))
    ok(0)
    A, B = to64(a), to64(dy)
    name = "f32" if out == torch.float32 else "bf16"
    for g, (lo, hi) in enumerate(clamp_offsets(ends, ends[-1])):
        check(got[g], A[lo:hi].T @ B[lo:hi], np.abs(A[lo:hi]).T @ np.abs(B[lo:hi]), max(hi - lo, 1), name)
