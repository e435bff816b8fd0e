"""fp32 gradients of weights against 64 bits, by their norm.

The tensor cores cut each addition of sixteen products to 24 bits of the partial
sum, an error of its sign: after n additions of independent terms the cuts add up
to about n / sqrt(3) times 2^-24 of the result (the mean cut is half a unit, the
partial sums grow as the square root of the number of terms).  The kernels start
a fresh accumulator every 768 tokens, 48 additions, which makes that 1.65e-6 at
most however many tokens there are; the cuts' scatter and the additions of the
partial sums, rounded to nearest, stay below 0.35e-6.  One accumulator over 8192
tokens is at 6.4e-6, over 2101 at 2.2e-6 (measured)."""
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from operators_util import generator, ok

pytestmark = pytest.mark.gpu
BOUND = 2.0e-6


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


# columns TMA can read (CTA pairs), and odd ones (plain loads)
@pytest.mark.parametrize("K,N", [(264, 200), (263, 201)])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_partial_sums_of_long_groups(K, N, add, dtype):
    rows = [800, 2101, 0, 767, 8192, 769, 12000]
    gen = generator(sum(rows) + N)
    ends = [sum(rows[:i]) for i in range(len(rows) + 1)]
    a, b = normal(gen, ends[-1], K).to(dtype), normal(gen, ends[-1], N).to(dtype)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    c = normal(gen, len(rows), K, N) * 30.0 if add else None
    got = ttc.gemm_grouped_wgrad(a, b, offsets, c=c, alpha=0.5, beta=1.5 if add else 0.0)
    ok(0)
    for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
        want = 0.5 * (a[lo:hi].double().T @ b[lo:hi].double())
        if add:
            want += 1.5 * c[g].double()
        error = (got[g].double() - want).norm()
        assert error <= BOUND * want.norm(), (hi - lo, float(error / want.norm()))


def test_knob_of_plain_loads():
    """The same operands on either kernel."""
    gen = generator(3)
    a, b = normal(gen, 8192, 264).bfloat16(), normal(gen, 8192, 200).bfloat16()
    offsets = torch.tensor([0, 8192], dtype=torch.int32, device="cuda")
    want = a.double().T @ b.double()
    try:
        for plain in (0, 1):
            assert ttc.ttc_set_knob("force_generic_load", plain) == 0
            got = ttc.gemm_grouped_wgrad(a, b, offsets)
            ok(0)
            assert (got[0].double() - want).norm() <= BOUND * want.norm(), plain
    finally:
        ttc.ttc_set_knob("force_generic_load", 0)
