"""GELU of negative values in fp32, relative to the value itself, in each kernel of
the scaled int8 product: an accumulator of one, so that the product is the token's
scale exactly.

gelu(v) = v / (1 + exp(-w)), w = 2 sqrt(2/pi) (v + 0.044715 v^3).  Relative errors, in
units of 2^-24: w has two constants, two products, a fused sum of terms of one
sign and a product, 6 at most, which exp turns into 6 |w|; __expf itself is documented
with 2 + 1.173 |w| units in the last place, 2 each; the sum 1; the quotient
2 units in the last place, 4; the logistic's slope passes at most all of it on."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from operators_util import ok

pytestmark = pytest.mark.gpu


# few tokens; some hundred; rows TMA cannot read, many: the fp16 copies
@pytest.mark.parametrize("M,pitch", [(16, 16), (200, 16), (1024, 17)])
def test_relative_error_of_negative_values(M, pitch):
    N, K = 40, 16
    gen = torch.Generator(device="cuda").manual_seed(M)
    a = torch.zeros((M, pitch), dtype=torch.int8, device="cuda")[:, :K]
    b = torch.zeros((N, pitch), dtype=torch.int8, device="cuda")[:, :K]
    a[:, 0] = 1
    b[:, 0] = -1
    scale_a = 6.0 * torch.rand(M, generator=gen, device="cuda")
    scale_a[:2] = torch.tensor([6.0, 2.0 ** -20])
    scale_b = torch.ones(N, device="cuda")
    got = ttc.gemm_i8_scaled(a, scale_a, b, scale_b, out_dtype=torch.float32, act="gelu_tanh").cpu().double().numpy()
    ok(0)
    v = -scale_a.cpu().double().numpy()[:, None]
    w = 2.0 * np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3)
    want = v / (1.0 + np.exp(-w))
    units = 6.0 * np.abs(w) + 2.0 * (2.0 + 1.173 * np.abs(w)) + 1.0 + 4.0
    assert (np.abs(got - want) <= units * 2.0 ** -24 * np.abs(want)).all()
