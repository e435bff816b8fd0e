"""Blocks with an infinity or a NaN, quantized from every type: the scale is that value itself, every
other bit of the block's neighbours as it is defined, and products with it are NaN."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from feed_forward_util import F8, TOP, f8_bound, f8_exact, f8_product, quantize64, within
from operators_util import FLOAT, generator, ok, to64

pytestmark = pytest.mark.gpu


def blocks_of(dtype, rows, cols):
    """128 x 128 blocks: ordinary, +inf, -inf, NaN, NaN beside inf, the largest finite number."""
    x = torch.randn((rows * 128, cols * 128), generator=generator(3), device="cuda").to(FLOAT[dtype])
    most = torch.finfo(FLOAT[dtype]).max
    for i, v in enumerate([None, float("inf"), -float("inf"), float("nan"), (float("nan"), float("inf")), most, -most]):
        r, c = divmod(i * 2 % (rows * cols), cols)
        if v is not None:
            for k, y in enumerate(v if isinstance(v, tuple) else (v,)):
                x[r * 128 + 17, c * 128 + 90 + k] = y
    return x


@pytest.mark.parametrize("q", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block,turn", [(1, False), (128, False), (1, True), (128, True)])
@pytest.mark.parametrize("pad", [0, 1])  # 16 bytes a load; an element a load
def test_scales_of_infinities_and_nan(block, turn, dtype, q, pad):
    x = blocks_of(dtype, 4, 4)
    wide = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, :x.shape[1]] = x
    got, scale = ttc.quantize_blocks(wide[:, :x.shape[1]], block_rows=block, transpose=turn, dtype=F8[q])
    ok(0)
    want, s = quantize64(x, q, block, turn)
    scale = scale.cpu()
    assert torch.isinf(s).any() and torch.isnan(s).any()
    assert torch.equal(torch.isnan(scale), torch.isnan(s))
    there = ~torch.isnan(s)
    assert torch.equal(scale[there].view(torch.int32), s[there].view(torch.int32))
    assert torch.equal(got.cpu().contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [3, 1500])  # few tokens, CTA pairs
@pytest.mark.parametrize("block", [1, 128])
def test_their_products(block, rows, dtype):
    """A token's infinity makes its row NaN, an infinite weight its block's columns, and nothing else."""
    N, K = 1664, 512
    gen = generator(4)
    x = torch.randn((rows, K), generator=gen, device="cuda").to(FLOAT[dtype])
    w = torch.randn((N, K), generator=gen, device="cuda").to(FLOAT[dtype])
    x[1, 300], w[700, 40] = float("inf"), -float("inf")
    a, b = ttc.quantize_blocks(x), ttc.quantize_blocks(w, block_rows=block)
    d = to64(ttc.gemm_f8_blocks(*a, *b, out_dtype=torch.float32))
    ok(0)
    bad = np.zeros((rows, N), dtype=bool)
    bad[1] = True
    bad[:, slice(640, 768) if block == 128 else slice(700, 701)] = True
    assert np.isnan(d[bad]).all()
    sa, sb = to64(a[1]), to64(b[1])
    sa[~np.isfinite(sa)] = 0.0
    sb[~np.isfinite(sb)] = 0.0
    want, s_abs = f8_product(f8_exact(a[0]), sa, f8_exact(b[0]), sb, block)
    within(d[~bad], want[~bad], f8_bound(K, s_abs)[~bad], "f32", "d")
