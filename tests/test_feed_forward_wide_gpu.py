"""GPU parity of the gated feed-forward block and of the block-scaled fp8 product where the
tiles of 64 rows no longer fit one wave, so that CTA pairs take them, and with hundreds of
groups, against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from feed_forward_util import check_gated, f8_bound, f8_product, within
from operators_util import generator, to64
from test_f8_blocks_gpu import Product
from test_gated_gpu import Gated, ends

pytestmark = pytest.mark.gpu

PATTERNS = {
    "edges": [127, 128, 129, 1, 255, 256, 257, 0, 16, 15, 17, 300], "sparse": [0] * 9 + [700] + [0] * 6 + [701],
    "large_among_few": [0] * 50 + [700] + [0] * 30 + [701],
    "uneven": [1, 1400, 0, 3, 64, 65], "even": [192] * 8, "one": [1333],
}


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("pattern", sorted(PATTERNS))
def test_f8_group_sizes(pattern, block):
    o = ends(PATTERNS[pattern])
    Product(o, o[-1], 1160, 400, block=block, seed=len(pattern)).verify()


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("n,k", [(1025, 64), (1160, 127), (1283, 400), (1792, 130), (1281, 1024), (1408, 1), (1288, 129), (1151, 2000)])
def test_f8_widths(n, k, block):
    Product(None, 1301, n, k, seed=n + k, block=block).verify("f32" if k % 2 else "bf16")


@pytest.mark.parametrize("n", [1, 8, 40, 100, 129, 136, 256, 257])
def test_f8_narrow(n):
    """Rows enough that one or two blocks of columns are more than a wave."""
    Product(None, 10201, n, 264, seed=n, block=128 if n % 2 else 1).verify("bf16" if n % 8 else "f16")


@pytest.mark.parametrize("ta", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", [1, 128])
def test_f8_types(ta, tb, block):
    Product(None, 1290, 1160, 528, ta, tb, block, seed=3, negative=True).verify("f32")


@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh"])
@pytest.mark.parametrize("add,bias", [(False, False), (True, False), (False, True), (True, True)])
def test_f8_epilogue(out, act, add, bias):
    Product([0, 400, 400, 1340, 1347], 1347, 1168, 256, seed=5, bias=bias).verify(out, act, add)
    p = Product(None, 1270, 1164, 256, block=1, seed=4, bias=bias)
    p.verify(out, act, add, ldd=1167)
    if add:
        p.verify(out, act, True, ldd=1168, in_place=True)
        p.verify(out, act, True, ldd=1165, in_place=True)


@pytest.mark.parametrize("pad,shift,gap", [((16, 32, 0, 0), 0, 0), ((16, 0, 3, 2), 0, 64), ((0, 0, 0, 1), 16, 16)])
@pytest.mark.parametrize("block", [1, 128])
def test_f8_pitches_and_alignment(pad, shift, gap, block):
    p = Product([0, 500, 500, 1399, 1400], 1400, 1160, 264, block=block, seed=9, pad=pad, shift=shift, gap=gap, bias=True)
    p.verify("bf16", ldd=1163, d_shift=3)
    p.verify("f32", ldd=1168)
    p.verify("bf16", ldd=1176, d_shift=4)


@pytest.mark.parametrize("offsets", [[20, 90, 900, 1350], [-5, 40, 5000], [50, 50, 50], [1300, 0], [-9, -3, 1400]])
def test_offsets_that_leave_rows_out_or_the_matrix(offsets):
    Product(offsets, 1400, 1160, 200, seed=11).verify()
    p = Gated(offsets, 1400, 1032, 72, "bf16", "row", seed=12)
    p.verify()
    p.verify_grad()


def test_f8_scales():
    """NaN, zero and infinite scales stay in their rows and blocks; small blocks beside
    large ones keep their sums."""
    M, N = 1300, 1160
    p = Product(None, M, N, 512, seed=3)
    p.SA[0][2, 1] = float("nan")
    p.SA[0][700, :] = 0.0
    p.SB[0][1, 2] = float("inf")
    got = to64(p.call("f32"))
    assert np.isnan(got[2]).all()
    assert np.isnan(got[700, 128:256]).all() and not np.isfinite(got[:, 128:256]).any()
    assert (got[700, :128] == 0).all() and (got[700, 256:] == 0).all()
    a, sa = p.a64()
    b, sb = p.b64(0)
    sb[1, 2] = 0.0
    sa[2, 1] = 0.0
    want, s_abs = f8_product(a, sa, b, sb, 128)
    pick = np.ix_([i for i in range(M) if i != 2], [j for j in range(N) if not 128 <= j < 256])
    within(got[pick], want[pick], f8_bound(512, s_abs[pick]), "f32", "d")
    p = Product(None, M, N, 1024, seed=13)
    p.SA[0][:, ::2] *= 2.0 ** 18
    p.verify("f32")


def test_f8_no_reduction():
    Product(None, 1300, 1160, 0, bias=True).verify("f32", "gelu_tanh", add=True)


@pytest.mark.parametrize("groups,size", [(400, 66), (1000, 65), (1024, 3), (500, 20), (384, 9)])
def test_hundreds_of_groups(groups, size):
    rng = np.random.default_rng(groups)
    sizes = rng.integers(0, 2 * size + 1, groups)
    sizes[rng.integers(0, groups)] += 130
    sizes[0] += max(0, size * groups - int(sizes.sum()))  # the mean is at least `size`
    o = ends(sizes)
    Product(o, o[-1], 136, 136, block=1, seed=groups).verify()
    Product(o, o[-1], 72, 200, block=128, seed=groups).verify("f32")
    p = Gated(o, o[-1], 72, 72, "bf16", "col", seed=groups)
    p.verify()
    p.verify_grad()
    p = Gated(o, o[-1], 40, 104, "f16", "row", seed=groups)
    p.verify("gelu_tanh")
    p.verify_grad("gelu_tanh")


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pattern", sorted(PATTERNS))
def test_gated_group_sizes(pattern, dtype, layout):
    o = ends(PATTERNS[pattern])
    Gated(o, o[-1], 712, 136, dtype, layout, seed=len(pattern)).verify()


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("n,k", [(641, 64), (1000, 63), (776, 333), (1024, 8), (648, 1000), (704, 128), (1091, 65), (904, 1)])
def test_gated_widths(n, k, layout):
    Gated(None, 1301, n, k, "bf16", layout, seed=n + k).verify(save=n % 2 == 0)


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pattern", sorted(PATTERNS))
def test_gradient_group_sizes(pattern, dtype, layout):
    o = ends(PATTERNS[pattern])
    Gated(o, o[-1], 1096, 136, dtype, layout, seed=len(pattern)).verify_grad(save=len(pattern) % 2 == 0)


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("n,k", [(1025, 64), (1000, 63), (1160, 333), (1024, 8), (1032, 1000), (1091, 65), (1096, 1)])
def test_gradient_widths(n, k, layout):
    p = Gated(None, 1301, n, k, "bf16", layout, seed=n + k)
    p.verify_grad(save=n % 2 == 0)
    p.verify_grad(in_place=True)


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("save", [False, True])
def test_gradient_activations(dtype, act, save):
    for o, layout in (([0, 400, 400, 1340, 1347], "col"), (None, "row")):
        p = Gated(o, 1347, 1040, 320, dtype, layout, seed=3, scale=3.0)
        p.verify_grad(act, save)
        p.verify_grad(act, save, in_place=True)


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("pad,shift,gap", [((8, 16, 24, 8), 0, 64), ((8, 8, 8, 8), 8, 8), ((8, 8, 1, 3), 0, 0), ((8, 8, 8, 4), 0, 0)])
def test_gradient_pitches_and_alignment(pad, shift, gap, layout):
    p = Gated([0, 500, 500, 1399, 1400], 1400, 1032, 264, "bf16", layout, seed=9, pad=pad, shift=shift, gap=gap)
    p.verify_grad("gelu_tanh")
    p.verify_grad("silu", in_place=True)


@pytest.mark.parametrize("n", [1, 8, 40, 64, 100, 128, 136])
def test_gated_narrow(n):
    p = Gated(None, 10201, n, 72, "bf16", "col", seed=n)
    p.verify()
    p.verify_grad()


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("save", [False, True])
def test_gated_activations(dtype, act, save):
    for o, layout in (([0, 400, 400, 1340, 1347], "col"), (None, "row")):
        Gated(o, 1347, 656, 320, dtype, layout, seed=3, scale=3.0).verify(act, save)


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("pad,shift,gap", [((8, 16, 24, 8), 0, 64), ((8, 8, 8, 8), 8, 8), ((8, 8, 1, 3), 0, 0), ((8, 8, 8, 4), 0, 0)])
def test_gated_pitches_and_alignment(pad, shift, gap, layout):
    Gated([0, 500, 500, 1399, 1400], 1400, 648, 264, "bf16", layout, seed=9, pad=pad, shift=shift, gap=gap).verify("gelu_tanh")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("layout", ["col", "row"])
def test_gated_groups_do_not_leak(layout, value):
    o = ends([200, 300, 730, 90])
    p = Gated(o, o[-1], 648, 200, "bf16", layout, seed=12)
    p.A[200:500] = value
    for buf, views in p.W:
        views[1].fill_(value)
    p.forward("silu", True)
    d, kept = to64(p.view(p.d, p.ldd)), to64(p.view(p.kept, p.ldp))
    a = to64(p.A)
    for g, (lo, hi) in enumerate(zip(o, o[1:])):
        if g == 1:
            assert not np.isfinite(kept[lo:hi, :2 * p.N]).any()
            continue
        x = a[lo:hi]
        q = [(x @ p.w64(i, g), np.abs(x) @ np.abs(p.w64(i, g))) for i in range(2)]
        check_gated(d[lo:hi, :p.N], q[0][0], q[1][0], q[0][1], q[1][1], p.K, "silu", "bf16")


@pytest.mark.parametrize("rows,n", [(1300, 648), (100, 648)])
def test_the_same_call_gives_the_same_bits(rows, n):
    gen = generator(8)
    a = torch.randn((rows, 520), generator=gen, device="cuda").bfloat16()
    w = torch.randn((2 * n, 520), generator=gen, device="cuda").bfloat16() / 20
    first = ttc.gemm_gated(a, w[:n].t(), w[n:].t(), pre=True)
    qa, sa = ttc.quantize_blocks(a)
    qw, sw = ttc.quantize_blocks(w, block_rows=128)
    f8 = ttc.gemm_f8_blocks(qa, sa, qw, sw)
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(first, ttc.gemm_gated(a, w[:n].t(), w[n:].t(), pre=True)))
        assert torch.equal(f8, ttc.gemm_f8_blocks(qa, sa, qw, sw))


@pytest.mark.parametrize("rows,n", [(40, 136), (300, 264), (2000, 1160)])
@pytest.mark.parametrize("block", [1, 128])
def test_groups_that_share_weights(rows, n, block):
    """Weights and scales expanded over the groups, stride 0, give what copies of them give."""
    gen = generator(31)
    groups, k = 3, 264
    cut = torch.tensor([0, rows // 4, rows // 2, rows - 1], dtype=torch.int32, device="cuda")
    a = torch.randn((rows, k), generator=gen, device="cuda").bfloat16()
    w = torch.randn((2 * n, k), generator=gen, device="cuda").bfloat16() / 16
    one = [w[:n].t()[None].expand(groups, k, n), w[n:].t()[None].expand(groups, k, n)]
    many = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in one]
    outs = [torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pres = [torch.zeros((rows, 2 * n), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for x, out, pre in zip((one, many), outs, pres):
        ttc.gemm_gated(a, *x, out, offsets=cut, pre=pre)
    assert torch.equal(*outs) and torch.equal(*pres) and outs[0][:-1].abs().sum() > 0
    dy = torch.randn((rows, k), generator=gen, device="cuda").bfloat16()
    grads = [torch.zeros_like(pres[0]) for _ in range(2)]
    for x, d in zip((one[0], many[0]), grads):
        ttc.gemm_gated_grad(dy, x, pres[0], d, offsets=cut)
    assert torch.equal(*grads)
    qa, sa = ttc.quantize_blocks(a)
    qw, sw = ttc.quantize_blocks(w[:n], block_rows=block)
    shared = [t[None].expand(groups, *t.shape) for t in (qw, sw)]
    # rows on 16-byte boundaries, as the quantizer leaves them
    copy = torch.empty((groups, n, qw.stride(0)), dtype=torch.uint8, device="cuda")[..., :k].view(qw.dtype)
    copy.view(torch.uint8).copy_(shared[0].view(torch.uint8))
    outs = [torch.zeros((rows, n), device="cuda") for _ in range(2)]
    ttc.gemm_f8_blocks(qa, sa, *shared, outs[0], offsets=cut)
    ttc.gemm_f8_blocks(qa, sa, copy, shared[1].contiguous(), outs[1], offsets=cut)
    assert torch.equal(*outs) and outs[0][:-1].abs().sum() > 0
