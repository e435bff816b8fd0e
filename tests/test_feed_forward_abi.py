"""CPU-side checks of the gated feed-forward and the block-scaled fp8 entry points:
what they refuse before any GPU work, and what they take as empty; the same of their
torch wrappers."""
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from tiled_tensor_core_02_gb300 import _build

F16, BF16, I8, F32, E4M3, E5M2 = (ttc.DTYPE[k] for k in ("f16", "bf16", "i8", "f32", "f8_e4m3", "f8_e5m2"))
R, C = ttc.ROW_MAJOR, ttc.COL_MAJOR
SILU = ttc.ACT["silu"]
P = 1 << 24  # fake, never-dereferenced addresses, far enough apart
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return ttc.load()


def gated(groups=4, M=64, N=32, K=48, A=P, lda=48, offsets=P * 9, Bg=P * 3, Bu=P * 4, ldb=None, strideB=32 * 48, layout=C, D=P * 6,
          ldd=32, gate=None, up=None, ldp=64, act=SILU, dtype=BF16):
    ldb = max(K if layout == C else N, 1) if ldb is None else ldb
    return ttc.ttc_gemm_gated(groups, M, N, K, A, lda, offsets, Bg, Bu, ldb, strideB, layout, D, ldd, gate, up, ldp, act, dtype,
                              None)


KEPT = dict(gate=P * 12, up=P * 12 + 64)


@pytest.mark.parametrize("kw", [
    dict(groups=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(strideB=-1), dict(layout=2), dict(act=4), dict(act=-1), dict(dtype=7),
    dict(dtype=E4M3), dict(lda=47), dict(ldb=47), dict(layout=R, ldb=31), dict(ldd=31),
    dict(A=None), dict(Bg=None), dict(Bu=None), dict(D=None), dict(offsets=None),
    dict(A=P + 1), dict(Bg=P * 3 + 1), dict(Bu=P * 4 + 1), dict(D=P * 6 + 1), dict(offsets=P * 9 + 2),
    dict(D=P), dict(D=P * 3), dict(D=P * 4), dict(D=P + 64 * 48 * 2 - 2), dict(D=P * 4 + 4 * 32 * 48 * 2 - 2),
    dict(gate=P * 12), dict(up=P * 12), dict(KEPT, ldp=31), dict(KEPT, gate=P * 12 + 1), dict(KEPT, up=P * 12),
    dict(KEPT, up=P * 12 + 62), dict(KEPT, gate=P * 6), dict(KEPT, up=P * 6 + 62), dict(KEPT, gate=P), dict(KEPT, up=P * 3),
    dict(KEPT, gate=P * 12, up=P * 12 + 66), dict(KEPT, ldp=63),
])
def test_gated_invalid(kw):
    assert gated(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=I8), dict(dtype=F32), dict(groups=1025), dict(M=1 << 31), dict(N=1 << 31, ldd=1 << 31),
                                dict(strideB=1 << 41), dict(ldd=1 << 31), dict(KEPT, ldp=1 << 31)])
def test_gated_unsupported(kw):
    assert gated(**kw) == UNSUPPORTED


# Outputs in the rows of an input's buffer, beside it: of 80 columns A (or the weights) takes the first 48 (32)
# and an output the next 32.
WIDE = dict(lda=80, ldd=80)
ROWS = dict(layout=R, ldb=80, ldd=80, strideB=48 * 80)
BESIDE_GATED = [dict(WIDE, D=P + 2 * 48), dict(KEPT, lda=80, gate=P + 2 * 48, up=P * 12, ldp=80), dict(ROWS, D=P * 3 + 2 * 32),
                dict(ROWS, D=P * 4 + 2 * 48), dict(ROWS, D=P * 4 + 2 * (48 * 80 + 40)),
                dict(D=P * 3 + 2 * 32 * 48, strideB=1 << 20), dict(groups=1, offsets=None, strideB=7, D=P * 4 + 2 * 32 * 48)]
BESIDE_GRAD = [dict(WIDE, D=P + 2 * 48), dict(lda=128, lddp=128, dgate=P + 2 * 48, dup=P + 2 * 88), dict(ROWS, D=P * 3 + 2 * 32),
               dict(ROWS, lddp=80, dup=P * 3 + 2 * 33, dgate=P * 14)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are taken would run on these addresses")
@pytest.mark.parametrize("call,kw", [(0, kw) for kw in BESIDE_GATED] + [(1, kw) for kw in BESIDE_GRAD])
def test_outputs_beside_inputs_are_taken(call, kw):
    assert (grad if call else gated)(**kw) == 3  # as far as the missing GPU


@pytest.mark.parametrize("kw", [dict(WIDE, D=P + 2 * 47), dict(WIDE, D=P + 2 * 49), dict(WIDE, ldd=81, D=P + 2 * 48),
                                dict(WIDE, D=P - 2 * 31), dict(ROWS, D=P * 3 + 2 * 31), dict(ROWS, D=P * 4 + 2 * 49),
                                dict(ROWS, strideB=48 * 80 + 1, D=P * 4 + 2 * 32 + 2 * 80 * 47), dict(ROWS, strideB=1, D=P * 3 + 2 * 32),
                                dict(D=P * 3 + 2 * 32 * 48 - 2, strideB=1 << 20), dict(D=P * 3 + 2 * 3 * (1 << 20), strideB=1 << 20)])
def test_gated_beside_and_over(kw):
    assert gated(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(WIDE, D=P + 2 * 47), dict(lda=128, lddp=128, dgate=P + 2 * 48, dup=P + 2 * 97),
                                dict(ROWS, lddp=80, dup=P * 3 + 2 * 49, dgate=P * 14), dict(ROWS, D=P * 3 + 2 * 31)])
def test_grad_beside_and_over(kw):
    assert grad(**kw) == INVALID


def test_gated_empty():
    for kw in (dict(groups=0), dict(M=0), dict(N=0), dict(M=0, A=None, Bg=None, Bu=None, D=None, offsets=None)):
        assert gated(**kw) == 0


def grad(groups=4, M=64, N=32, K=48, A=P, lda=48, offsets=P * 9, B=P * 3, ldb=None, strideB=32 * 48, layout=C, gate=P * 12,
         up=P * 12 + 64, ldp=64, dgate=P * 14, dup=P * 14 + 64, lddp=64, D=None, ldd=32, act=SILU, dtype=BF16):
    ldb = max(K if layout == C else N, 1) if ldb is None else ldb
    return ttc.ttc_gemm_gated_grad(groups, M, N, K, A, lda, offsets, B, ldb, strideB, layout, gate, up, ldp, dgate, dup, lddp, D,
                                   ldd, act, dtype, None)


@pytest.mark.parametrize("kw", [
    dict(groups=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(strideB=-1), dict(layout=2), dict(act=4), dict(dtype=7),
    dict(lda=47), dict(ldb=47), dict(layout=R, ldb=31), dict(ldp=31), dict(lddp=31), dict(D=P * 6, ldd=31),
    dict(A=None), dict(B=None), dict(gate=None), dict(up=None), dict(dgate=None), dict(dup=None), dict(offsets=None),
    dict(A=P + 1), dict(B=P * 3 + 1), dict(gate=P * 12 + 1), dict(up=P * 12 + 63), dict(dgate=P * 14 + 1), dict(dup=P * 14 + 63),
    dict(D=P * 6 + 1), dict(offsets=P * 9 + 2), dict(dgate=P), dict(dup=P * 3), dict(D=P), dict(D=P * 3),
    dict(dup=P * 14), dict(dup=P * 14 + 62), dict(dgate=P * 12), dict(dup=P * 12 + 64), dict(dgate=P * 12 + 64, dup=P * 12),
    dict(dgate=P * 12, dup=P * 12 + 64, lddp=66), dict(D=P * 12), dict(D=P * 14 + 64), dict(D=P * 14, dgate=P * 14 + 32),
])
def test_grad_invalid(kw):
    assert grad(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=I8), dict(dtype=F32), dict(groups=1025), dict(M=1 << 31), dict(ldp=1 << 31),
                                dict(lddp=1 << 31), dict(strideB=1 << 41), dict(D=P * 6, ldd=1 << 31)])
def test_grad_unsupported(kw):
    assert grad(**kw) == UNSUPPORTED


def test_grad_empty():
    for kw in (dict(groups=0), dict(M=0), dict(N=0), dict(M=0, gate=None, dgate=None)):
        assert grad(**kw) == 0


def quantize(rows=8, cols=256, X=P, ldx=256, dtype=BF16, block=1, turn=0, Q=P * 3, ldq=256, q=E4M3, scale=P * 6, lds=2):
    return ttc.ttc_quantize_blocks(rows, cols, X, ldx, dtype, block, turn, Q, ldq, q, scale, lds, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(dtype=8), dict(q=8), dict(block=0), dict(block=64), dict(block=-1), dict(turn=2), dict(turn=-1),
    dict(X=None), dict(Q=None), dict(scale=None), dict(ldx=255), dict(ldq=255), dict(lds=1), dict(turn=1, ldq=7), dict(turn=1, lds=0),
    dict(X=P + 1), dict(dtype=F32, X=P + 2), dict(scale=P * 6 + 2), dict(Q=P), dict(scale=P), dict(scale=P * 3),
])
def test_quantize_invalid(kw):
    assert quantize(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=I8), dict(dtype=E4M3), dict(q=I8), dict(q=BF16), dict(rows=1 << 31), dict(ldq=1 << 31),
                                dict(lds=1 << 31)])
def test_quantize_unsupported(kw):
    assert quantize(**kw) == UNSUPPORTED


def test_quantize_empty():
    assert quantize(rows=0) == 0 and quantize(cols=0, X=None, Q=None, scale=None) == 0


def f8(groups=4, M=64, N=160, K=300, A=P, lda=304, ta=E4M3, sa=P * 2, ldsa=3, offsets=P * 9, B=P * 3, ldb=304, strideB=160 * 304,
       tb=E4M3, sb=P * 4, ldsb=3, strideSB=6, block=128, Cp=None, ldc=160, D=P * 6, ldd=160, bias=None, strideBias=160, act=0, out=BF16):
    return ttc.ttc_gemm_f8_blocks(groups, M, N, K, A, lda, ta, sa, ldsa, offsets, B, ldb, strideB, tb, sb, ldsb, strideSB, block, Cp,
                                  ldc, D, ldd, bias, strideBias, act, out, None)


@pytest.mark.parametrize("kw", [
    dict(groups=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(strideB=-1), dict(strideSB=-1), dict(strideBias=-1),
    dict(ta=9), dict(tb=-1), dict(out=6), dict(act=SILU), dict(act=-1), dict(block=2), dict(block=0), dict(offsets=None),
    dict(A=None), dict(B=None), dict(sa=None), dict(sb=None), dict(D=None), dict(lda=299), dict(ldb=299), dict(ldsa=2), dict(ldsb=2),
    dict(ldd=159), dict(Cp=P * 12, ldc=159), dict(sa=P * 2 + 2), dict(sb=P * 4 + 1), dict(bias=P * 12 + 2), dict(D=P * 6 + 1),
    dict(out=F32, D=P * 6 + 2), dict(Cp=P * 12 + 1), dict(offsets=P * 9 + 1), dict(D=P), dict(D=P * 3), dict(D=P * 2), dict(D=P * 4),
    dict(Cp=P * 6, ldc=161), dict(Cp=P * 6 + 2), dict(D=P * 12, bias=P * 12 + 640),
])
def test_f8_invalid(kw):
    assert f8(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(ta=I8), dict(tb=BF16), dict(out=I8), dict(out=E4M3), dict(groups=1025), dict(M=1 << 31),
                                dict(K=1 << 31, lda=1 << 31, ldb=1 << 31, ldsa=1 << 24, ldsb=1 << 24), dict(ldsa=1 << 31),
                                dict(strideB=1 << 41), dict(strideSB=1 << 41), dict(ldd=1 << 31)])
def test_f8_unsupported(kw):
    assert f8(**kw) == UNSUPPORTED


# The offsets of the four groups (20 bytes at P * 9) are an input too: written while tiles are being dealt out,
# parts of the grid would disagree about them.
END = P * 9 + 20


@pytest.mark.parametrize("call,kw", [
    (gated, dict(D=END - 2)), (gated, dict(D=P * 9 + 2 - 64 * 32 * 2)), (gated, dict(ldd=80, D=END - 2 - 160)),
    (gated, dict(K=0, D=P * 9)), (gated, dict(KEPT, gate=END - 2, up=P * 10)), (gated, dict(KEPT, up=P * 9 + 2 - 64 * 64 * 2 + 64)),
    (gated, dict(groups=1, D=P * 9 + 6)), (grad, dict(D=END - 2)), (grad, dict(dgate=END - 2, dup=P * 10)),
    (grad, dict(dup=END - 2, dgate=P * 10)), (grad, dict(gate=P * 9, up=P * 9 + 64, dgate=P * 9, dup=P * 9 + 64)),
    (f8, dict(D=END - 2)), (f8, dict(D=P * 9 + 2 - 64 * 160 * 2)), (f8, dict(K=0, D=P * 9)), (f8, dict(out=F32, D=END - 4)),
    (f8, dict(Cp=P * 9, D=P * 9)),
])
def test_results_over_offsets(call, kw):
    assert call(**kw) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are taken would run on these addresses")
@pytest.mark.parametrize("call,kw", [
    (gated, dict(D=END)), (gated, dict(D=P * 9 - 64 * 32 * 2)), (gated, dict(ldd=80, D=END - 160)), (gated, dict(groups=1, D=P * 9 + 8)),
    (grad, dict(D=END)), (f8, dict(D=END)), (f8, dict(D=P * 9 - 64 * 160 * 2)),
])
def test_results_beside_offsets(call, kw):
    assert call(**kw) == 3  # as far as the missing GPU


def test_f8_empty():
    assert f8(groups=0) == 0 and f8(M=0) == 0 and f8(N=0, A=None, B=None, D=None) == 0


def test_other_calls_refuse_the_new_names():
    """SiLU and the 8-bit floats stay unknown to the calls that lack them."""
    assert ttc.ttc_gemm(64, 64, 64, P, 64, R, P * 2, 64, C, None, 64, P * 3, 64, 1.0, 0.0, None, SILU, BF16, None) == INVALID
    assert ttc.ttc_gemm(64, 64, 64, P, 64, R, P * 2, 64, C, None, 64, P * 3, 64, 1.0, 0.0, None, 0, E4M3, None) == INVALID
    assert ttc.ttc_gemm_grouped(4, 64, 32, 48, P, 48, P * 9, P * 3, 48, 32 * 48, C, P * 6, 32, 1.0, None, 0, SILU, BF16, None) == INVALID
    assert ttc.ttc_quantize_rows(8, 64, P, 64, E4M3, P * 3, 64, P * 6, None) == INVALID


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


I32, FL, E4, E5 = torch.int32, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2


@pytest.mark.parametrize("call", [
    lambda: ttc.gemm_gated(t(4, 8, dtype=FL), t(8, 5, dtype=FL), t(8, 5, dtype=FL)),
    lambda: ttc.gemm_gated(t(4, 8), t(7, 5), t(7, 5)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(8, 6)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(5, 8).T),
    lambda: ttc.gemm_gated(t(4, 8), t(2, 8, 5), t(2, 8, 5)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(8, 5), offsets=t(2, dtype=I32)),
    lambda: ttc.gemm_gated(t(4, 8), t(2, 8, 5), t(2, 8, 5), offsets=t(4, dtype=I32)),
    lambda: ttc.gemm_gated(t(4, 8), t(2, 8, 5), t(2, 8, 5), offsets=t(3, dtype=torch.int64)),
    lambda: ttc.gemm_gated(t(4, 8), t(2, 8, 5), t(2, 8, 5), offsets=t(0, dtype=I32)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5, dtype=torch.float16), t(8, 5)),
    lambda: ttc.gemm_gated(t(8, 4).T, t(8, 5), t(8, 5)),
    lambda: ttc.gemm_gated(t(1, 8).expand(4, 8), t(8, 5), t(8, 5)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(8, 5), t(4, 6)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(8, 5), t(5, 4).T),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(8, 5), pre=t(4, 5)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(8, 5), pre=t(3, 10)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(8, 5), pre=t(4, 10, dtype=FL)),
    lambda: ttc.gemm_gated(t(4, 8), t(8, 5), t(8, 5)),  # not on a GPU
    lambda: ttc.gemm_gated_grad(t(4, 8), t(8, 5), t(4, 9)),
    lambda: ttc.gemm_gated_grad(t(4, 8), t(8, 5), t(3, 10)),
    lambda: ttc.gemm_gated_grad(t(4, 8), t(8, 5), t(4, 10), t(4, 12)),
    lambda: ttc.gemm_gated_grad(t(4, 8), t(8, 5), t(4, 10), out=t(4, 6)),
    lambda: ttc.gemm_gated_grad(t(4, 8), t(8, 5), t(10, 4).T),
    lambda: ttc.gemm_gated_grad(t(4, 8), t(8, 5), t(4, 10, dtype=torch.float16)),
    lambda: ttc.gemm_gated_grad(t(4, 8), t(8, 5), t(4, 10), t(4, 10)),  # not on a GPU
    lambda: ttc.quantize_blocks(t(4, 8, dtype=torch.float64)),
    lambda: ttc.quantize_blocks(t(8, 4).T),
    lambda: ttc.quantize_blocks(t(4, 8), block_rows=2),
    lambda: ttc.quantize_blocks(t(4, 8), dtype=torch.int8),
    lambda: ttc.quantize_blocks(t(4, 8), t(4, 7, dtype=E4)),
    lambda: ttc.quantize_blocks(t(4, 8), t(4, 8, dtype=E4), transpose=True),
    lambda: ttc.quantize_blocks(t(4, 8), t(4, 8)),
    lambda: ttc.quantize_blocks(t(4, 8), scale=t(4, 2, dtype=FL)),
    lambda: ttc.quantize_blocks(t(4, 8), scale=t(4, 1)),
    lambda: ttc.gemm_f8_blocks(t(4, 8), t(4, 1, dtype=FL), t(5, 8, dtype=E4), t(5, 1, dtype=FL)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(5, 7, dtype=E4), t(5, 1, dtype=FL)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 2, dtype=FL), t(5, 8, dtype=E4), t(5, 1, dtype=FL)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(5, 8, dtype=E4), t(4, 1, dtype=FL)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1), t(5, 8, dtype=E4), t(5, 1, dtype=FL)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(5, 8, dtype=E4), t(5, 1, dtype=FL), t(4, 5, dtype=I32)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(5, 8, dtype=E4), t(5, 1, dtype=FL), c=t(4, 5, dtype=FL)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(5, 8, dtype=E4), t(5, 1, dtype=FL), c=t(4, 6)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(5, 8, dtype=E4), t(5, 1, dtype=FL), bias=t(4, dtype=FL)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(2, 5, 8, dtype=E4), t(2, 5, 1, dtype=FL)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(2, 5, 8, dtype=E4), t(2, 5, 1, dtype=FL), offsets=t(4, dtype=I32)),
    lambda: ttc.gemm_f8_blocks(t(4, 8, dtype=E4), t(4, 1, dtype=FL), t(5, 8, dtype=E5), t(5, 1, dtype=FL)),  # not on a GPU
])
def test_wrappers_refuse(call):
    with pytest.raises(ValueError):
        call()
