"""CPU-side checks of the grouped and scaled int8 entry points: what they
refuse before any GPU work, and what they take as empty."""
import pytest

import tiled_tensor_core_02_gb300 as ttc
from tiled_tensor_core_02_gb300 import _build

F16, BF16, I8, F32 = (ttc.DTYPE[k] for k in ("f16", "bf16", "i8", "f32"))
R, C = ttc.ROW_MAJOR, ttc.COL_MAJOR
P = 1 << 24  # fake, never-dereferenced addresses, far enough apart
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return ttc.load()


def grouped(groups=4, M=64, N=32, K=48, A=P, lda=None, offsets=P * 9, B=P * 3, ldb=None, strideB=None, layout=C, D=P * 6,
            ldd=None, alpha=1.0, bias=None, strideBias=0, act=0, dtype=BF16):
    lda = max(K, 1) if lda is None else lda
    ldb = max(K if layout == C else N, 1) if ldb is None else ldb
    return ttc.ttc_gemm_grouped(groups, M, N, K, A, lda, offsets, B, ldb, N * K if strideB is None else strideB, layout, D,
                                N if ldd is None else ldd, alpha, bias, strideBias, act, dtype, None)


@pytest.mark.parametrize("kw", [
    dict(groups=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(strideB=-1), dict(strideBias=-1),
    dict(layout=2), dict(act=3), dict(dtype=7), dict(dtype=-1),
    dict(lda=47), dict(ldb=47), dict(layout=R, ldb=31), dict(ldd=31),
    dict(A=None), dict(B=None), dict(D=None), dict(offsets=None),
    dict(A=P + 1), dict(B=P * 3 + 1), dict(D=P * 6 + 1), dict(offsets=P * 9 + 2), dict(bias=P + 2),
    dict(D=P), dict(D=P * 3), dict(D=P + 64 * 48 * 2 - 2), dict(D=P * 3 + 4 * 32 * 48 * 2 - 2),
])
def test_grouped_invalid(kw):
    assert grouped(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=I8), dict(dtype=F32), dict(groups=1025), dict(M=1 << 31), dict(N=1 << 31, ldd=1 << 31),
                                dict(strideB=1 << 41), dict(ldd=1 << 31)])
def test_grouped_unsupported(kw):
    assert grouped(**kw) == UNSUPPORTED


def test_grouped_empty():
    for kw in (dict(groups=0), dict(M=0), dict(N=0), dict(M=0, A=None, B=None, D=None, offsets=None)):
        assert grouped(**kw) == 0


def wgrad(groups=4, M=64, N=32, K=48, A=P, lda=None, B=P * 3, ldb=None, offsets=P * 9, C=None, ldc=None, strideC=None,
          D=P * 6, ldd=None, strideD=None, alpha=1.0, beta=0.0, dtype=BF16, out=F32):
    return ttc.ttc_gemm_grouped_wgrad(groups, M, N, K, A, K if lda is None else lda, B, N if ldb is None else ldb, offsets,
                                      C, N if ldc is None else ldc, N * K if strideC is None else strideC, D,
                                      N if ldd is None else ldd, N * K if strideD is None else strideD, alpha, beta, dtype,
                                      out, None)


@pytest.mark.parametrize("kw", [
    dict(groups=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(strideC=-1), dict(strideD=-1), dict(dtype=9), dict(out=9),
    dict(lda=47), dict(ldb=31), dict(ldd=31), dict(beta=1.0), dict(beta=1.0, C=P * 12, ldc=31),
    dict(A=None), dict(B=None), dict(D=None), dict(offsets=None), dict(D=P * 6 + 2), dict(out=BF16, D=P * 6 + 1),
    dict(beta=1.0, C=P * 12 + 2), dict(A=P + 1), dict(offsets=P * 9 + 1),
    dict(strideD=32 * 48 - 1), dict(ldd=40, strideD=47 * 40 + 31),
    dict(beta=1.0, C=P * 6, ldc=40, strideC=48 * 40), dict(beta=1.0, C=P * 6, strideC=32 * 48 + 4),
    dict(beta=1.0, C=P * 6 + 16), dict(D=P), dict(D=P * 3),
])
def test_wgrad_invalid(kw):
    assert wgrad(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=I8), dict(dtype=F32), dict(out=F16), dict(out=I8), dict(groups=1025),
                                dict(M=1 << 31), dict(strideD=1 << 41)])
def test_wgrad_unsupported(kw):
    assert wgrad(**kw) == UNSUPPORTED


def test_wgrad_empty():
    for kw in (dict(groups=0), dict(N=0), dict(K=0)):
        assert wgrad(**kw) == 0


def quantize(rows=8, cols=64, X=P, ldx=64, dtype=BF16, Q=P * 3, ldq=64, scale=P * 6):
    return ttc.ttc_quantize_rows(rows, cols, X, ldx, dtype, Q, ldq, scale, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=-1), dict(dtype=8), dict(X=None), dict(Q=None), dict(scale=None), dict(ldx=63), dict(ldq=63),
    dict(X=P + 1), dict(dtype=F32, X=P + 2), dict(scale=P * 6 + 2), dict(Q=P), dict(scale=P), dict(scale=P * 3),
])
def test_quantize_invalid(kw):
    assert quantize(**kw) == INVALID


def test_quantize_unsupported_and_empty():
    assert quantize(dtype=I8) == UNSUPPORTED
    assert quantize(rows=1 << 31) == UNSUPPORTED
    assert quantize(rows=0) == 0


def scaled(M=8, N=16, K=64, A=P, lda=None, sa=P * 2, B=P * 3, ldb=None, sb=P * 4, D=P * 6, ldd=16, bias=None, act=0,
           out=BF16, ws=None, nbytes=0):
    return ttc.ttc_gemm_i8_scaled(M, N, K, A, K if lda is None else lda, sa, B, K if ldb is None else ldb, sb, D, ldd, bias,
                                  act, out, ws, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(act=5), dict(out=5), dict(lda=63), dict(ldb=63), dict(ldd=15),
    dict(A=None), dict(B=None), dict(D=None), dict(sa=None), dict(sb=None), dict(sa=P + 2), dict(sb=P + 1), dict(bias=P + 2),
    dict(D=P * 6 + 1), dict(out=F32, D=P * 6 + 2), dict(D=P), dict(D=P * 3),
])
def test_i8_scaled_invalid(kw):
    assert scaled(**kw) == INVALID


def test_i8_scaled_unsupported_and_empty():
    assert scaled(out=I8) == UNSUPPORTED
    assert scaled(K=131072) == UNSUPPORTED
    assert scaled(M=1 << 31) == UNSUPPORTED
    assert scaled(M=0) == 0 and scaled(N=0, A=None, B=None, D=None) == 0


def test_the_first_products_still_refuse_fp32():
    assert ttc.ttc_gemm(64, 64, 64, P, 64, R, P * 2, 64, C, None, 64, P * 3, 64, 1.0, 0.0, None, 0, F32, None) == INVALID
