"""GPU parity of the quantization of rows and of the scaled int8 product."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from operators_util import FLOAT, act64, generator, half_ulp, ok, padded, stream, to64

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- quantization of rows

def quantize_reference(x):
    """The definition in fp32, operation by operation (numpy rounds each to nearest even)."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
        scale = (top / np.float32(127)).astype(np.float32)
        small = scale < np.float32(2.0 ** -126)
        scale = np.where(small, np.float32(0), scale).astype(np.float32)
        inv = np.where(small | ~np.isfinite(scale), np.float32(0), np.float32(1) / np.where(small, 1, scale)).astype(np.float32)
        q = np.rint(np.where(inv[:, None] == 0, 0, (x * inv[:, None]).astype(np.float32)))
    return q.astype(np.int8), scale


def quantize(x, rows, cols, ldx, dtype, ldq=None, shift=0):
    ldq = cols if ldq is None else ldq
    q = torch.full((max(rows * ldq, 1) + 8 + shift,), 55, dtype=torch.int8, device="cuda")
    scale = torch.full((rows,), -1.0, device="cuda")
    ok(ttc.ttc_quantize_rows(rows, cols, x, ldx, ttc.DTYPE[dtype], q.data_ptr() + shift, ldq, scale.data_ptr(), stream()))
    body = q[shift:shift + rows * ldq].view(rows, ldq).cpu().numpy()
    assert (body[:, cols:] == 55).all() and (q[:shift] == 55).all() and (q[shift + rows * ldq:] == 55).all()
    return body[:, :cols], scale.cpu().numpy()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 64), (9, 256), (17, 1000), (300, 1032), (4, 4099), (33, 4096),
                                       (7, 8200), (3, 14336), (2, 20000)])
def test_quantize_rows(rows, cols, dtype):
    gen = generator(rows * 31 + cols)
    buf, x = padded(rows, cols, cols, FLOAT[dtype], gen, scale=3.0)
    q, scale = quantize(buf.data_ptr(), rows, cols, cols, dtype)
    want_q, want_s = quantize_reference(x.float().cpu().numpy())
    assert np.array_equal(scale, want_s)
    assert np.array_equal(q, want_q)
    # what the integers stand for, in 64 bits: half a scale, and 127 roundings' worth of 2^-23 of it
    x64 = to64(x)
    err = np.abs(q * scale[:, None].astype(np.float64) - x64)
    assert (err <= scale[:, None] * (0.5 + 127 * 2.0 ** -22)).all()
    assert np.abs(q).max() == 127


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad_x,pad_q,shift_x,shift_q", [(0, 0, 1, 0), (8, 8, 0, 0), (3, 0, 0, 0), (0, 5, 0, 1), (16, 16, 8, 8)])
def test_quantize_pitches_and_alignment(pad_x, pad_q, shift_x, shift_q, dtype):
    rows, cols = 11, 520
    buf, x = padded(rows, cols, cols + pad_x, FLOAT[dtype], generator(5), offset=shift_x)
    q, scale = quantize(buf.data_ptr() + shift_x * buf.element_size(), rows, cols, cols + pad_x, dtype, cols + pad_q, shift_q)
    want_q, want_s = quantize_reference(x.float().cpu().numpy())
    assert np.array_equal(scale, want_s) and np.array_equal(q, want_q)


@pytest.mark.parametrize("cols", [64, 999, 4096])
def test_quantize_special_rows(cols):
    """Zeros, the least numbers, the largest, a NaN, infinities: see the definition."""
    rows = 9
    x = torch.randn((rows, cols), generator=generator(6), device="cuda")
    x[0] = 0.0
    x[1] = 1e-45
    x[2] = 1e-38          # scale below 2^-126: counts as zeros
    x[3] *= 2.0e-36       # scale just above it
    x[4, cols // 2] = float("nan")
    x[5, cols - 1] = float("-inf")
    x[6] = 3.4e38
    x[7] = -x[7].abs()
    q, scale = quantize(x.data_ptr(), rows, cols, cols, "f32")
    want_q, want_s = quantize_reference(x.cpu().numpy())
    assert np.array_equal(scale, want_s, equal_nan=True) and np.array_equal(q, want_q)
    assert scale[0] == 0 and scale[1] == 0 and scale[2] == 0 and scale[3] > 0
    assert np.isnan(scale[4]) and np.isinf(scale[5]) and (q[[0, 1, 2, 4, 5]] == 0).all()
    assert (q[6] == 127).all()


def test_quantize_many_rows_and_no_columns():
    rows, cols = 70000, 24
    x = torch.randn((rows, cols), generator=generator(7), device="cuda").to(torch.bfloat16)
    q, scale = quantize(x.data_ptr(), rows, cols, cols, "bf16")
    want_q, want_s = quantize_reference(x.float().cpu().numpy())
    assert np.array_equal(scale, want_s) and np.array_equal(q, want_q)
    _, scale = quantize(None, 5, 0, 0, "bf16", 3)
    assert (scale == 0).all()


# ---------------------------------------------------------------- the scaled product

def i8(rows, cols, ld, seed, offset=0, extreme=False):
    rng = np.random.default_rng(seed)
    buf = np.full(offset + rows * ld + 16, 77, dtype=np.int8)
    body = buf[offset:offset + rows * ld].reshape(rows, ld)
    body[:, :cols] = -128 if extreme else rng.integers(-128, 128, (rows, cols), dtype=np.int8)
    return torch.from_numpy(buf).cuda(), body[:, :cols].copy()


def scaled(M, N, K, out="bf16", act="none", bias=True, pad=(0, 0, 0), shift=0, seed=0, extreme=False, workspace="ask",
           unit=False):
    """Runs the product; returns D as float64 and the float64 result with its error bound."""
    lda, ldb, ldd = K + pad[0], K + pad[1], N + pad[2]
    a_dev, a = i8(M, K, max(lda, 1), seed, shift, extreme)
    b_dev, b = i8(N, K, max(ldb, 1), seed + 1, shift, extreme)
    gen = generator(seed)
    sa = torch.ones(M, device="cuda") if unit else 0.01 * torch.exp(torch.randn(M, generator=gen, device="cuda"))
    sb = torch.ones(N, device="cuda") if unit else 0.01 * torch.exp(torch.randn(N, generator=gen, device="cuda"))
    bv = torch.randn(N, generator=gen, device="cuda") if bias else None
    esize = 4 if out == "f32" else 2
    D = torch.full((M * ldd + 8 + shift,), -7.0, dtype=FLOAT[out], device="cuda")
    pa, pb, pd = a_dev.data_ptr() + shift, b_dev.data_ptr() + shift, D.data_ptr() + shift * esize
    need = ttc.ttc_gemm_i8_scaled_workspace_size(M, N, K, pa, max(lda, 1), pb, max(ldb, 1), pd, ldd, ttc.DTYPE[out])
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda") if workspace == "ask" and need else None
    ok(ttc.ttc_gemm_i8_scaled(M, N, K, pa, max(lda, 1), sa.data_ptr(), pb, max(ldb, 1), sb.data_ptr(), pd, ldd,
                              None if bv is None else bv.data_ptr(), ttc.ACT[act], ttc.DTYPE[out],
                              None if ws is None else ws.data_ptr(), 0 if ws is None else need, stream()))
    full = to64(D)
    body = full[shift:shift + M * ldd].reshape(M, ldd)
    assert (body[:, N:] == -7.0).all() and (full[:shift] == -7.0).all() and (full[shift + M * ldd:] == -7.0).all()
    s = a.astype(np.float64) @ b.astype(np.float64).T  # exact: below 2^53
    v = s * to64(sa)[:, None] * to64(sb)[None, :]
    mag = np.abs(v)
    if bv is not None:
        v, mag = v + to64(bv), mag + np.abs(to64(bv))
    want = act64(v, act)
    # the sum is exact; its conversion, two scales and the bias are four roundings, the
    # activation a few more (2^-20 of |v|), then the output's
    tol = 1.13 * 4 * 2.0 ** -24 * mag + (2.0 ** -20 * mag if act == "gelu_tanh" else 0.0) + \
        half_ulp(np.maximum(np.abs(body[:, :N]), np.abs(want)), out)
    return body[:, :N], want, tol, s


def verify(*args, **kw):
    got, want, tol, _ = scaled(*args, **kw)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside the bound, first at {np.argwhere(bad)[0]}: " \
                          f"{got[tuple(np.argwhere(bad)[0])]} against {want[tuple(np.argwhere(bad)[0])]}"


SHAPES = [(1, 1, 1), (1, 4096, 4096), (2, 130, 16), (7, 300, 1000), (8, 128, 4096), (9, 64, 2049), (16, 520, 515),
          (17, 129, 77), (24, 1000, 1024), (32, 256, 256), (33, 300, 520), (64, 512, 1040), (100, 333, 700),
          (130, 1025, 4097), (300, 264, 264), (257, 776, 2064)]


@pytest.mark.parametrize("workspace", ["ask", "none"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, workspace):
    verify(*shape, out="f32", workspace=workspace, seed=sum(shape))


@pytest.mark.parametrize("shape", [(96, 8192, 8192), (128, 520, 4096), (250, 1000, 2048), (48, 776, 16384), (20, 264, 16400),
                                   (10, 136, 32768), (65, 2000, 16384), (3, 14336, 256), (33, 40, 2064)],
                         ids=lambda s: "x".join(map(str, s)))
def test_token_blocks_and_long_reductions(shape):
    """Every block of tokens, K from one stage to many, tiles that fill several
    waves; sums exact, bit for bit."""
    got, _, _, s = scaled(*shape, out="f32", bias=False, unit=True, seed=sum(shape), workspace="none")
    assert np.array_equal(got, s.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh"])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M", [5, 200])
def test_outputs_and_epilogue(M, out, act):
    verify(M, 400, 512, out=out, act=act, seed=3)
    verify(M, 400, 512, out=out, act=act, bias=False, seed=4)


@pytest.mark.parametrize("workspace", ["ask", "none"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 8192), (40, 300, 4096), (600, 600, 3000), (520, 1030, 1500)])
def test_sums_are_exact(M, N, K, workspace):
    """Scales of one and an fp32 result: every sum below 2^24 is the integer, bit for bit."""
    got, _, _, s = scaled(M, N, K, out="f32", bias=False, unit=True, seed=5, workspace=workspace)
    small = np.abs(s) < 2 ** 24
    assert small.any() and np.array_equal(got[small], s[small])
    assert np.array_equal(got, s.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("workspace", ["ask", "none"])
@pytest.mark.parametrize("M,N,K", [(4, 136, 131071), (300, 300, 8192), (520, 520, 5000)])
def test_extremes(M, N, K, workspace):
    """-128 everywhere: every 1024 of K add up to 2^24, the largest sums are just inside int32."""
    got, _, _, s = scaled(M, N, K, out="f32", bias=False, unit=True, seed=6, extreme=True, workspace=workspace)
    assert np.array_equal(got, s.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M", [6, 300])
@pytest.mark.parametrize("pad,shift", [((1, 3, 5), 0), ((16, 32, 8), 0), ((0, 0, 0), 1), ((16, 16, 16), 16), ((8, 4, 2), 2)])
def test_pitches_and_alignment(pad, shift, M, out):
    verify(M, 330, 528, out=out, pad=pad, shift=shift, seed=7)


def test_no_reduction_and_poisoned_rows():
    """K == 0 leaves act(bias); a token whose scale is NaN or infinite gets no number, the others theirs."""
    verify(5, 40, 0, out="bf16", act="relu", seed=8)
    for M in (6, 300):
        K, N = 512, 300
        _, a = i8(M, K, K, 9)
        x = torch.from_numpy(a.astype(np.float32)).cuda()
        x[2, 7] = float("nan")
        x[4, 9] = float("inf")
        q = torch.empty((M, K), dtype=torch.int8, device="cuda")
        sa = torch.empty(M, device="cuda")
        ok(ttc.ttc_quantize_rows(M, K, x.data_ptr(), K, ttc.DTYPE["f32"], q.data_ptr(), K, sa.data_ptr(), stream()))
        b_dev, _ = i8(N, K, K, 10)
        sb = torch.ones(N, device="cuda")
        D = torch.zeros((M, N), device="cuda")
        need = ttc.ttc_gemm_i8_scaled_workspace_size(M, N, K, q.data_ptr(), K, b_dev.data_ptr(), K, D.data_ptr(), N,
                                                     ttc.DTYPE["f32"])
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        ok(ttc.ttc_gemm_i8_scaled(M, N, K, q.data_ptr(), K, sa.data_ptr(), b_dev.data_ptr(), K, sb.data_ptr(),
                                  D.data_ptr(), N, None, 0, ttc.DTYPE["f32"], ws.data_ptr(), need, stream()))
        bad = ~torch.isfinite(D).cpu().numpy()
        assert bad[[2, 4]].all() and not np.delete(bad, [2, 4], axis=0).any()


def test_quantized_product_against_the_float_one():
    """Rows quantized, multiplied and scaled back: against the 64-bit product of
    what the integers stand for, and within the quantization's own error of the
    product of the unquantized operands."""
    M, N, K = 70, 260, 512
    gen = generator(11)
    x = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((N, K), generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    parts = []
    for t, rows in ((x, M), (w, N)):
        q = torch.empty((rows, K), dtype=torch.int8, device="cuda")
        s = torch.empty(rows, device="cuda")
        ok(ttc.ttc_quantize_rows(rows, K, t.data_ptr(), K, ttc.DTYPE["bf16"], q.data_ptr(), K, s.data_ptr(), stream()))
        parts += [q, s]
    qx, sx, qw, sw = parts
    D = torch.empty((M, N), device="cuda")
    ok(ttc.ttc_gemm_i8_scaled(M, N, K, qx.data_ptr(), K, sx.data_ptr(), qw.data_ptr(), K, sw.data_ptr(), D.data_ptr(), N,
                              None, 0, ttc.DTYPE["f32"], None, 0, stream()))
    vx, vw = to64(qx) * to64(sx)[:, None], to64(qw) * to64(sw)[:, None]
    got = to64(D)
    assert (np.abs(got - vx @ vw.T) <= 2.0 ** -21 * (np.abs(vx) @ np.abs(vw).T)).all()
    ex, ew = 0.5001 * to64(sx)[:, None] * np.ones_like(vx), 0.5001 * to64(sw)[:, None] * np.ones_like(vw)
    bound = ex @ np.abs(to64(w)).T + np.abs(to64(x)) @ ew.T + ex @ ew.T + 2.0 ** -20 * (np.abs(vx) @ np.abs(vw).T)
    assert (np.abs(got - to64(x) @ to64(w).T) <= bound).all()


def test_side_stream_and_graph():
    M, N, K = 12, 300, 1024
    a_dev, _ = i8(M, K, K, 12)
    b_dev, _ = i8(N, K, K, 13)
    sa, sb = torch.full((M,), 0.01, device="cuda"), torch.full((N,), 0.02, device="cuda")
    outs = [torch.zeros((M, N), device="cuda") for _ in range(3)]

    def call(out):
        return ttc.ttc_gemm_i8_scaled(M, N, K, a_dev.data_ptr(), K, sa.data_ptr(), b_dev.data_ptr(), K, sb.data_ptr(),
                                      out.data_ptr(), N, None, 0, ttc.DTYPE["f32"], None, 0, stream())

    ok(call(outs[0]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ok(call(outs[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert call(outs[2]) == 0
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# Sizes between the kernels: token blocks of 128 and few channels, many tokens with
# and without the copies, rows that TMA cannot read on either side of their limit.
@pytest.mark.parametrize("workspace", ["ask", "none"])
@pytest.mark.parametrize("M,N,K", [(320, 520, 2048), (1024, 2056, 512), (700, 4096, 1040), (1100, 4099, 2048), (128, 1000, 333),
                                   (129, 1000, 333), (2050, 136, 128)])
def test_between_the_kernels(M, N, K, workspace):
    for out in ("f32", "f16", "bf16"):
        verify(M, N, K, out=out, act="relu", workspace=workspace, seed=M)


@pytest.mark.parametrize("M,N,K", [(1100, 4099, 2048), (2050, 4097, 1024)])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_columns_behind_the_last_whole_vector(M, N, K, out):
    verify(M, N, K, out=out, pad=(0, 0, -N % 8), seed=N)
