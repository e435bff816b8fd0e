"""GPU parity of the products grouped by expert and of their weights' gradient
against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from operators_util import FLOAT, act64, check, clamp_offsets, generator, ok, padded, stream, to64

pytestmark = pytest.mark.gpu


class Grouped:
    """One grouped product: operands with NaN in every padding element."""

    def __init__(self, offsets, M, N, K, dtype="bf16", layout="col", seed=0, bias=True, pad=(0, 0, 0), shift=0,
                 shared=False, gap=0):
        gen = generator(seed)
        self.G, self.M, self.N, self.K, self.dtype, self.layout = len(offsets) - 1, M, N, K, dtype, layout
        self.raw = list(offsets)
        self.lda, self.ldd = K + pad[0], N + pad[2]
        br, bc = (N, K) if layout == "col" else (K, N)
        self.ldb = bc + pad[1]
        self.strideB = 0 if shared else br * self.ldb + gap
        self.abuf, self.A = padded(M, K, max(self.lda, 1), FLOAT[dtype], gen, offset=shift)
        nB = 1 if shared else self.G
        self.bbuf = torch.full((shift + max(nB - 1, 0) * self.strideB + max(br * self.ldb, 1) + 8,), float("nan"),
                               dtype=FLOAT[dtype], device="cuda")
        self.B = []
        for g in range(nB):
            v = self.bbuf[shift + g * self.strideB:shift + g * self.strideB + br * self.ldb].view(br, self.ldb)[:, :bc]
            v.copy_(torch.randn((br, bc), generator=gen, device="cuda") / max(K, 1) ** 0.5)
            self.B.append(v)
        self.bias = torch.randn((self.G, N), generator=gen, device="cuda") if bias else None
        self.offsets = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        self.shift = shift

    def b64(self, g):
        b = to64(self.B[0 if len(self.B) == 1 else g])
        return b.T if self.layout == "col" else b

    def call(self, act="none", alpha=1.0, fill=-7.0, s=None):
        self.dbuf = torch.full((self.shift + self.M * self.ldd + 8,), fill, dtype=FLOAT[self.dtype], device="cuda")
        e = 2
        ok(ttc.ttc_gemm_grouped(
            self.G, self.M, self.N, self.K, self.abuf.data_ptr() + self.shift * e, max(self.lda, 1),
            self.offsets.data_ptr(), self.bbuf.data_ptr() + self.shift * e, max(self.ldb, 1), self.strideB,
            ttc.COL_MAJOR if self.layout == "col" else ttc.ROW_MAJOR, self.dbuf.data_ptr() + self.shift * e, self.ldd,
            alpha, None if self.bias is None else self.bias.data_ptr(), self.N, ttc.ACT[act], ttc.DTYPE[self.dtype],
            stream() if s is None else s))
        return self.dbuf[self.shift:self.shift + self.M * self.ldd].view(self.M, self.ldd)

    def verify(self, act="none", alpha=1.0, fill=-7.0):
        d = self.call(act, alpha, fill)
        got, a = to64(d), to64(self.A)
        covered = np.zeros(self.M, dtype=bool)
        for g, (lo, hi) in enumerate(clamp_offsets(self.raw, self.M)):
            if hi == lo:
                continue
            b = self.b64(g)
            want, s_abs = alpha * (a[lo:hi] @ b), abs(alpha) * (np.abs(a[lo:hi]) @ np.abs(b))
            if self.bias is not None:
                bias = to64(self.bias[g])
                want, s_abs = want + bias, s_abs + np.abs(bias)
            check(got[lo:hi, :self.N], act64(want, act), s_abs, self.K, self.dtype)
            covered[lo:hi] = True
        assert (got[~covered] == fill).all(), "rows of no group were written"
        assert (got[:, self.N:] == fill).all(), "the pitch padding was written"
        assert (to64(self.dbuf[:self.shift]) == fill).all() and \
            (to64(self.dbuf[self.shift + self.M * self.ldd:]) == fill).all()


def ends(sizes):
    return [0] + list(np.cumsum(sizes))


# sizes of the groups: one token, none at all, all in one, ragged around the
# tiles' edges, more groups than rows
PATTERNS = {
    "one": [1], "empty_first_last": [0, 5, 0, 0, 3, 0], "all_in_one": [0, 0, 260, 0],
    "edges": [127, 128, 129, 1, 255, 256, 257, 0, 16, 15, 17], "ones": [1] * 40, "sparse": [0] * 50 + [2] + [0] * 30 + [1],
}


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pattern", sorted(PATTERNS))
def test_group_sizes(pattern, dtype, layout):
    o = ends(PATTERNS[pattern])
    Grouped(o, o[-1], 264, 200, dtype, layout, seed=len(pattern)).verify()


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("n,k", [(1, 1), (8, 16), (7, 333), (129, 64), (256, 63), (300, 65), (520, 1000), (1024, 8),
                                 (31, 2048), (136, 4096)])
def test_widths(n, k, layout):
    o = ends([3, 70, 0, 1, 130])
    Grouped(o, o[-1], n, k, "bf16", layout, seed=n + k).verify("none", 1.0)


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh"])
@pytest.mark.parametrize("alpha", [1.0, -0.5])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_epilogue(dtype, alpha, act):
    o = ends([40, 0, 300, 7])
    Grouped(o, o[-1], 272, 320, dtype, "col", seed=3).verify(act, alpha)
    Grouped(o, o[-1], 272, 320, dtype, "row", seed=4, bias=False).verify(act, alpha)


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("pad,shift,gap", [((3, 5, 7), 0, 0), ((8, 16, 24), 0, 64), ((0, 0, 0), 1, 3), ((8, 8, 8), 8, 4)])
def test_pitches_and_alignment(pad, shift, gap, layout):
    """Odd and padded pitches, bases off the 16-byte boundary, groups whose B
    starts off it; NaN in every padding element."""
    o = ends([33, 1, 0, 140])
    Grouped(o, o[-1], 272, 264, "bf16", layout, seed=9, pad=pad, shift=shift, gap=gap).verify("relu")


def test_shared_weights_and_no_reduction():
    o = ends([5, 0, 60])
    Grouped(o, o[-1], 96, 128, "f16", "col", seed=5, shared=True).verify()
    Grouped(o, o[-1], 96, 0, "bf16", "col", seed=6).verify("gelu_tanh")


@pytest.mark.parametrize("offsets", [[2, 9, 20], [-5, 4, 1000], [0, 30, 12, 40], [50, 50, 50], [64, 0]])
def test_offsets_that_leave_rows_out_or_the_matrix(offsets):
    """Rows of no group stay as they were; offsets beyond the matrix count as
    its end, descending ones as an empty group.  (Where a later group starts
    inside an earlier one the shared rows are undefined: not looked at.)"""
    p = Grouped(offsets, 50, 136, 72, "bf16", "col", seed=11)
    if offsets == [0, 30, 12, 40]:
        d = to64(p.call())
        a = to64(p.A)
        for g, (lo, hi) in ((0, (0, 12)), (2, (30, 40))):
            b, bias = p.b64(g), to64(p.bias[g])
            check(d[lo:hi], a[lo:hi] @ b + bias, np.abs(a[lo:hi]) @ np.abs(b) + np.abs(bias), p.K, "bf16")
        assert (d[40:] == -7.0).all()
    else:
        p.verify()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("layout", ["col", "row"])
def test_other_groups_rows_and_weights_do_not_leak(layout, value):
    """A NaN or infinity in one group's rows and weights reaches its own rows only."""
    o = ends([20, 30, 130, 9])
    p = Grouped(o, o[-1], 136, 200, "bf16", layout, seed=12)
    clean = to64(p.call()).copy()
    p.A[20:50] = value
    p.B[1].fill_(value)
    dirty = to64(p.call())
    keep = np.r_[0:20, 50:o[-1]]
    assert np.array_equal(dirty[keep], clean[keep])
    assert not np.isfinite(dirty[20:50]).any()


def test_most_groups():
    sizes = [(7 * i) % 3 for i in range(1024)]
    o = ends(sizes)
    Grouped(o, o[-1], 40, 72, "bf16", "col", seed=13).verify()


def test_large_groups_take_many_tiles():
    o = ends([700, 0, 1500, 333])
    for layout in ("col", "row"):
        Grouped(o, o[-1], 1040, 328, "bf16", layout, seed=14).verify("gelu_tanh")


def test_side_stream_and_graph():
    """On a stream of its own, and replayed from a graph after new offsets were
    written to the same place."""
    o = ends([10, 0, 90, 3])
    p = Grouped(o, o[-1], 264, 264, "bf16", "col", seed=15)
    want = p.call().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert torch.equal(p.call(s=s.cuda_stream), want)
    torch.cuda.synchronize()
    out = torch.zeros((p.M, p.ldd), dtype=FLOAT["bf16"], device="cuda")
    args = (p.G, p.M, p.N, p.K, p.abuf.data_ptr(), p.lda, p.offsets.data_ptr(), p.bbuf.data_ptr(), p.ldb, p.strideB,
            ttc.COL_MAJOR, out.data_ptr(), p.ldd, 1.0, p.bias.data_ptr(), p.N, 0, ttc.DTYPE["bf16"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert ttc.ttc_gemm_grouped(*args, stream()) == 0
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    q = Grouped(ends([50, 20, 30, 3]), p.M, 264, 264, "bf16", "col", seed=15)
    p.offsets.copy_(q.offsets)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, q.call())


# ---------------------------------------------------------------- the weights' gradient

class Wgrad:
    def __init__(self, offsets, M, N, K, dtype="bf16", out="f32", seed=0, beta=0.0, pad=(0, 0, 0, 0), shift=0, gap=0):
        gen = generator(seed)
        self.G, self.M, self.N, self.K, self.dtype, self.out, self.beta = len(offsets) - 1, M, N, K, dtype, out, beta
        self.raw, self.shift = list(offsets), shift
        self.lda, self.ldb, self.ldc, self.ldd = K + pad[0], N + pad[1], N + pad[2], N + pad[3]
        self.abuf, self.A = padded(M, K, self.lda, FLOAT[dtype], gen, offset=shift)
        self.bbuf, self.B = padded(M, N, self.ldb, FLOAT[dtype], gen, offset=shift)
        self.strideC, self.strideD = K * self.ldc + gap, K * self.ldd + gap
        self.cbuf = torch.full((self.G * self.strideC,), float("nan"), dtype=FLOAT[out], device="cuda")
        for g in range(self.G):
            self.block(self.cbuf, g, self.strideC, self.ldc)[:, :N].copy_(torch.randn((K, N), generator=gen, device="cuda"))
        self.offsets = torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def block(self, buf, g, stride, ld):
        return buf[g * stride:g * stride + self.K * ld].view(self.K, ld)

    def call(self, alpha=1.0, in_place=False, fill=-7.0):
        e = 2
        if in_place:
            self.dbuf = self.cbuf.clone()
            c, ldd, strideD = self.dbuf, self.ldc, self.strideC
        else:
            self.dbuf = torch.full((self.G * self.strideD,), fill, dtype=FLOAT[self.out], device="cuda")
            c, ldd, strideD = self.cbuf, self.ldd, self.strideD
        ok(ttc.ttc_gemm_grouped_wgrad(
            self.G, self.M, self.N, self.K, self.abuf.data_ptr() + self.shift * e, self.lda,
            self.bbuf.data_ptr() + self.shift * e, self.ldb, self.offsets.data_ptr(),
            c.data_ptr() if self.beta else None, self.ldc, self.strideC, self.dbuf.data_ptr(), ldd, strideD, alpha,
            self.beta, ttc.DTYPE[self.dtype], ttc.DTYPE[self.out], stream()))
        return [self.block(self.dbuf, g, strideD, ldd) for g in range(self.G)]

    def verify(self, alpha=1.0, in_place=False, fill=-7.0):
        d = self.call(alpha, in_place, fill)
        a, b = to64(self.A), to64(self.B)
        for g, (lo, hi) in enumerate(clamp_offsets(self.raw, self.M)):
            want, s_abs = alpha * (a[lo:hi].T @ b[lo:hi]), abs(alpha) * (np.abs(a[lo:hi]).T @ np.abs(b[lo:hi]))
            if self.beta:
                c = to64(self.block(self.cbuf, g, self.strideC, self.ldc)[:, :self.N])
                want, s_abs = want + self.beta * c, s_abs + np.abs(self.beta * c)
            got = to64(d[g])
            check(got[:, :self.N], want, s_abs, hi - lo, self.out, slope=1.0)
            pad = got[:, self.N:]
            assert np.isnan(pad).all() if in_place else (pad == fill).all(), "the pitch padding was written"


@pytest.mark.parametrize("out", ["f32", "same"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pattern", sorted(PATTERNS))
def test_wgrad_group_sizes(pattern, dtype, out):
    o = ends(PATTERNS[pattern])
    Wgrad(o, o[-1], 136, 200, dtype, dtype if out == "same" else out, seed=len(pattern)).verify()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n,k", [(1, 1), (8, 7), (64, 129), (257, 40), (300, 256), (520, 264), (1000, 24)])
def test_wgrad_widths(n, k, out):
    o = ends([3, 64, 0, 1, 129])
    Wgrad(o, o[-1], n, k, "bf16", out, seed=n + k).verify()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [264, 261])
def test_wgrad_adds_to_what_is_there(n, in_place, out):
    """beta C, an empty group among them, into another array or in place."""
    o = ends([50, 0, 200])
    Wgrad(o, o[-1], n, 136, "bf16", out, seed=21, beta=1.0).verify(0.5, in_place)
    Wgrad(o, o[-1], n, 136, "bf16", out, seed=22, beta=-0.25, pad=(0, 0, 8, 8)).verify(1.0, in_place)


@pytest.mark.parametrize("pad,shift,gap", [((3, 5, 7, 1), 0, 0), ((8, 16, 24, 8), 0, 64), ((0, 0, 0, 0), 1, 3),
                                           ((8, 8, 8, 8), 8, 4)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_wgrad_pitches_and_alignment(out, pad, shift, gap):
    o = ends([33, 1, 0, 140])
    Wgrad(o, o[-1], 136, 264, "bf16", out, seed=23, beta=1.0, pad=pad, shift=shift, gap=gap).verify()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("sizes", [[20, 30, 131, 9], [64, 1, 63, 17]])
def test_wgrad_rows_of_other_groups_do_not_leak(sizes, value):
    """The last k-block of a group reaches into the next group's rows: a NaN or
    an infinity there, or in rows of no group, must not reach its sums."""
    o = ends(sizes)
    M = o[-1] + 40  # rows of no group behind the last one
    p = Wgrad(o, M, 264, 272, "bf16", "f32", seed=24)
    clean = [to64(x).copy() for x in p.call()]
    for t in (p.A, p.B):
        t[o[1]:o[2]] = value
        t[o[-1]:] = value
    dirty = [to64(x) for x in p.call()]
    for g in (0, 2, 3):
        assert np.array_equal(dirty[g], clean[g])
    assert not np.isfinite(dirty[1]).any()


def test_wgrad_large():
    o = ends([1000, 0, 2100, 333, 1])
    Wgrad(o, o[-1], 776, 520, "bf16", "f32", seed=25, beta=1.0).verify()
    Wgrad(o, o[-1], 520, 776, "f16", "f16", seed=26).verify()


def test_wgrad_no_rows_and_offsets_outside():
    for offsets, M in (([0, 0, 0], 0), ([-3, 10, 99], 30), ([5, 2, 20], 30)):
        Wgrad(offsets, M, 136, 72, "bf16", "f32", seed=27, beta=1.0).verify()


def test_gradients_against_differences():
    """L = sum(G * forward(A, B)): the kernels' gradients of A and B against
    central differences of the 64-bit forward along random directions.  L is
    linear in each, so differences are exact but for 64-bit rounding; the
    kernels' errors are bounded term by term."""
    o = ends([6, 0, 17, 40])
    M, N, K = o[-1], 72, 56
    p = Grouped(o, M, N, K, "bf16", "row", seed=31, bias=False)
    gen = generator(32)
    G = torch.randn((M, N), generator=gen, device="cuda").to(torch.bfloat16)
    dA = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    dB = torch.empty((p.G, K, N), device="cuda")
    # the forward's weights are K x N row-major; the gradient of A reads them as N x K column-major
    ok(ttc.ttc_gemm_grouped(p.G, M, K, N, G.data_ptr(), N, p.offsets.data_ptr(), p.bbuf.data_ptr(), N, K * N,
                            ttc.COL_MAJOR, dA.data_ptr(), K, 1.0, None, 0, 0, ttc.DTYPE["bf16"], stream()))
    ok(ttc.ttc_gemm_grouped_wgrad(p.G, M, N, K, p.abuf.data_ptr(), K, G.data_ptr(), N, p.offsets.data_ptr(), None, N,
                                  K * N, dB.data_ptr(), N, K * N, 1.0, 0.0, ttc.DTYPE["bf16"], ttc.DTYPE["f32"],
                                  stream()))
    a, b, g64 = to64(p.A), [p.b64(g) for g in range(p.G)], to64(G)

    def loss(a, b):
        return sum(float((g64[lo:hi] * (a[lo:hi] @ b[g])).sum()) for g, (lo, hi) in enumerate(clamp_offsets(o, M)))

    rng = np.random.default_rng(33)
    got_a, got_b = to64(dA), to64(dB)
    for _ in range(4):
        va = rng.standard_normal(a.shape)
        vb = [rng.standard_normal(x.shape) for x in b]
        da = (loss(a + va, b) - loss(a - va, b)) / 2.0
        db = (loss(a, [x + v for x, v in zip(b, vb)]) - loss(a, [x - v for x, v in zip(b, vb)])) / 2.0
        tol_a = tol_b = 1e-9
        for g, (lo, hi) in enumerate(clamp_offsets(o, M)):
            s = np.abs(g64[lo:hi]) @ np.abs(b[g]).T
            tol_a += float((np.abs(va[lo:hi]) * (2 * N * 2.0 ** -24 * s + 2.0 ** -8 * np.abs(got_a[lo:hi]))).sum())
            s = np.abs(a[lo:hi]).T @ np.abs(g64[lo:hi])
            tol_b += float((np.abs(vb[g]) * (2 * (hi - lo) + 1) * 2.0 ** -24 * s).sum())
        assert abs((got_a * va).sum() - da) <= tol_a
        assert abs(sum((got_b[g] * vb[g]).sum() for g in range(p.G)) - db) <= tol_b


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n,pad", [(261, 3), (258, 6), (390, 10), (7, 1), (1021, 3)])
def test_wgrad_columns_behind_the_last_whole_vector(n, pad, out):
    """Widths that end inside a 16-byte vector, rows that start on one; half a tile
    or more lies behind the last column."""
    for in_place in (False, True):
        Wgrad([0, 130, 130, 700], 700, n, 300, out=out, beta=1.0, pad=(4, pad, pad, pad), seed=n).verify(in_place=in_place)
    Wgrad([0, 130, 130, 700], 700, n, 300, out=out, pad=(4, pad, pad, pad), seed=n).verify(alpha=0.5)


@pytest.mark.parametrize("n,pad", [(261, 3), (390, 10), (1021, 3)])
def test_columns_behind_the_last_whole_vector(n, pad):
    for layout in ("row", "col"):
        Grouped([0, 130, 130, 700], 700, n, 320, layout=layout, pad=(0, pad if layout == "row" else 0, pad), seed=n).verify()


@pytest.mark.parametrize("beta", [1.0, 0.5])
@pytest.mark.parametrize("n,ldd", [(264, 264), (261, 264), (520, 523)])
def test_wgrad_in_place_and_apart_agree(n, ldd, beta):
    """fp32 gradients added to in place and out of it differ by roundings only; the
    padding stays as it is."""
    M, K, groups = 700, 300, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    a = torch.randn((M, K + 4), generator=g, device="cuda").bfloat16()[:, :K]
    b = torch.randn((M, -(-n // 8) * 8), generator=g, device="cuda").bfloat16()[:, :n]
    offsets = torch.tensor([0, 130, 130, 700], dtype=torch.int32, device="cuda")
    first = torch.randn((groups, K, ldd), generator=g, device="cuda")
    buf = first.clone()
    ttc.gemm_grouped_wgrad(a, b, offsets, c=buf[:, :, :n], out=buf[:, :, :n], beta=beta)
    apart = ttc.gemm_grouped_wgrad(a, b, offsets, c=first[:, :, :n], beta=beta)
    assert torch.equal(buf[:, :, n:], first[:, :, n:])
    assert torch.equal(buf[1, :, :n], beta * first[1, :, :n])  # an empty group
    # the partial sums are the same; C joins them first or last, a rounding of each partial result either
    # way, and of 570 products of normal values none is near 200
    size = apart.abs().double() + first[:, :, :n].abs().double() + 200.0
    assert ((buf[:, :, :n].double() - apart.double()).abs() <= 8 * 2.0 ** -24 * size).all()
