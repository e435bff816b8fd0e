"""GPU parity of the block-scaled 8-bit floats: the quantizer bit for bit against its
definition, the product against a plain 64-bit implementation."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from feed_forward_util import F8, TOP, f8_bound, f8_exact, f8_product, quantize64, within
from operators_util import FLOAT, act64, clamp_offsets, generator, ok, stream, to64

pytestmark = pytest.mark.gpu
CODE = {"e4m3": ttc.DTYPE["f8_e4m3"], "e5m2": ttc.DTYPE["f8_e5m2"]}


# ------------------------------------------------------------------ quantizer

def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def quantize(x, view_ld, rows, cols, dtype, q, block, turn, ldq_pad=0, lds_pad=0, shift=0):
    r, c = (cols, rows) if turn else (rows, cols)
    ldq, lds = c + ldq_pad, -(-c // 128) + lds_pad
    qbuf = torch.full((shift + r * ldq + 16,), 0x5A, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((-(-r // block) * lds + 4,), -3.0, device="cuda")
    ok(ttc.ttc_quantize_blocks(rows, cols, x, view_ld, ttc.DTYPE[dtype], block, int(turn), qbuf.data_ptr() + shift, ldq, CODE[q],
                               sbuf.data_ptr(), lds, stream()))
    got = qbuf[shift:shift + r * ldq].view(r, ldq)
    assert (got[:, c:] == 0x5A).all() and (qbuf[:shift] == 0x5A).all() and (qbuf[shift + r * ldq:] == 0x5A).all()
    s = sbuf[:-(-r // block) * lds].view(-(-r // block), lds)
    assert (s[:, -(-c // 128):] == -3.0).all() and (sbuf[-4:] == -3.0).all()
    return got[:, :c], s[:, :-(-c // 128)]


def compare(x, got, q, block, turn):
    want, scale = quantize64(x, q, block, turn)
    assert torch.equal(got[1].cpu().contiguous().view(torch.int32), scale.contiguous().view(torch.int32)) or \
        torch.equal(torch.nan_to_num(got[1].cpu(), nan=-5.0), torch.nan_to_num(scale, nan=-5.0))
    assert torch.equal(bits(got[0]), bits(want))


@pytest.mark.parametrize("q", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block,turn", [(1, False), (128, False), (1, True), (128, True)])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 127), (129, 129), (5, 1024), (256, 8), (130, 1100), (16, 4096),
                                       (300, 333), (128, 128)])
def test_quantize(rows, cols, block, turn, dtype, q):
    gen = generator(rows + cols)
    x = (torch.randn((rows, cols), generator=gen, device="cuda") * torch.exp(2.0 * torch.randn((rows, 1), generator=gen, device="cuda"))).to(FLOAT[dtype])
    compare(x, quantize(x.data_ptr(), cols, rows, cols, dtype, q, block, turn), q, block, turn)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block,turn", [(1, False), (128, False), (1, True), (128, True)])
@pytest.mark.parametrize("pad,shift", [((8, 8, 0), 0), ((8, 16, 3), 0), ((3, 5, 1), 0), ((8, 8, 0), 1), ((8, 8, 0), 8)])
def test_quantize_pitches(pad, shift, block, turn, dtype):
    rows, cols = 200, 392
    gen = generator(5)
    ld = cols + pad[0]
    buf = torch.full((shift + rows * ld,), float("nan"), dtype=FLOAT[dtype], device="cuda")
    x = buf[shift:].view(rows, ld)[:, :cols]
    x.copy_(torch.randn((rows, cols), generator=gen, device="cuda"))
    got = quantize(buf.data_ptr() + shift * buf.element_size(), ld, rows, cols, dtype, "e4m3", block, turn, pad[1], pad[2], shift)
    compare(x, got, "e4m3", block, turn)


@pytest.mark.parametrize("q", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block,turn", [(1, False), (128, False), (1, True), (128, True)])
def test_quantize_extremes(block, turn, q):
    """Zeros, the least and the largest numbers, NaN, infinities, each in blocks of their own."""
    big = torch.finfo(torch.float32).max
    rows = [[0.0], [1e-38, -3e-39], [1.2e-38], [2.0 ** -126 * TOP[q]], [2.0 ** -127 * TOP[q]], [big, -big, 1.0], [float("nan"), 1.0],
            [float("inf"), 2.0], [-float("inf")], [1.0, 2.0 ** -20], [-0.0], [TOP[q], TOP[q] / 2, 1.0]]
    x = torch.zeros((128 * len(rows), 256), device="cuda")
    for i, v in enumerate(rows):
        x[i * 128 + 5, 3:3 + len(v)] = torch.tensor(v)
        x[i * 128 + 9, 130:130 + len(v)] = torch.tensor(v)
    if turn:
        x = x.t().contiguous()
    compare(x, quantize(x.data_ptr(), x.shape[1], x.shape[0], x.shape[1], "f32", q, block, turn), q, block, turn)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_square_blocks_of_a_transpose_hold_the_same_values(dtype):
    x = torch.randn((300, 500), generator=generator(8), device="cuda").to(FLOAT[dtype])
    q, s = ttc.quantize_blocks(x, block_rows=128)
    t, st = ttc.quantize_blocks(x, block_rows=128, transpose=True)
    assert torch.equal(bits(q.t()), bits(t)) and torch.equal(s.t(), st)


# ------------------------------------------------------------------ product

class Product:
    """Operands with 0x7F (a NaN of both formats) in every padding byte, NaN in padding scales."""

    def __init__(self, offsets, M, N, K, ta="e4m3", tb="e4m3", block=128, seed=0, pad=(0, 0, 0, 0), shift=0, gap=0, bias=False,
                 align=True, negative=False):
        gen = generator(seed)
        self.raw, self.G = offsets, 1 if offsets is None else len(offsets) - 1
        self.M, self.N, self.K, self.ta, self.tb, self.block, self.shift = M, N, K, ta, tb, block, shift
        up = (lambda v: -(-v // 16) * 16) if align else (lambda v: v)
        self.lda, self.ldb = max(up(K) + pad[0], 1), max(up(K) + pad[1], 1)
        self.kb, self.sbr = -(-K // 128), -(-N // block)
        self.ldsa, self.ldsb = self.kb + pad[2], self.kb + pad[3]
        self.strideB, self.strideSB = N * self.ldb + gap, self.sbr * self.ldsb + (3 if gap else 0)
        self.abuf, self.A = self.values(1, M, self.lda, M * self.lda, ta, gen)
        self.bbuf, self.B = self.values(self.G, N, self.ldb, self.strideB, tb, gen)
        self.sabuf, self.SA = self.scales(1, M, self.ldsa, 0, gen, 1.0, negative)
        self.sbbuf, self.SB = self.scales(self.G, self.sbr, self.ldsb, self.strideSB, gen, 1.0 / (TOP[ta] * TOP[tb] * max(K, 1) ** 0.5) * 16, negative)
        self.bias = torch.randn((self.G, N), generator=gen, device="cuda") if bias else None
        self.offsets = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def values(self, count, rows, ld, stride, kind, gen):
        buf = torch.full((self.shift + count * stride + 16,), 0x7F, dtype=torch.uint8, device="cuda")
        out = []
        for i in range(count):
            v = buf[self.shift + i * stride:self.shift + i * stride + rows * ld].view(rows, ld)[:, :self.K]
            r = torch.randn((rows, self.K), generator=gen, device="cuda") * (TOP[kind] / 4)
            v.copy_(r.clamp(-TOP[kind], TOP[kind]).to(F8[kind]).view(torch.uint8))
            out.append(v)
        return buf, out

    def scales(self, count, rows, ld, stride, gen, size, negative):
        stride = stride or rows * ld
        buf = torch.full((count * stride + 4,), float("nan"), device="cuda")
        out = []
        for i in range(count):
            v = buf[i * stride:i * stride + rows * ld].view(rows, ld)[:, :self.kb]
            s = torch.exp(0.7 * torch.randn((rows, self.kb), generator=gen, device="cuda")) * size
            v.copy_(s * torch.where(torch.rand((rows, self.kb), generator=gen, device="cuda") < 0.3, -1.0, 1.0) if negative else s)
            out.append(v)
        return buf, out

    def groups(self):
        return [(0, 0, self.M)] if self.raw is None else [(g, lo, hi) for g, (lo, hi) in enumerate(clamp_offsets(self.raw, self.M))]

    def call(self, out="bf16", act="none", C=None, ldc=None, d=None, ldd=None, d_shift=0, fill=-7.0, s=None):
        self.ldd = self.N if ldd is None else ldd
        self.d = torch.full((d_shift + self.M * self.ldd + 8,), fill, dtype=FLOAT[out], device="cuda") if d is None else d
        e = self.d.element_size()
        ok(ttc.ttc_gemm_f8_blocks(
            self.G, self.M, self.N, self.K, self.abuf.data_ptr() + self.shift, self.lda, CODE[self.ta], self.sabuf.data_ptr(), self.ldsa,
            None if self.offsets is None else self.offsets.data_ptr(), self.bbuf.data_ptr() + self.shift, self.ldb, self.strideB,
            CODE[self.tb], self.sbbuf.data_ptr(), self.ldsb, self.strideSB, self.block, None if C is None else C.data_ptr(),
            self.ldd if ldc is None else ldc, self.d.data_ptr() + d_shift * e, self.ldd, None if self.bias is None else self.bias.data_ptr(),
            self.N, ttc.ACT[act], ttc.DTYPE[out], stream() if s is None else s))
        return self.d[d_shift:d_shift + self.M * self.ldd].view(self.M, self.ldd)

    def a64(self):
        return f8_exact(self.A[0].contiguous().view(F8[self.ta])), to64(self.SA[0])

    def b64(self, g):
        return f8_exact(self.B[g].contiguous().view(F8[self.tb])), to64(self.SB[g])

    def verify(self, out="bf16", act="none", add=False, ldd=None, ldc=None, d_shift=0, in_place=False):
        fill = -7.0
        C = c64 = None
        if add:
            ldc = (self.N if ldd is None else ldd) if ldc is None else ldc
            C = torch.full((d_shift + self.M * ldc + 8,), float("nan"), dtype=FLOAT[out], device="cuda")
            v = C[:self.M * ldc].view(self.M, ldc)[:, :self.N]
            v.copy_(torch.randn((self.M, self.N), generator=generator(77), device="cuda"))
            c64 = to64(v)
        got = to64(self.call(out, act, C, ldc, C if in_place else None, ldd, 0 if in_place else d_shift, fill))
        a, sa = self.a64()
        covered = np.zeros(self.M, dtype=bool)
        for g, lo, hi in self.groups():
            covered[lo:hi] = True
            if hi == lo:
                continue
            b, sb = self.b64(g)
            want, s_abs = f8_product(a[lo:hi], sa[lo:hi], b, sb, self.block)
            tol = f8_bound(self.K, s_abs)
            for extra in ([] if c64 is None else [c64[lo:hi]]) + ([] if self.bias is None else [to64(self.bias[g])[None, :]]):
                want = want + extra
                tol = tol + 4.0 * 2.0 ** -24 * (s_abs + np.abs(extra))
            # through an activation of slope at most 1.13, and its own roundings
            tol = tol if act == "none" else 1.13 * tol + 2.0 ** -20 * np.abs(want)
            within(got[lo:hi, :self.N], act64(want, act), tol, out, "d")
        if not in_place:
            assert (got[~covered] == fill).all(), "rows of no group were written"
            assert (got[:, self.N:] == fill).all(), "the pitch padding was written"
            assert (to64(self.d[:d_shift]) == fill).all() and (to64(self.d[d_shift + self.M * self.ldd:]) == fill).all()
        else:
            assert np.isnan(got[:, self.N:]).all()


def ends(sizes):
    return [0] + [int(v) for v in np.cumsum(sizes)]


PATTERNS = {
    "one": [1], "empty_first_last": [0, 5, 0, 0, 3, 0], "all_in_one": [0, 0, 260, 0],
    "edges": [127, 128, 129, 1, 255, 256, 257, 0, 16, 15, 17], "ones": [1] * 40, "sparse": [0] * 50 + [2] + [0] * 30 + [1],
    "many": [3, 0, 1, 2] * 60 + [70],
}


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("pattern", sorted(PATTERNS))
def test_group_sizes(pattern, block):
    o = ends(PATTERNS[pattern])
    Product(o, o[-1], 264, 400, block=block, seed=len(pattern)).verify()


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 257, 600])
def test_dense_rows(M, block):
    Product(None, M, 520, 656, block=block, seed=M).verify()


@pytest.mark.parametrize("M", [3, 50, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (8, 16), (7, 333), (129, 64), (256, 127), (300, 129), (520, 1000), (1024, 8), (31, 2048),
                                 (136, 4096), (128, 128), (255, 256), (264, 384)])
def test_widths(n, k, M):
    Product(None, M, n, k, seed=n + k, block=128 if n % 2 == 0 else 1).verify("f32" if k % 2 else "bf16")


@pytest.mark.parametrize("ta", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M", [9, 40, 290])
@pytest.mark.parametrize("block", [1, 128])
def test_types(ta, tb, M, block):
    Product(None, M, 264, 528, ta, tb, block, seed=M, negative=True).verify("f32")


@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh"])
@pytest.mark.parametrize("add,bias", [(False, False), (True, False), (False, True), (True, True)])
def test_epilogue(out, act, add, bias):
    for o, M in (([0, 40, 40, 340, 347], 347), (None, 21), (None, 300)):
        Product(o, M, 272, 384, seed=M, bias=bias).verify(out, act, add)
    p = Product(None, 270, 140, 256, block=1, seed=4, bias=bias)
    p.verify(out, act, add, ldd=143)
    if add:
        p.verify(out, act, True, ldd=144, in_place=True)
        p.verify(out, act, True, ldd=141, in_place=True)


@pytest.mark.parametrize("pad,shift,gap", [((16, 32, 0, 0), 0, 0), ((16, 0, 3, 2), 0, 64), ((3, 5, 1, 1), 0, 5), ((0, 0, 0, 0), 1, 0),
                                           ((16, 16, 0, 1), 16, 16)])
@pytest.mark.parametrize("M", [20, 60, 400])
@pytest.mark.parametrize("block", [1, 128])
def test_pitches_and_alignment(pad, shift, gap, M, block):
    p = Product([0, M // 3, M // 3, M - 1, M], M, 136, 264, block=block, seed=9, pad=pad, shift=shift, gap=gap, bias=True)
    p.verify("bf16", ldd=139, d_shift=3)
    p.verify("f32", ldd=144)
    Product(None, M, 136, 263, block=block, seed=9, align=False).verify("f16")


@pytest.mark.parametrize("offsets", [[2, 9, 20], [-5, 4, 1000], [50, 50, 50], [64, 0]])
def test_offsets_that_leave_rows_out_or_the_matrix(offsets):
    Product(offsets, 50, 136, 200, seed=11).verify()
    Product([o * 10 for o in offsets], 500, 136, 200, seed=11).verify()


def test_no_reduction():
    for M in (5, 300):
        Product(None, M, 96, 0, bias=True).verify("f32", "gelu_tanh", add=True)
        Product(None, M, 96, 0).verify("bf16")


@pytest.mark.parametrize("M", [6, 40, 300])
def test_nan_and_zero_scales_stay_where_they_are(M):
    """A row with a NaN scale, as a quantized row with a NaN has, is NaN; a scale of zero
    leaves its block out; other rows are as they were.  So for a block of 128 weights."""
    p = Product(None, M, 392, 512, seed=3)
    p.SA[0][2, 1] = float("nan")
    p.SA[0][3, :] = 0.0
    p.SB[0][1, 2] = float("inf")
    p.A[0][0, :] = 0
    got = to64(p.call("f32"))
    assert np.isnan(got[2]).all()
    inf = got[:, 128:256]
    assert np.isnan(inf[0]).all() and np.isnan(inf[3]).all() and not np.isfinite(inf).any()
    assert (got[3, :128] == 0).all() and (got[0, :128] == 0).all()
    a, sa = p.a64()
    b, sb = p.b64(0)
    sb[1, 2] = 0.0
    sa[2, 1] = 0.0
    want, s_abs = f8_product(a, sa, b, sb, 128)
    rows, cols = [i for i in range(M) if i != 2], [j for j in range(392) if not 128 <= j < 256]
    pick = np.ix_(rows, cols)
    within(got[pick], want[pick], f8_bound(512, s_abs[pick]), "f32", "d")


@pytest.mark.parametrize("M", [6, 40, 300])
def test_sums_keep_small_terms(M):
    """Blocks of alternating size, 2^18 apart: each block's sum is fp32, so small ones are
    not lost beside the large ones of another row's scale."""
    p = Product(None, M, 264, 1024, seed=13)
    p.SA[0][:, ::2] *= 2.0 ** 18
    p.verify("f32")


def test_quantized_product_end_to_end():
    """Forward and both gradients of a linear layer by quantized products, against the
    products of what the quantizer's values stand for."""
    M, K, N = 200, 264, 392
    gen = generator(40)
    x = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    w = torch.randn((N, K), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((M, N), generator=gen, device="cuda").bfloat16()
    qx, sx = ttc.quantize_blocks(x)
    qw, sw = ttc.quantize_blocks(w, block_rows=128)
    y = ttc.gemm_f8_blocks(qx, sx, qw, sw, out_dtype=torch.float32)
    qd, sd = ttc.quantize_blocks(dy)
    qwt, swt = ttc.quantize_blocks(w, block_rows=128, transpose=True)
    dx = ttc.gemm_f8_blocks(qd, sd, qwt, swt, out_dtype=torch.float32)
    qdt, sdt = ttc.quantize_blocks(dy, transpose=True, dtype=torch.float8_e5m2)
    qxt, sxt = ttc.quantize_blocks(x, transpose=True)
    dw = torch.zeros((N, K), device="cuda")
    for _ in range(2):
        ttc.gemm_f8_blocks(qdt, sdt, qxt, sxt, dw, c=dw)
    for got, a, sa, b, sb, block, times in ((y, qx, sx, qw, sw, 128, 1), (dx, qd, sd, qwt, swt, 128, 1), (dw, qdt, sdt, qxt, sxt, 1, 2)):
        want, s_abs = f8_product(f8_exact(a), to64(sa), f8_exact(b), to64(sb), block)
        within(to64(got), times * want, times * f8_bound(a.shape[1], s_abs) + 2.0 ** -23 * s_abs, "f32", "product")
    ok(0)


def test_graph_on_another_stream():
    p = Product(None, 40, 264, 400, seed=5)
    want = p.call().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.d.fill_(0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        assert ttc.ttc_gemm_f8_blocks(1, p.M, p.N, p.K, p.abuf.data_ptr(), p.lda, CODE["e4m3"], p.sabuf.data_ptr(), p.ldsa, None,
                                      p.bbuf.data_ptr(), p.ldb, 0, CODE["e4m3"], p.sbbuf.data_ptr(), p.ldsb, 0, 128, None, p.N,
                                      p.d.data_ptr(), p.N, None, 0, 0, ttc.DTYPE["bf16"], s.cuda_stream) == 0
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.d[:p.M * p.N].view(p.M, p.N), want)
