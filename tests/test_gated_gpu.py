"""GPU parity of the gated feed-forward block and its gradient against a plain 64-bit
implementation."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from feed_forward_util import check_gated, check_gated_grad, check_kept
from operators_util import FLOAT, clamp_offsets, generator, ok, padded, stream, to64

pytestmark = pytest.mark.gpu
FILL = -7.0


class Gated:
    """Operands of one block with NaN in every padding element.  pad: of A, of the weights,
    of D, of the kept projections."""

    def __init__(self, offsets, M, N, K, dtype="bf16", layout="col", seed=0, pad=(0, 0, 0, 0), shift=0, scale=1.0, gap=0):
        gen = generator(seed)
        self.raw = offsets
        self.G = 1 if offsets is None else len(offsets) - 1
        self.M, self.N, self.K, self.dtype, self.layout, self.shift, self.pad = M, N, K, dtype, layout, shift, pad
        self.lda = max(K + pad[0], 1)
        br, bc = (N, K) if layout == "col" else (K, N)
        self.ldb = max(bc + pad[1], 1)
        self.strideB = br * self.ldb + gap
        self.abuf, self.A = padded(M, K, self.lda, FLOAT[dtype], gen, offset=shift)
        self.A *= scale
        self.W = []
        for _ in range(2):
            buf = torch.full((shift + self.G * self.strideB + 8,), float("nan"), dtype=FLOAT[dtype], device="cuda")
            views = []
            for g in range(self.G):
                at = shift + g * self.strideB
                v = buf[at:at + br * self.ldb].view(br, self.ldb)[:, :bc]
                v.copy_(torch.randn((br, bc), generator=gen, device="cuda") / max(K, 1) ** 0.5)
                views.append(v)
            self.W.append((buf, views))
        self.ldd, self.ldp = N + pad[2], 2 * N + pad[3]
        self.pbuf, self.P = padded(M, 2 * N, self.ldp, FLOAT[dtype], gen, offset=shift)
        self.P *= 2.0
        self.offsets = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
        self.lay = ttc.COL_MAJOR if layout == "col" else ttc.ROW_MAJOR

    def at(self, buf, column=0):
        return buf.data_ptr() + 2 * (self.shift + column)

    def buffer(self, ld, fill=FILL):
        return torch.full((self.shift + self.M * ld + 8,), fill, dtype=FLOAT[self.dtype], device="cuda")

    def view(self, buf, ld):
        return buf[self.shift:self.shift + self.M * ld].view(self.M, ld)

    def w64(self, which, g):
        w = to64(self.W[which][1][g])
        return w.T if self.layout == "col" else w

    def groups(self):
        return [(0, 0, self.M)] if self.raw is None else [(g, lo, hi) for g, (lo, hi) in enumerate(clamp_offsets(self.raw, self.M))]

    def forward(self, act, save, s=None):
        self.d, self.kept = self.buffer(self.ldd), self.buffer(self.ldp)
        ok(ttc.ttc_gemm_gated(
            self.G, self.M, self.N, self.K, self.at(self.abuf), self.lda, None if self.offsets is None else self.offsets.data_ptr(),
            self.at(self.W[0][0]), self.at(self.W[1][0]), self.ldb, self.strideB, self.lay, self.at(self.d), self.ldd,
            self.at(self.kept) if save else None, self.at(self.kept, self.N) if save else None, self.ldp, ttc.ACT[act],
            ttc.DTYPE[self.dtype], stream() if s is None else s))

    def untouched(self, buf, ld, cols, covered):
        v = to64(self.view(buf, ld))
        assert (v[~covered] == FILL).all(), "rows of no group were written"
        assert (v[:, cols:] == FILL).all(), "the pitch padding was written"
        assert (to64(buf[:self.shift]) == FILL).all() and (to64(buf[self.shift + self.M * ld:]) == FILL).all()

    def verify(self, act="silu", save=True):
        self.forward(act, save)
        a, d, kept = to64(self.A), to64(self.view(self.d, self.ldd)), to64(self.view(self.kept, self.ldp))
        covered = np.zeros(self.M, dtype=bool)
        for g, lo, hi in self.groups():
            covered[lo:hi] = True
            x, N = a[lo:hi], self.N
            p = [(x @ self.w64(i, g), np.abs(x) @ np.abs(self.w64(i, g))) for i in range(2)]
            check_gated(d[lo:hi, :N], p[0][0], p[1][0], p[0][1], p[1][1], self.K, act, self.dtype)
            if save:
                for i in range(2):
                    check_kept(kept[lo:hi, i * N:i * N + N], *p[i], self.K, self.dtype)
        self.untouched(self.d, self.ldd, self.N, covered)
        self.untouched(self.kept, self.ldp, 2 * self.N if save else 0, covered)

    def verify_grad(self, act="silu", save=True, in_place=False, s=None):
        before = to64(self.P)
        N = self.N
        h = self.buffer(self.ldd)
        dp = self.pbuf if in_place else self.buffer(self.ldp)
        ok(ttc.ttc_gemm_gated_grad(
            self.G, self.M, N, self.K, self.at(self.abuf), self.lda, None if self.offsets is None else self.offsets.data_ptr(),
            self.at(self.W[0][0]), self.ldb, self.strideB, self.lay, self.at(self.pbuf), self.at(self.pbuf, N), self.ldp,
            self.at(dp), self.at(dp, N), self.ldp, self.at(h) if save else None, self.ldd, ttc.ACT[act], ttc.DTYPE[self.dtype],
            stream() if s is None else s))
        a, got, d = to64(self.A), to64(self.view(dp, self.ldp)), to64(self.view(h, self.ldd))
        covered = np.zeros(self.M, dtype=bool)
        for g, lo, hi in self.groups():
            covered[lo:hi] = True
            w = self.w64(0, g)
            check_gated_grad(got[lo:hi, :N], got[lo:hi, N:2 * N], d[lo:hi, :N] if save else None, before[lo:hi, :N],
                             before[lo:hi, N:], a[lo:hi] @ w, np.abs(a[lo:hi]) @ np.abs(w), self.K, act, self.dtype)
        if in_place:
            assert (got[~covered, :2 * N] == before[~covered]).all()
        else:
            self.untouched(dp, self.ldp, 2 * N, covered)
        self.untouched(h, self.ldd, N if save else 0, covered)
        self.P = self.view(self.pbuf, self.ldp)[:, :2 * N]


def ends(sizes):
    return [0] + [int(v) for v in np.cumsum(sizes)]


PATTERNS = {
    "one": [1], "empty_first_last": [0, 5, 0, 0, 3, 0], "all_in_one": [0, 0, 260, 0],
    "edges": [127, 128, 129, 1, 255, 256, 257, 0, 16, 15, 17], "ones": [1] * 40, "sparse": [0] * 50 + [2] + [0] * 30 + [1],
    "many": [3, 0, 1, 2] * 60 + [70],
}


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pattern", sorted(PATTERNS))
def test_group_sizes(pattern, dtype, layout):
    o = ends(PATTERNS[pattern])
    p = Gated(o, o[-1], 200, 136, dtype, layout, seed=len(pattern))
    p.verify()
    p.verify_grad()


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 257, 600])
def test_dense_rows(M, layout):
    p = Gated(None, M, 328, 264, "bf16", layout, seed=M)
    p.verify(save=M % 2 == 1)
    p.verify_grad(save=M % 2 == 0)


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (8, 16), (7, 333), (129, 64), (64, 63), (128, 65), (520, 1000), (1024, 8), (31, 2048),
                                 (136, 4096), (1000, 136), (192, 128), (56, 56)])
def test_widths(n, k, M, layout):
    p = Gated(None, M, n, k, "bf16", layout, seed=n + k)
    p.verify()
    p.verify_grad()


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("save", [False, True])
def test_activations(dtype, act, save):
    for o, M, layout in (([0, 40, 40, 340, 347], 347, "col"), (None, 21, "row"), (None, 515, "col")):
        p = Gated(o, M, 272, 320, dtype, layout, seed=3, scale=3.0)
        p.verify(act, save)
        p.verify_grad(act, save)
        p.verify_grad(act, save, in_place=True)


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("pad,shift,gap", [((3, 5, 7, 1), 0, 0), ((8, 16, 24, 8), 0, 64), ((0, 0, 0, 0), 1, 3), ((8, 8, 8, 8), 8, 8),
                                           ((8, 8, 1, 3), 0, 0), ((8, 8, 8, 4), 0, 0)])
@pytest.mark.parametrize("M", [20, 400])
def test_pitches_and_alignment(pad, shift, gap, layout, M):
    """Odd and padded pitches, bases off the 16-byte boundary, groups whose weights start
    off it; NaN in every padding element."""
    p = Gated([0, M // 3, M // 3, M - 1, M], M, 136, 264, "bf16", layout, seed=9, pad=pad, shift=shift, gap=gap)
    p.verify("gelu_tanh")
    p.verify_grad("silu")
    p.verify_grad("silu", in_place=True)


@pytest.mark.parametrize("offsets", [[2, 9, 20], [-5, 4, 1000], [50, 50, 50], [64, 0]])
def test_offsets_that_leave_rows_out_or_the_matrix(offsets):
    p = Gated(offsets, 50, 136, 72, "bf16", "col", seed=11)
    p.verify()
    p.verify_grad()
    p = Gated([o * 10 for o in offsets], 500, 136, 72, "bf16", "row", seed=12)
    p.verify()
    p.verify_grad()


def test_no_reduction():
    """K == 0: both products are zero."""
    for M in (5, 300):
        p = Gated(None, M, 96, 0, "f16", "col", seed=5)
        p.verify()
        p.verify_grad()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("layout", ["col", "row"])
def test_other_groups_rows_and_weights_do_not_leak(layout, value):
    """A NaN or infinity in one group's rows and weights reaches its own rows only."""
    o = ends([20, 30, 130, 9])
    p = Gated(o, o[-1], 136, 200, "bf16", layout, seed=12)
    p.A[20:50] = value
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


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu", "none"])
@pytest.mark.parametrize("M", [4, 300])
def test_far_values(act, M):
    """Gates far out on both sides, where exp overflows: no NaN of the kernel's own.  One
    product a sum, so that both are exact."""
    values = [0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 15.9, -15.9, 16.1, -16.1, 80.0, -80.0, 88.0, -88.0, 90.0, -90.0, 1e4, -1e4, 1e18, -1e18]
    N = len(values)
    g = torch.tensor(values, dtype=torch.bfloat16, device="cuda")
    a = torch.ones((M, 1), dtype=torch.bfloat16, device="cuda")
    u = torch.linspace(0.5, 2.0, N, device="cuda").bfloat16()
    out, pre = ttc.gemm_gated(a, g[None, :], u[None, :], pre=True, act=act)
    v, w = to64(g), to64(u)
    one = np.ones((M, 1))
    assert (to64(pre) == np.concatenate((v, w))).all()
    check_gated(to64(out), one * v, one * w, one * np.abs(v), one * w, 1, act, "bf16")
    dpre = ttc.gemm_gated_grad(a, u[None, :], pre, act=act)
    got = to64(dpre)
    check_gated_grad(got[:, :N], got[:, N:], None, one * v, one * w, one * w, one * w, 1, act, "bf16")


def test_gradient_against_differences():
    """The whole block's gradients, by the library's calls, against central differences of
    the plain block in 64 bits on the same 16-bit numbers.  The kept projections and their
    gradients are rounded to bf16 (2^-8 each, twice in a product), as is the operand of the next
    product: within 3 %% of the gradient's norm for random directions."""
    M, K, N = 48, 40, 56
    gen = generator(21)
    make = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    x, w, v = make(M, K), (make(2 * N, K) * 0.2), (make(K, N) * 0.2)
    dy = make(M, K)
    out, pre = ttc.gemm_gated(x, w[:N].t(), w[N:].t(), pre=True)
    again = torch.empty_like(out)
    dpre = ttc.gemm_gated_grad(dy, v, pre, out=again)
    dx = ttc.gemm(dpre, w)
    one = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    dw = ttc.gemm_grouped_wgrad(dpre, x, one)[0]
    dv = ttc.gemm_grouped_wgrad(dy, again, one)[0]

    def loss(x, w, v):
        g, u = x @ w[:N].T, x @ w[N:].T
        return float((g / (1 + np.exp(-g)) * u @ v.T * to64(dy)).sum())

    rng = np.random.default_rng(3)
    at = [to64(t) for t in (x, w, v)]
    for i, grad in enumerate((dx, dw, dv)):
        for _ in range(4):
            d = rng.standard_normal(at[i].shape)
            moved = [[t + s * 1e-5 * d if j == i else t for j, t in enumerate(at)] for s in (1, -1)]
            want = (loss(*moved[0]) - loss(*moved[1])) / 2e-5
            got = float((to64(grad) * d).sum())
            assert abs(got - want) < 0.03 * np.linalg.norm(to64(grad)), (i, got, want)


def test_graph_and_streams():
    """Captured and replayed on another stream; two graphs over the same weights."""
    p = Gated(None, 70, 264, 136, "bf16", "col", seed=31)
    p.verify()
    want, kept = p.d.clone(), p.kept.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            assert ttc.ttc_gemm_gated(1, p.M, p.N, p.K, p.at(p.abuf), p.lda, None, p.at(p.W[0][0]), p.at(p.W[1][0]), p.ldb, 0,
                                      p.lay, p.at(p.d), p.ldd, p.at(p.kept), p.at(p.kept, p.N), p.ldp, ttc.ACT["silu"],
                                      ttc.DTYPE["bf16"], s.cuda_stream) == 0
        graphs.append(g)
    p.d.fill_(FILL)
    p.kept.fill_(FILL)
    torch.cuda.synchronize()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(p.d, want) and torch.equal(p.kept, kept)
    ok(0)
