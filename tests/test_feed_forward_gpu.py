"""The gated feed-forward and the block-scaled fp8 operators as they are used: their torch
wrappers, on streams and back to back, from graphs and threads, past 2^31 elements, on
plain loads, in stalled pipelines, and the example that trains and serves with them."""
import os
import sys
import threading

import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from feed_forward_util import check_gated, check_gated_grad, check_kept, f8_bound, f8_exact, f8_product, quantize64, within
from operators_util import clamp_offsets, generator, ok, stream, to64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.fixture
def knob():
    names = []

    def set_knob(name, value):
        assert ttc.ttc_set_knob(name, value) == 0
        names.append(name)

    yield set_knob
    for name in names:
        ttc.ttc_set_knob(name, 0)


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=generator(seed), device="cuda") * scale).to(dtype)


OFFSETS = [3, 40, 40, 170, 199]  # rows before the first group and after the last, an empty group


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("transposed", [False, True])
def test_gated_wrappers(dtype, grouped, transposed):
    M, K, N, G = 205, 96, 136, 4
    name = "f16" if dtype == torch.float16 else "bf16"
    x = normal(1, M, K + 8, dtype=dtype)[:, :K]
    lead = (G,) if grouped else ()
    # both weights one matrix, the gate's rows (or columns) first
    w = normal(2, *lead, 2 * N, K, dtype=dtype, scale=0.1) if transposed else normal(2, *lead, K, 2 * N, dtype=dtype, scale=0.1)
    gate, up = (w[..., :N, :].mT, w[..., N:, :].mT) if transposed else (w[..., :N], w[..., N:])
    offsets = torch.tensor(OFFSETS, dtype=torch.int32, device="cuda") if grouped else None
    out = torch.full((M, N + 8), 7.0, dtype=dtype, device="cuda")[:, :N]
    pre = torch.full((M, 2 * N + 16), 7.0, dtype=dtype, device="cuda")[:, :2 * N]
    assert ttc.gemm_gated(x, gate, up, out, offsets=offsets, pre=pre, act="gelu_tanh") is out
    again, pre2 = ttc.gemm_gated(x, gate, up, offsets=offsets, pre=True, act="gelu_tanh")
    plain = ttc.gemm_gated(x, gate, up, offsets=offsets, act="gelu_tanh")
    wd = normal(3, *lead, N, K, dtype=dtype, scale=0.1)  # K x N read backwards
    dy = normal(4, M, K, dtype=dtype)
    h = torch.full_like(out, 5.0)
    dpre = torch.full((M, 2 * N), 5.0, dtype=dtype, device="cuda")
    assert ttc.gemm_gated_grad(dy, wd.mT, pre, dpre, h, offsets=offsets, act="gelu_tanh") is dpre
    covered = np.zeros(M, dtype=bool)
    for g, (lo, hi) in enumerate(clamp_offsets(OFFSETS, M) if grouped else [(0, M)]):
        covered[lo:hi] = True
        pick = (lambda t: to64(t[g])) if grouped else to64  # noqa: B023
        X, Gw, Uw, D = to64(x)[lo:hi], pick(gate), pick(up), to64(dy)[lo:hi]
        p = [(X @ m, np.abs(X) @ np.abs(m)) for m in (Gw, Uw)]
        check_gated(to64(out)[lo:hi], p[0][0], p[1][0], p[0][1], p[1][1], K, "gelu_tanh", name)
        kept = to64(pre)[lo:hi]
        for i in range(2):
            check_kept(kept[:, i * N:i * N + N], *p[i], K, name)
        B = pick(wd).T
        got = to64(dpre)[lo:hi]
        check_gated_grad(got[:, :N], got[:, N:], to64(h)[lo:hi], kept[:, :N], kept[:, N:], D @ B, np.abs(D) @ np.abs(B), K,
                         "gelu_tanh", name)
        assert torch.equal(again[lo:hi], out[lo:hi]) and torch.equal(plain[lo:hi], out[lo:hi])
        assert torch.equal(pre2[lo:hi], pre[lo:hi])
    for t, fill in ((out, 7.0), (pre, 7.0), (h, 5.0), (dpre, 5.0)):
        assert (to64(t)[~covered] == fill).all()


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("block", [1, 128])
def test_f8_wrappers(grouped, block):
    M, N, K, G = 205, 300, 520, 4
    a, sa = ttc.quantize_blocks(normal(1, M, K))
    parts = [ttc.quantize_blocks(normal(2 + g, N, K), block_rows=block, dtype=torch.float8_e5m2) for g in range(G if grouped else 1)]
    # a group's rows a few apart in one buffer
    pitch = parts[0][0].stride(0)
    room = torch.zeros((len(parts), N + 3, pitch), dtype=torch.uint8, device="cuda")
    for g, (q, _) in enumerate(parts):
        room[g, :N, :K].copy_(q.contiguous().view(torch.uint8))
    b = room.view(torch.float8_e5m2)[:, :N, :K]
    sb = torch.stack([s for _, s in parts])
    bias = normal(9, len(parts), N, dtype=torch.float32)
    if not grouped:
        b, sb, bias = b[0], sb[0], bias[0]
    offsets = torch.tensor(OFFSETS, dtype=torch.int32, device="cuda") if grouped else None
    c = normal(10, M, N, dtype=torch.float32)
    before = to64(c)
    out = ttc.gemm_f8_blocks(a, sa, b, sb, c, offsets=offsets, c=c, bias=bias)
    assert out is c
    half = ttc.gemm_f8_blocks(a, sa, b, sb, offsets=offsets)
    assert half.dtype == torch.bfloat16
    covered = np.zeros(M, dtype=bool)
    for g, (lo, hi) in enumerate(clamp_offsets(OFFSETS, M) if grouped else [(0, M)]):
        covered[lo:hi] = True
        want, s_abs = f8_product(f8_exact(a)[lo:hi], to64(sa)[lo:hi], f8_exact(parts[g][0]), to64(parts[g][1]), block)
        within(to64(half)[lo:hi], want, f8_bound(K, s_abs), "bf16", "d")
        extra = before[lo:hi] + (to64(bias[g]) if grouped else to64(bias))
        size = s_abs + np.abs(before[lo:hi]) + np.abs(extra)
        within(to64(out)[lo:hi], want + extra, f8_bound(K, s_abs) + 8.0 * 2.0 ** -24 * size, "f32", "d")
    assert (to64(out)[~covered] == before[~covered]).all()


def test_quantizer_wrapper_on_strided_views():
    for x in (normal(1, 200, 400)[:, 8:392], normal(2, 1, 300, dtype=torch.float32), normal(3, 130, 1), normal(4, 64, 1024)[::2]):
        for block in (1, 128):
            for turn in (False, True):
                q, s = ttc.quantize_blocks(x, block_rows=block, transpose=turn)
                want, scale = quantize64(x, "e4m3", block, turn)
                assert torch.equal(q.cpu().contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))
                assert torch.equal(s.cpu(), scale) and q.stride(0) % 16 == 0


# ------------------------------------------------------------------ streams, graphs, threads

class Chain:
    """A gated layer forward and back with an update of its weights in between, then its
    weights and result through the 8-bit products."""

    def __init__(self, rows, width, hidden, seed):
        self.x, self.dy = normal(seed, rows, width), normal(seed + 1, rows, width)
        self.w0, self.wd = normal(seed + 2, 2 * hidden, width, scale=0.1), normal(seed + 3, width, hidden, scale=0.1)
        self.w = self.w0.clone()
        self.n = hidden
        self.rows = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        empty = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.h, self.pre, self.dpre, self.h2 = (empty(rows, k * hidden) for k in (1, 2, 2, 1))
        self.dx, self.grad = empty(rows, width), empty(2 * hidden, width, dtype=torch.float32)
        up = lambda v: -(-v // 16) * 16  # noqa: E731
        f8 = lambda r, c: empty(r, up(c), dtype=torch.float8_e4m3fn)[:, :c]  # noqa: E731
        f32 = lambda r, c: empty(r, c, dtype=torch.float32)  # noqa: E731
        kb = lambda v: -(-v // 128)  # noqa: E731
        self.qx, self.sx = f8(rows, width), f32(rows, kb(width))
        self.qw, self.sw = f8(2 * hidden, width), f32(kb(2 * hidden), kb(width))
        self.qt, self.st = f8(width, rows), f32(width, kb(rows))
        self.qd, self.sd = f8(2 * hidden, rows), f32(2 * hidden, kb(rows))
        self.out, self.gram = empty(rows, 2 * hidden), f32(2 * hidden, width)
        torch.cuda.synchronize()

    def steps(self):
        n = self.n
        gate, up = self.w[:n].t(), self.w[n:].t()
        yield lambda: self.w.copy_(self.w0)
        yield lambda: ttc.gemm_gated(self.x, gate, up, self.h, pre=self.pre)
        yield lambda: ttc.gemm_gated_grad(self.dy, self.wd, self.pre, self.dpre, self.h2)
        yield lambda: ttc.gemm(self.dpre, self.w, out=self.dx)
        yield lambda: ttc.gemm_grouped_wgrad(self.dpre, self.x, self.rows, out=self.grad[None])
        yield lambda: ttc.gemm_grouped_wgrad(self.dpre, self.x, self.rows, c=self.w[None], out=self.w[None], alpha=-0.1, beta=1.0)
        yield lambda: ttc.gemm_gated(self.x, gate, up, self.h, act="gelu_tanh")
        yield lambda: ttc.quantize_blocks(self.x, self.qx, self.sx)
        yield lambda: ttc.quantize_blocks(self.w, self.qw, self.sw, block_rows=128)
        yield lambda: ttc.gemm_f8_blocks(self.qx, self.sx, self.qw, self.sw, self.out)
        yield lambda: ttc.quantize_blocks(self.out, self.qd, self.sd, transpose=True)
        yield lambda: ttc.quantize_blocks(self.x, self.qt, self.st, transpose=True)
        yield lambda: ttc.gemm_f8_blocks(self.qd, self.sd, self.qt, self.st, self.gram)
        yield lambda: ttc.gemm_f8_blocks(self.qd, self.sd, self.qt, self.st, self.gram, c=self.gram)

    def results(self):
        return [t.clone() for t in (self.h, self.pre, self.dpre, self.h2, self.dx, self.grad, self.w, self.out, self.gram)] + \
            [t.contiguous().view(torch.uint8) for t in (self.qx, self.qw, self.qd)]

    def one_by_one(self):
        for step in self.steps():
            step()
            torch.cuda.synchronize()
        return self.results()

    def at_once(self):
        for step in self.steps():
            step()


SHAPES = [(700, 256, 520), (24, 512, 256), (350, 131, 257), (1300, 1024, 2048), (100, 384, 136)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("shape", SHAPES)
def test_back_to_back_and_from_graphs(shape):
    """Two graphs that share every buffer, one after the other, and 20 rounds without new memory."""
    c = Chain(*shape, seed=1)
    want = c.one_by_one()
    for _ in range(3):
        c.at_once()
    assert same(c.results(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph, stream=s):
            c.at_once()
    for t in (c.h, c.pre, c.dpre, c.dx, c.out, c.gram):
        t.zero_()
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert same(c.results(), want)
    del graph, graphs
    free = torch.cuda.mem_get_info()[0]
    for _ in range(20):
        c.at_once()
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] < 1 << 20
    ok(0)


def test_threads_on_their_own_streams():
    chains = [Chain(*shape, seed=10 + i) for i, shape in enumerate(SHAPES)]
    wants = [c.one_by_one() for c in chains]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(6):
                    chains[i].at_once()
                got = chains[i].results()
            s.synchronize()
            if not same(got, wants[i]):
                wrong.append(i)
        except Exception as e:  # a refused call: told to the test
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(chains))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_new_results_on_a_stream_of_the_callers():
    """The wrappers' own results, made on another stream, with the current one busy."""
    x, w = normal(1, 300, 256), normal(2, 512, 256, scale=0.1)
    dy, wd = normal(3, 300, 128), normal(4, 128, 256, scale=0.1)

    def calls(s):
        h, pre = ttc.gemm_gated(x, w[:256].t(), w[256:].t(), pre=True, stream=s)
        dpre = ttc.gemm_gated_grad(dy, wd, pre, stream=s)
        q = ttc.quantize_blocks(x, stream=s)
        qw = ttc.quantize_blocks(w, block_rows=128, stream=s)
        return h, pre, dpre, ttc.gemm_f8_blocks(*q, *qw, stream=s)

    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(50_000_000)
    got = calls(s.cuda_stream)
    s.synchronize()
    assert same(got, want)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ plain loads, stalled pipelines

def verify_gated(M, K, N, seed=0):
    x, w, wd = normal(seed, M, K), normal(seed + 1, 2 * N, K, scale=0.1), normal(seed + 2, K, N, scale=0.1)
    dy = normal(seed + 3, M, K)
    out, pre = ttc.gemm_gated(x, w[:N].t(), w[N:].t(), pre=True)
    h = torch.empty_like(out)
    dpre = to64(ttc.gemm_gated_grad(dy, wd, pre, out=h))
    ok(0)
    X, D, B, kept = to64(x), to64(dy), to64(wd), to64(pre)
    p = [(X @ m, np.abs(X) @ np.abs(m)) for m in (to64(w[:N]).T, to64(w[N:]).T)]
    check_gated(to64(out), p[0][0], p[1][0], p[0][1], p[1][1], K, "silu", "bf16")
    check_gated_grad(dpre[:, :N], dpre[:, N:], to64(h), kept[:, :N], kept[:, N:], D @ B, np.abs(D) @ np.abs(B), K, "silu", "bf16")


def verify_f8(M, N, K, block):
    a, sa = ttc.quantize_blocks(normal(M, M, K))
    b, sb = ttc.quantize_blocks(normal(N, N, K), block_rows=block)
    got = ttc.gemm_f8_blocks(a, sa, b, sb, out_dtype=torch.float32)
    ok(0)
    want, s_abs = f8_product(f8_exact(a), to64(sa), f8_exact(b), to64(sb), block)
    within(to64(got), want, f8_bound(K, s_abs), "f32", "d")


@pytest.mark.parametrize("M", [20, 300])
def test_plain_loads_of_aligned_operands(knob, M):
    knob("force_generic_load", 1)
    verify_gated(M, 264, 136)
    verify_f8(M, 264, 400, 128)
    verify_f8(M, 264, 400, 1)


# few tokens, CTA pairs, plain loads
@pytest.mark.parametrize("M,plain", [(20, False), (2600, False), (2600, True)])
def test_stalled_gated_products_time_out(knob, M, plain):
    if plain:
        knob("force_generic_load", 1)
    x, w, wd, pre = normal(1, M, 256), normal(2, 1024, 256), normal(3, 256, 512), normal(4, M, 1024)
    knob("timeout_ns", 20_000_000)
    knob("inject_stall", 1)
    ttc.gemm_gated(x, w[:512].t(), w[512:].t())
    assert ttc.STATUS[ttc.ttc_get_device_error(stream())] == "TTC_ERR_TIMEOUT"
    ttc.gemm_gated_grad(x, wd, pre)
    assert ttc.STATUS[ttc.ttc_get_device_error(stream())] == "TTC_ERR_TIMEOUT"
    knob("inject_stall", 0)
    knob("timeout_ns", 0)
    verify_gated(M, 256, 512)


@pytest.mark.parametrize("M,N,K", [(10, 512, 1024), (60, 512, 640), (2600, 1600, 1024)])
@pytest.mark.parametrize("block", [1, 128])
def test_stalled_f8_products_time_out(knob, M, N, K, block):
    a, sa = ttc.quantize_blocks(normal(1, M, K))
    b, sb = ttc.quantize_blocks(normal(2, N, K), block_rows=block)
    knob("timeout_ns", 20_000_000)
    knob("inject_stall", 1)
    ttc.gemm_f8_blocks(a, sa, b, sb)
    assert ttc.STATUS[ttc.ttc_get_device_error(stream())] == "TTC_ERR_TIMEOUT"
    knob("inject_stall", 0)
    knob("timeout_ns", 0)
    verify_f8(M, N, K, block)


# ------------------------------------------------------------------ sizes

@pytest.mark.parametrize("M,N,K,block", [(2600, 1600, 1100, 128), (2600, 1600, 1100, 1), (1111, 4100, 777, 128), (5000, 520, 128, 1)])
def test_f8_on_many_tiles(M, N, K, block):
    """Several rounds of tiles a pair, halves of tiles in the last."""
    verify_f8(M, N, K, block)


@pytest.mark.parametrize("M,K,N", [(2600, 512, 1600), (4000, 64, 2056)])
def test_gated_on_many_tiles(M, K, N):
    verify_gated(M, K, N)


@pytest.mark.parametrize("K", [64, 63])  # CTA pairs, plain loads
def test_kept_projections_beyond_2_31(K):
    M, N = 270_000, 4104
    assert M * 2 * N > 1 << 31
    x, w, wd = normal(1, M, K), normal(2, 2 * N, K, scale=0.2), normal(3, N, K, scale=0.2)
    out, pre = ttc.gemm_gated(x, w[:N].t(), w[N:].t(), pre=True)
    rows = [slice(0, 40), slice(261_600, 261_700), slice(M - 70, M)]
    kept = [to64(pre[r]) for r in rows]
    ttc.gemm_gated_grad(x, wd.t(), pre, pre)  # in place
    ok(0)
    for r, k in zip(rows, kept):
        X, B = to64(x[r]), to64(wd).T
        p = [(X @ m, np.abs(X) @ np.abs(m)) for m in (to64(w[:N]).T, to64(w[N:]).T)]
        check_gated(to64(out[r]), p[0][0], p[1][0], p[0][1], p[1][1], K, "silu", "bf16")
        for i in range(2):
            check_kept(k[:, i * N:i * N + N], *p[i], K, "bf16")
        got = to64(pre[r])
        check_gated_grad(got[:, :N], got[:, N:], None, k[:, :N], k[:, N:], X @ B, np.abs(X) @ np.abs(B), K, "silu", "bf16")


@pytest.mark.parametrize("block,turn", [(1, False), (128, False), (1, True), (128, True)])
def test_quantizing_beyond_2_31(block, turn):
    rows, cols = 140_000, 16_000
    assert rows * cols > 1 << 31
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 20_000):
        x[i:i + 20_000] = normal(i, 20_000, cols)
    q, s = ttc.quantize_blocks(x, block_rows=block, transpose=turn)
    ok(0)
    for r, c in ((0, 0), (134_144, 256), (rows - 96, cols - 128)):
        r -= r % 128
        c -= c % 128
        part = x[r:r + 128, c:c + 128]
        want, scale = quantize64(part, "e4m3", block, turn)
        got = q[c:c + 128, r:r + 128] if turn else q[r:r + 128, c:c + 128]
        assert torch.equal(got.cpu().contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))
        a, b = (c, r) if turn else (r, c)
        assert torch.equal(s[a // block:a // block + scale.shape[0], b // 128:b // 128 + 1].cpu(), scale)


@pytest.mark.parametrize("rows", [3, 300])  # few tokens, CTA pairs
def test_f8_weights_beyond_2_31(rows):
    groups, N, K = 40, 14336, 4096
    assert groups * N * K > 1 << 31
    b = torch.empty((groups, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    sb = torch.empty((groups, N // 128, K // 128), device="cuda")
    for g in range(groups):
        ttc.quantize_blocks(normal(g, N, K), b[g], sb[g], block_rows=128)
    a, sa = ttc.quantize_blocks(normal(99, groups * rows, K))
    offsets = torch.arange(0, groups * rows + 1, rows, dtype=torch.int32, device="cuda")
    got = ttc.gemm_f8_blocks(a, sa, b, sb, offsets=offsets)
    ok(0)
    for g in (0, 3, 38, 39):
        part = slice(g * rows, g * rows + 3)
        want, s_abs = f8_product(f8_exact(a[part]), to64(sa[part]), f8_exact(b[g]), to64(sb[g]), 128)
        within(to64(got[part]), want, f8_bound(K, s_abs), "bf16", "d")


def test_f8_result_beyond_2_31():
    M, N, K = 530_000, 4104, 256
    assert M * N > 1 << 31
    a, sa = ttc.quantize_blocks(normal(1, M, K))
    b, sb = ttc.quantize_blocks(normal(2, N, K))
    got = ttc.gemm_f8_blocks(a, sa, b, sb)
    ok(0)
    for r in (slice(0, 64), slice(523_200, 523_400), slice(M - 70, M)):
        want, s_abs = f8_product(f8_exact(a[r]), to64(sa[r]), f8_exact(b), to64(sb), 1)
        within(to64(got[r]), want, f8_bound(K, s_abs), "bf16", "d")


# ------------------------------------------------------------------ example

def test_gated_layer_example_runs():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import gated_layer

    losses, weights = gated_layer.train(tokens=256, steps=3)
    assert len(losses) == 3 and all(np.isfinite(losses))
    assert all(np.isfinite(list(gated_layer.serve(weights).values())))
    ok(0)


def test_gated_layer_example_gradients():
    """Its gradients against the formulas in 64 bits on the same numbers: every rounding to
    bf16 on the way is at most 2^-8 of its value, and at most four follow one another."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import gated_layer

    M, K, N = 200, 64, 96
    x, w, wd, dy = normal(1, M, K), normal(2, 2 * N, K, scale=0.2), normal(3, K, N, scale=0.2), normal(4, M, K)
    y, pre = gated_layer.forward(x, w, wd, keep=True)
    dw, dwd = torch.empty((2 * N, K), device="cuda"), torch.empty((K, N), device="cuda")
    dx = gated_layer.backward(x, w, wd, pre, dy, dw, dwd, add=False)
    X, W, V, D = (t.double().cpu().requires_grad_() for t in (x, w, wd, dy))
    p = X @ W.T
    loss = ((torch.nn.functional.silu(p[:, :N]) * p[:, N:]) @ V.T * D.detach()).sum()
    loss.backward()
    for got, want in ((dx, X.grad), (dw, W.grad), (dwd, V.grad)):
        assert float((got.double().cpu() - want).norm()) <= 4 * 2.0 ** -8 * float(want.norm())
