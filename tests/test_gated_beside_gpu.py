"""Gated blocks whose results lie beside their operands, in the rows of one buffer, against a
plain 64-bit implementation: few tokens, CTA pairs and plain loads."""
import numpy as np
import pytest
import torch

import tiled_tensor_core_02_gb300 as ttc
from feed_forward_util import check_gated, check_gated_grad, check_kept
from operators_util import generator, ok, to64

pytestmark = pytest.mark.gpu

# rows, N, K, columns of padding behind the last matrix
SIZES = [(5, 64, 128, 0), (2000, 1088, 192, 0), (70, 51, 33, 2)]


def wide(rows, parts, pad, gen, dtype=torch.bfloat16):
    """One buffer of `rows` rows and its parts side by side: (columns, filled); what is not filled is NaN."""
    ld = sum(n for n, _ in parts) + pad
    buf = torch.full((rows, ld), float("nan"), dtype=dtype, device="cuda")
    out, at = [], 0
    for n, size in parts:
        v = buf[:, at:at + n]
        if size:
            v.copy_(torch.randn((rows, n), generator=gen, device="cuda") * size)
        out.append(v)
        at += n
    return buf, out


def weights(buf, at, groups, rows, cols):
    """`groups` matrices of `rows` rows one below the other, from column `at` of the buffer on."""
    return buf.as_strided((groups, rows, cols), (rows * buf.stride(0), buf.stride(0), 1), buf.storage_offset() + at)


def offsets_of(groups, M):
    return None if groups == 1 else torch.tensor([0, M // 3, M], dtype=torch.int32, device="cuda")


def parts_of(groups, M):
    return [(0, 0, M)] if groups == 1 else [(0, 0, M // 3), (1, M // 3, M)]


def same(got, want):
    return torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16))


@pytest.mark.parametrize("M,N,K,pad", SIZES)
@pytest.mark.parametrize("groups", [1, 2])
def test_forward_beside_the_tokens(M, N, K, pad, groups):
    gen = generator(M)
    buf, (a, d, pre, tail) = wide(M, [(K, 1.0), (N, 0), (2 * N, 0), (8, 0)], pad, gen)
    w = torch.randn((2, groups, N, K), generator=gen, device="cuda").bfloat16().mul_(K ** -0.5).transpose(2, 3)
    before = a.clone()
    take = (lambda t: t[0]) if groups == 1 else (lambda t: t)
    ttc.gemm_gated(a, take(w[0]), take(w[1]), d, offsets=offsets_of(groups, M), pre=pre)
    ok(0)
    assert same(a, before) and torch.isnan(tail).all()
    for g, lo, hi in parts_of(groups, M):
        x, p = to64(before[lo:hi]), [to64(w[i, g]) for i in range(2)]
        s, t = [x @ v for v in p], [np.abs(x) @ np.abs(v) for v in p]
        check_gated(to64(d[lo:hi]), s[0], s[1], t[0], t[1], K, "silu", "bf16")
        for i in range(2):
            check_kept(to64(pre[lo:hi, i * N:i * N + N]), s[i], t[i], K, "bf16")


@pytest.mark.parametrize("M,N,K,pad", SIZES)
@pytest.mark.parametrize("groups", [1, 2])
def test_forward_beside_the_weights(M, N, K, pad, groups):
    gen = generator(M + 1)
    buf, (wg, wu, d, tail) = wide(max(M, groups * K), [(N, K ** -0.5), (N, K ** -0.5), (N, 0), (8, 0)], pad, gen)
    a = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    before = buf[:, :2 * N].clone()
    b = [weights(buf, i * N, groups, K, N) for i in range(2)]
    take = (lambda t: t[0]) if groups == 1 else (lambda t: t)
    ttc.gemm_gated(a, take(b[0]), take(b[1]), d[:M], offsets=offsets_of(groups, M), act="gelu_tanh")
    ok(0)
    assert same(buf[:, :2 * N], before) and torch.isnan(tail).all() and torch.isnan(d[M:]).all()
    for g, lo, hi in parts_of(groups, M):
        x, p = to64(a[lo:hi]), [to64(b[i][g]) for i in range(2)]
        s, t = [x @ v for v in p], [np.abs(x) @ np.abs(v) for v in p]
        check_gated(to64(d[lo:hi]), s[0], s[1], t[0], t[1], K, "gelu_tanh", "bf16")


@pytest.mark.parametrize("M,N,K,pad", SIZES)
@pytest.mark.parametrize("groups,in_place", [(1, False), (2, True)])
def test_gradient_beside_the_tokens(M, N, K, pad, groups, in_place):
    gen = generator(M + 2)
    buf, (a, pre, dpre, d, tail) = wide(M, [(K, 1.0), (2 * N, 2.0), (2 * N, 0), (N, 0), (8, 0)], pad, gen)
    w = torch.randn((groups, N, K), generator=gen, device="cuda").bfloat16().mul_(K ** -0.5).transpose(1, 2)
    before = buf[:, :K + 2 * N].clone()
    got = ttc.gemm_gated_grad(a, w[0] if groups == 1 else w, pre, pre if in_place else dpre, d, offsets=offsets_of(groups, M))
    ok(0)
    assert same(a, before[:, :K]) and (in_place or same(pre, before[:, K:])) and torch.isnan(tail).all()
    kept = to64(before[:, K:])
    for g, lo, hi in parts_of(groups, M):
        x, v = to64(before[lo:hi, :K]), to64(w[g])
        check_gated_grad(to64(got[lo:hi, :N]), to64(got[lo:hi, N:]), to64(d[lo:hi]), kept[lo:hi, :N], kept[lo:hi, N:], x @ v,
                         np.abs(x) @ np.abs(v), K, "silu", "bf16")


@pytest.mark.parametrize("M,N,K,pad", SIZES)
@pytest.mark.parametrize("groups", [1, 2])
def test_gradient_beside_the_weights(M, N, K, pad, groups):
    gen = generator(M + 3)
    buf, (w, dpre, d, tail) = wide(max(M, groups * K), [(N, K ** -0.5), (2 * N, 0), (N, 0), (8, 0)], pad, gen)
    a = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    pre = torch.randn((M, 2 * N), generator=gen, device="cuda").bfloat16()
    before, b = buf[:, :N].clone(), weights(buf, 0, groups, K, N)
    got = ttc.gemm_gated_grad(a, b[0] if groups == 1 else b, pre, dpre[:M], d[:M], offsets=offsets_of(groups, M))
    ok(0)
    assert same(buf[:, :N], before) and torch.isnan(tail).all() and torch.isnan(buf[M:, N:]).all()
    for g, lo, hi in parts_of(groups, M):
        x, v = to64(a[lo:hi]), to64(b[g])
        check_gated_grad(to64(got[lo:hi, :N]), to64(got[lo:hi, N:]), to64(d[lo:hi]), to64(pre[lo:hi, :N]), to64(pre[lo:hi, N:]),
                         x @ v, np.abs(x) @ np.abs(v), K, "silu", "bf16")
