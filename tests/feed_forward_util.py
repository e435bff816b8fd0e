"""Plain 64-bit forms of the gated feed-forward and the block-scaled fp8 operators, and
the bounds their kernels are held to."""
import math

import numpy as np
import torch

from operators_util import half_ulp, sum_bound

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}


def logistic(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def gate(v, act):
    """act and its derivative."""
    if act == "silu":
        s = logistic(v)
        return v * s, s + v * s * (1.0 - s)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * v * v)
    if act == "relu":
        return np.where(v < 0, 0.0, v), (v > 0).astype(np.float64)
    return v, np.ones_like(v)


def within(got, want, tol, dtype, what):
    """`got` within `tol` of `want`, and half a step of its type."""
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - want) <= tol + half_ulp(np.maximum(np.abs(got), np.abs(want)), dtype))
    if bad.any():
        i = np.unravel_index(np.argmax(bad), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: {got[i]!r} against "
                             f"{want[i]!r}, allowed {tol[i]:.3g}")


# What the activation and its derivative add, relative to the argument (value) and to
# one (slope): exp within 2 + 1.17 |v| units of 2^-23, quotients within 2, a few products.
# |act(v)| <= |v|, and where 1.17 |v| counts, exp(-|v|) has made the term small:
# (2 + 1.17 x) x exp(-x) <= 1.1 and (2 + 1.17 x) (1 + x) exp(-x) <= 3 for x >= 0.
VALUE, SLOPE = 2.0 ** -20, 2.0 ** -19


def check_gated(d, g, u, g_abs, u_abs, K, act, dtype):
    """D against act(g) * u: the errors of both sums through act's slope of at most 1.13
    and the product."""
    eg, eu = sum_bound(K, g_abs), sum_bound(K, u_abs)
    a = gate(g, act)[0]
    tol = (1.13 * eg + VALUE * np.abs(g)) * (np.abs(u) + eu) + (np.abs(a) + 2.0 ** -24) * eu + 2.0 ** -23 * np.abs(a * u)
    within(d, a * u, tol, dtype, "d")


def check_kept(got, want, s_abs, K, dtype):
    within(got, want, sum_bound(K, s_abs), dtype, "kept")


def check_gated_grad(dg, du, h, gate64, up64, dh, dh_abs, K, act, dtype):
    """dgate and dup (and D, unless None) against the formulas on the kept projections."""
    a, slope = gate(gate64, act)
    e = sum_bound(K, dh_abs)
    within(dg, dh * up64 * slope, (e * 1.13 + np.abs(dh) * SLOPE) * np.abs(up64), dtype, "dgate")
    within(du, dh * a, e * np.abs(a) + np.abs(dh) * (VALUE * np.abs(gate64) + 2.0 ** -23 * np.abs(a)), dtype, "dup")
    if h is not None:
        within(h, a * up64, (VALUE * np.abs(gate64) + 2.0 ** -23 * np.abs(a)) * np.abs(up64), dtype, "d")


def expand(scale, rows, K, block_rows):
    return np.repeat(np.repeat(scale, block_rows, axis=-2)[..., :rows, :], 128, axis=-1)[..., :K]


def f8_product(a, sa, b, sb, block_rows):
    """(sum, sum of magnitudes) of the scaled product in 64 bits."""
    A, B = a * expand(sa, a.shape[0], a.shape[1], 1), b * expand(sb, b.shape[0], b.shape[1], block_rows)
    return A @ B.T, np.abs(A) @ np.abs(B).T


def f8_bound(K, s_abs):
    """A block's 128 products with each addition cut, not rounded, to 24 bits (twice,
    as in sum_bound), the scales' product, an addition for every block, C and bias."""
    return (2.0 * min(K, 128) + 2.0 * math.ceil(K / 128) + 8.0) * 2.0 ** -24 * s_abs


def f8_exact(t):
    return t.detach().cpu().float().double().numpy()


def quantize64(x, q_dtype, block_rows, transpose):
    """(q, scale) by the definition, every step in the fp32 it names: bit for bit."""
    x = x.detach().cpu().float()
    x = x.t().contiguous() if transpose else x
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x, (0, -cols % 128, 0, -rows % block_rows))
    blocks = pad.reshape(pad.shape[0] // block_rows, block_rows, pad.shape[1] // 128, 128).numpy()
    most = np.abs(blocks).max(axis=(1, 3))  # NaN where there is one
    top = np.float32(TOP[q_dtype])
    with np.errstate(all="ignore"):
        scale = (most / top).astype(np.float32)
        finite = np.isfinite(most)
        scale = np.where(finite, np.where(scale < np.float32(2.0 ** -126), np.float32(0), scale), most).astype(np.float32)
        inv = np.where(finite & (scale > 0), np.float32(1) / scale, np.float32(0)).astype(np.float32)
        v = blocks * inv[:, None, :, None]
        v = np.where(inv[:, None, :, None] == 0, np.float32(0), np.clip(v, -top, top)).astype(np.float32)
    q = torch.from_numpy(v.reshape(pad.shape)[:rows, :cols].copy()).to(F8[q_dtype])
    return q, torch.from_numpy(scale)
