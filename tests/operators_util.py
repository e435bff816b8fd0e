"""Plain 64-bit forms of the grouped and scaled int8 operators, and the bounds
their kernels are held to."""
import math

import numpy as np
import torch

import tiled_tensor_core_02_gb300 as ttc

FLOAT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# bits of the significand behind its leading one, and the least exponent of a normal number
MANTISSA = {"f16": (10, -14), "bf16": (7, -126), "f32": (23, -126)}


def half_ulp(v, dtype):
    """Half the distance between neighbours of `dtype` at |v| (float64 array)."""
    bits, emin = MANTISSA[dtype]
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 1e-300))), emin)
    return 0.5 * 2.0 ** (e - bits)


def act64(v, act):
    if act == "relu":
        return np.where(v < 0, 0.0, v)
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def sum_bound(terms, s_abs):
    """Error of a sum of `terms` products accumulated in fp32 with each of them
    cut, not rounded, to 24 bits of a partial sum of at most s_abs (twice the
    terms: once for the product's alignment, once for the addition), plus eight
    roundings for scale, bias and what the activation computes."""
    return (2.0 * terms + 8.0) * 2.0 ** -24 * s_abs


def check(got, want, s_abs, terms, out, slope=1.13):
    """`got` against the unrounded float64 `want`: the accumulation's error
    through an activation of slope at most 1.13 (GELU's), a few fp32 roundings
    of the activation itself (2^-20 of |v| <= s_abs), and the output's rounding."""
    got = np.asarray(got, dtype=np.float64)
    tol = slope * sum_bound(terms, s_abs) + 2.0 ** -20 * s_abs + half_ulp(np.maximum(np.abs(got), np.abs(want)), out)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(bad), bad.shape)
        raise AssertionError(f"{int(bad.sum())} of {bad.size} outside the bound; first at {i}: "
                             f"{got[i]!r} against {want[i]!r}, allowed {tol[i]:.3g}")


def to64(t):
    return t.detach().cpu().double().numpy()


def stream():
    return torch.cuda.current_stream().cuda_stream


def ok(status):
    assert status == 0, ttc.STATUS.get(status, status)
    err = ttc.ttc_get_device_error(stream())
    assert err == 0, ttc.STATUS.get(err, err)


def clamp_offsets(offsets, rows):
    """(lo, hi) of every group as the library reads them."""
    o = [min(max(int(v), 0), rows) for v in offsets]
    return [(a, max(a, b)) for a, b in zip(o, o[1:])]


def padded(rows, cols, ld, dtype, gen, scale=1.0, fill=float("nan"), offset=0):
    """rows x cols normal values with pitch ld inside a buffer that is NaN
    (or `fill`) elsewhere, starting `offset` elements into it: (buffer, view)."""
    n = offset + max(rows, 1) * ld + 8
    buf = torch.full((n,), fill, dtype=dtype, device="cuda")
    view = buf[offset:offset + max(rows, 1) * ld].view(max(rows, 1), ld)[:rows, :cols]
    view.copy_(torch.randn((rows, cols), generator=gen, device="cuda") * scale)
    return buf, view


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g
