"""Python binding of the ttc C ABI (libttc.so): argument marshalling only.

Every step of the GEMM runs in the library's CUDA kernels.  There is no CPU
or PyTorch fallback: if libttc.so is missing or cannot be loaded, importing
the binding's entry points raises.

Names follow the C header include/ttc.h:
  ttc_gemm(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
           alpha, beta, bias, act, dtype, stream) -> status (int)
  ttc_get_device_error(stream) -> status
  ttc_status_string(status) -> str
  ttc_set_knob(knob, value) -> status
  ttc_launch_count() -> int
  ttc_gemm_grouped, ttc_gemm_grouped_wgrad, ttc_quantize_rows,
  ttc_gemm_i8_scaled[_workspace_size] -> status (size)
  ttc_gemm_gated, ttc_gemm_gated_grad, ttc_quantize_blocks, ttc_gemm_f8_blocks
  -> status
plus `gemm(...)`, `gemm_grouped(...)`, `gemm_grouped_wgrad(...)`,
`quantize_rows(...)`, `gemm_i8_scaled(...)`, `gemm_gated(...)`,
`gemm_gated_grad(...)`, `quantize_blocks(...)` and `gemm_f8_blocks(...)`,
convenience wrappers on torch tensors that read the layouts and leading
dimensions off the tensors' strides.
Their work goes to `stream`, an address, or to the current stream of the operands' device,
which need not be the current device; the caller orders it behind its inputs, and what
reads a result on another stream behind it.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

ROW_MAJOR, COL_MAJOR = 0, 1
ACT = {"none": 0, "relu": 1, "gelu_tanh": 2, "silu": 3}
DTYPE = {"f16": 0, "bf16": 1, "i8": 2, "f32": 3, "f8_e4m3": 4, "f8_e5m2": 5}
STATUS = {0: "TTC_OK", 1: "TTC_ERR_INVALID_ARG", 2: "TTC_ERR_UNSUPPORTED", 3: "TTC_ERR_CUDA",
          4: "TTC_ERR_TIMEOUT", 5: "TTC_ERR_SCRATCH_TOO_SMALL"}
STATIC_SCRATCH_BYTES = 16 * 1024 * 1024
KNOB = {"timeout_ns": 0, "inject_stall": 1, "force_generic_load": 2, "force_generic_store": 3,
        "tile_n": 4, "pair": 5, "swap_ab": 6, "split_k": 7, "pair_tile_n": 8,
        "group_m": 9, "gemv": 10, "conv_halo": 11, "pair_tail": 12, "pdl": 13, "i8_wide": 14, "pair_epi_warps": 15}

# Every symbol the C header declares (checked by the test suite).
EXPORTS = ("ttc_gemm", "ttc_gemm_strided_batched", "ttc_gemm_ws", "ttc_gemm_workspace_size",
           "ttc_gemm_workspace_size_staged",
           "ttc_gemm_static_scratch", "ttc_transpose", "ttc_conv2d_fprop",
           "ttc_gemm_grouped", "ttc_gemm_grouped_wgrad", "ttc_quantize_rows", "ttc_gemm_i8_scaled",
           "ttc_gemm_i8_scaled_workspace_size",
           "ttc_gemm_gated", "ttc_gemm_gated_grad", "ttc_quantize_blocks", "ttc_gemm_f8_blocks",
           "ttc_get_device_error", "ttc_status_string", "ttc_set_knob", "ttc_launch_count", "ttc_gemm_plan")

_lib = None


class TTCError(RuntimeError):
    def __init__(self, status: int, what: str = "ttc_gemm"):
        self.status = status
        super().__init__(f"{what} failed: {STATUS.get(status, status)}")


def library_path() -> str:
    return _build.LIB


def load():
    """Load libttc.so (it must have been built: __graft_entry__.build() or _build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise ImportError(f"libttc.so is not built ({_build.LIB}); run tiled_tensor_core_02_gb300._build.build()")
    L = ctypes.CDLL(_build.LIB)
    i64, vp, f, i = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int
    L.ttc_gemm.argtypes = [i64, i64, i64, vp, i64, i, vp, i64, i, vp, i64, vp, i64, f, f, vp, i, i, vp]
    L.ttc_gemm.restype = i
    L.ttc_gemm_strided_batched.argtypes = [i64, i64, i64, i64, vp, i64, i64, i, vp, i64, i64, i, vp, i64, i64,
                                           vp, i64, i64, f, f, vp, i, i, vp]
    L.ttc_gemm_strided_batched.restype = i
    L.ttc_conv2d_fprop.argtypes = [i64] * 13 + [vp, vp, vp, i64, vp, i64, f, f, vp, i, i, vp]
    L.ttc_conv2d_fprop.restype = i
    L.ttc_transpose.argtypes = [i64, i64, vp, i64, vp, i64, i, vp]
    L.ttc_transpose.restype = i
    L.ttc_gemm_ws.argtypes = [i64, i64, i64, vp, i64, i, vp, i64, i, vp, i64, vp, i64, f, f, vp, i, i, vp,
                              ctypes.c_size_t, vp]
    L.ttc_gemm_ws.restype = i
    L.ttc_gemm_static_scratch.argtypes = [i64, i64, i64, vp, i64, i, vp, i64, i, vp, i64, vp, i64, f, f,
                                          vp, i, i, vp]
    L.ttc_gemm_static_scratch.restype = i
    L.ttc_gemm_workspace_size.argtypes = [i64, i64, i64, vp, i64, i, vp, i64, i, i]
    L.ttc_gemm_workspace_size.restype = ctypes.c_size_t
    L.ttc_gemm_workspace_size_staged.argtypes = [i64, i64, i64, vp, i64, i, vp, i64, i, vp, i64, i]
    L.ttc_gemm_workspace_size_staged.restype = ctypes.c_size_t
    L.ttc_gemm_grouped.argtypes = [i64, i64, i64, i64, vp, i64, vp, vp, i64, i64, i, vp, i64, f, vp, i64, i, i, vp]
    L.ttc_gemm_grouped.restype = i
    L.ttc_gemm_grouped_wgrad.argtypes = [i64, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, i64, vp, i64, i64, f, f,
                                         i, i, vp]
    L.ttc_gemm_grouped_wgrad.restype = i
    L.ttc_quantize_rows.argtypes = [i64, i64, vp, i64, i, vp, i64, vp, vp]
    L.ttc_quantize_rows.restype = i
    L.ttc_gemm_i8_scaled.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, i64, vp, i, i, vp, ctypes.c_size_t,
                                     vp]
    L.ttc_gemm_i8_scaled.restype = i
    L.ttc_gemm_i8_scaled_workspace_size.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, i]
    L.ttc_gemm_i8_scaled_workspace_size.restype = ctypes.c_size_t
    L.ttc_gemm_gated.argtypes = [i64, i64, i64, i64, vp, i64, vp, vp, vp, i64, i64, i, vp, i64, vp, vp, i64, i, i, vp]
    L.ttc_gemm_gated.restype = i
    L.ttc_gemm_gated_grad.argtypes = [i64, i64, i64, i64, vp, i64, vp, vp, i64, i64, i, vp, vp, i64, vp, vp, i64, vp, i64, i,
                                      i, vp]
    L.ttc_gemm_gated_grad.restype = i
    L.ttc_quantize_blocks.argtypes = [i64, i64, vp, i64, i, i, i, vp, i64, i, vp, i64, vp]
    L.ttc_quantize_blocks.restype = i
    L.ttc_gemm_f8_blocks.argtypes = [i64, i64, i64, i64, vp, i64, i, vp, i64, vp, vp, i64, i64, i, vp, i64, i64, i, vp, i64,
                                     vp, i64, vp, i64, i, i, vp]
    L.ttc_gemm_f8_blocks.restype = i
    L.ttc_get_device_error.argtypes = [vp]
    L.ttc_get_device_error.restype = i
    L.ttc_status_string.argtypes = [i]
    L.ttc_status_string.restype = ctypes.c_char_p
    L.ttc_set_knob.argtypes = [i, i64]
    L.ttc_set_knob.restype = i
    L.ttc_launch_count.argtypes = []
    L.ttc_launch_count.restype = i64
    L.ttc_gemm_plan.argtypes = [i64, i64, i64, i64, vp, i64, i64, i, vp, i64, i64, i, vp, i64, i64, vp, i64, i64,
                                f, f, vp, i, i, vp, ctypes.c_size_t, i, ctypes.c_char_p, ctypes.c_size_t]
    L.ttc_gemm_plan.restype = i
    _lib = L
    return L


# ------------------------------------------------------------------ raw C-ABI names

def ttc_gemm(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd, alpha, beta, bias, act,
             dtype, stream) -> int:
    """Pointers are ints (device addresses) or None; stream is a cudaStream_t as int or None."""
    return load().ttc_gemm(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd, alpha, beta,
                           bias, act, dtype, stream)


def ttc_gemm_strided_batched(batch, M, N, K, A, lda, strideA, layoutA, B, ldb, strideB, layoutB, C, ldc,
                             strideC, D, ldd, strideD, alpha, beta, bias, act, dtype, stream) -> int:
    return load().ttc_gemm_strided_batched(batch, M, N, K, A, lda, strideA, layoutA, B, ldb, strideB,
                                           layoutB, C, ldc, strideC, D, ldd, strideD, alpha, beta, bias,
                                           act, dtype, stream)


def ttc_conv2d_fprop(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w, X, Wt, Cm, ldc, D,
                     ldd, alpha, beta, bias, act, dtype, stream) -> int:
    return load().ttc_conv2d_fprop(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w, X, Wt, Cm,
                                   ldc, D, ldd, alpha, beta, bias, act, dtype, stream)


def ttc_transpose(rows, cols, src, lds, dst, ldd, elem_bytes, stream) -> int:
    return load().ttc_transpose(rows, cols, src, lds, dst, ldd, elem_bytes, stream)


def ttc_gemm_grouped(groups, M, N, K, A, lda, offsets, B, ldb, strideB, layoutB, D, ldd, alpha, bias, strideBias,
                     act, dtype, stream) -> int:
    """offsets: device address of groups + 1 int32."""
    return load().ttc_gemm_grouped(groups, M, N, K, A, lda, offsets, B, ldb, strideB, layoutB, D, ldd, alpha, bias,
                                   strideBias, act, dtype, stream)


def ttc_gemm_grouped_wgrad(groups, M, N, K, A, lda, B, ldb, offsets, C, ldc, strideC, D, ldd, strideD, alpha, beta,
                           dtype, out_dtype, stream) -> int:
    return load().ttc_gemm_grouped_wgrad(groups, M, N, K, A, lda, B, ldb, offsets, C, ldc, strideC, D, ldd, strideD,
                                         alpha, beta, dtype, out_dtype, stream)


def ttc_quantize_rows(rows, cols, X, ldx, dtype, Q, ldq, scale, stream) -> int:
    return load().ttc_quantize_rows(rows, cols, X, ldx, dtype, Q, ldq, scale, stream)


def ttc_gemm_i8_scaled(M, N, K, A, lda, scaleA, B, ldb, scaleB, D, ldd, bias, act, out_dtype, workspace,
                       workspace_bytes, stream) -> int:
    return load().ttc_gemm_i8_scaled(M, N, K, A, lda, scaleA, B, ldb, scaleB, D, ldd, bias, act, out_dtype, workspace,
                                     workspace_bytes, stream)


def ttc_gemm_i8_scaled_workspace_size(M, N, K, A, lda, B, ldb, D, ldd, out_dtype) -> int:
    return load().ttc_gemm_i8_scaled_workspace_size(M, N, K, A, lda, B, ldb, D, ldd, out_dtype)


def ttc_gemm_gated(groups, M, N, K, A, lda, offsets, Bgate, Bup, ldb, strideB, layoutB, D, ldd, gate, up, ldp, act, dtype,
                   stream) -> int:
    """offsets: device address of groups + 1 int32, or None with one group; gate, up: None, or where to keep them."""
    return load().ttc_gemm_gated(groups, M, N, K, A, lda, offsets, Bgate, Bup, ldb, strideB, layoutB, D, ldd, gate, up, ldp,
                                 act, dtype, stream)


def ttc_gemm_gated_grad(groups, M, N, K, A, lda, offsets, B, ldb, strideB, layoutB, gate, up, ldp, dgate, dup, lddp, D, ldd,
                        act, dtype, stream) -> int:
    return load().ttc_gemm_gated_grad(groups, M, N, K, A, lda, offsets, B, ldb, strideB, layoutB, gate, up, ldp, dgate, dup,
                                      lddp, D, ldd, act, dtype, stream)


def ttc_quantize_blocks(rows, cols, X, ldx, dtype, block_rows, transpose, Q, ldq, q_dtype, scale, lds, stream) -> int:
    return load().ttc_quantize_blocks(rows, cols, X, ldx, dtype, block_rows, transpose, Q, ldq, q_dtype, scale, lds, stream)


def ttc_gemm_f8_blocks(groups, M, N, K, A, lda, typeA, scaleA, ldsa, offsets, B, ldb, strideB, typeB, scaleB, ldsb, strideSB,
                       block_rows_b, C, ldc, D, ldd, bias, strideBias, act, out_dtype, stream) -> int:
    return load().ttc_gemm_f8_blocks(groups, M, N, K, A, lda, typeA, scaleA, ldsa, offsets, B, ldb, strideB, typeB, scaleB,
                                     ldsb, strideSB, block_rows_b, C, ldc, D, ldd, bias, strideBias, act, out_dtype, stream)


def ttc_gemm_ws(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd, alpha, beta, bias, act,
                dtype, workspace, workspace_bytes, stream) -> int:
    return load().ttc_gemm_ws(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd, alpha, beta,
                              bias, act, dtype, workspace, workspace_bytes, stream)


def ttc_gemm_static_scratch(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd, alpha, beta,
                            bias, act, dtype, stream) -> int:
    """ttc_gemm_ws with the library's fixed device scratch array: for callers
    that cannot allocate device memory (see include/ttc.h)."""
    return load().ttc_gemm_static_scratch(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                                          alpha, beta, bias, act, dtype, stream)


def ttc_gemm_plan(batch, M, N, K, A, lda, strideA, layoutA, B, ldb, strideB, layoutB, C, ldc, strideC, D, ldd,
                  strideD, alpha, beta, bias, act, dtype, workspace, workspace_bytes, sm_count):
    """(status, plan): the launches the call would make on a device with
    sm_count SMs, planned on the host without a GPU (see include/ttc.h)."""
    buf = ctypes.create_string_buffer(4096)
    st = load().ttc_gemm_plan(batch, M, N, K, A, lda, strideA, layoutA, B, ldb, strideB, layoutB, C, ldc, strideC,
                              D, ldd, strideD, alpha, beta, bias, act, dtype, workspace, workspace_bytes, sm_count,
                              buf, len(buf))
    return st, buf.value.decode()


def ttc_gemm_workspace_size(M, N, K, A, lda, layoutA, B, ldb, layoutB, dtype) -> int:
    return load().ttc_gemm_workspace_size(M, N, K, A, lda, layoutA, B, ldb, layoutB, dtype)


def ttc_gemm_workspace_size_staged(M, N, K, A, lda, layoutA, B, ldb, layoutB, D, ldd, dtype) -> int:
    return load().ttc_gemm_workspace_size_staged(M, N, K, A, lda, layoutA, B, ldb, layoutB, D, ldd, dtype)


def ttc_get_device_error(stream=None) -> int:
    return load().ttc_get_device_error(stream)


def ttc_status_string(status: int) -> str:
    return load().ttc_status_string(status).decode()


def ttc_set_knob(knob, value: int) -> int:
    k = KNOB[knob] if isinstance(knob, str) else int(knob)
    return load().ttc_set_knob(k, int(value))


def ttc_launch_count() -> int:
    return load().ttc_launch_count()


# ------------------------------------------------------------------ torch convenience

def _matrix_layout(t, rows, cols):
    """(layout, ld) of a 2-D tensor viewed as a rows x cols matrix."""
    s0, s1 = t.stride()
    empty = rows == 0 or cols == 0
    # rows (columns) of which there are several start at least a row's (column's) length apart
    by_rows = empty or rows == 1 or s0 >= cols
    by_cols = empty or cols == 1 or s1 >= rows
    if cols == 1 and rows >= 1 and s0 == 1:
        return COL_MAJOR, max(s1, rows)
    if (s1 == 1 or cols == 1) and by_rows:
        return ROW_MAJOR, max(s0, cols, 1)
    if (s0 == 1 or rows == 1) and by_cols:
        return COL_MAJOR, max(s1, rows, 1)
    raise ValueError("operand must be row- or column-major (one unit stride, rows that do not overlap)")


def _stream_of(stream, device):
    """The address of the stream that a call's work goes to: the caller's, else the current one."""
    import torch

    if device.type != "cuda":
        raise ValueError("operands must be CUDA tensors")
    return torch.cuda.current_stream(device).cuda_stream if stream is None else stream


def _call(f, device, *args):
    """f(*args) with the operands' device as the current one, which is where the library works."""
    import torch

    if device.index == torch.cuda.current_device():
        return f(*args)
    with torch.cuda.device(device):
        return f(*args)


def _scratch(shape, dtype, device, stream):
    """A new tensor for work on `stream` (an address, or None: the current one).

    torch hands a freed block out again as soon as the stream it was allocated on
    has the work in order, so memory for another stream comes from that stream's blocks:
    one of the current stream's may still be read or written there."""
    import torch

    if stream is None or stream == torch.cuda.current_stream(device).cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    own = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(own):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(shape, dtype, device, stream):
    """_scratch for a result, which the current stream is going to read."""
    import torch

    t = _scratch(shape, dtype, device, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _result_pitch(t, rows, cols, what):
    """Pitch of a row-major tensor that holds a rows x cols matrix."""
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols:
        raise ValueError(f"{what} must be M x N")
    if (t.stride(1) != 1 and cols > 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError(f"{what} must be row-major")
    return max(t.stride(0), cols)


def gemm(a, b, c=None, out=None, *, alpha=1.0, beta=0.0, bias=None, act="none", stream=None,
         check=True):
    """D = act(alpha * a @ b + beta * c + bias) through the C ABI.

    a: M x K, b: K x N (torch CUDA tensors, fp16/bf16/int8, row- or column-major);
    c, out: M x N row-major (input dtype, int32 for int8).  Returns out."""
    import torch

    M, K = a.shape
    K2, N = b.shape
    if K2 != K:
        raise ValueError("inner dimensions differ")
    dt = {torch.float16: "f16", torch.bfloat16: "bf16", torch.int8: "i8"}[a.dtype]
    odt = torch.int32 if dt == "i8" else a.dtype
    if out is None:
        out = _result((M, N), odt, a.device, stream)
    la, lda = _matrix_layout(a, M, K)
    lb, ldb = _matrix_layout(b, K, N)
    ldd = _result_pitch(out, M, N, "out")
    if c is not None and beta != 0.0:  # read
        ldc = _result_pitch(c, M, N, "c")
        cptr = c.data_ptr()
    else:
        ldc, cptr = N, None
    for name, t in (("b", b), ("c", c), ("out", out), ("bias", bias)):
        if t is not None and t.device != a.device:
            raise ValueError(f"{name} must be on {a.device}")
    bptr = bias.data_ptr() if bias is not None else None
    stream = _stream_of(stream, a.device)
    st = _call(ttc_gemm, a.device, M, N, K, a.data_ptr(), lda, la, b.data_ptr(), ldb, lb, cptr, ldc, out.data_ptr(),
               ldd, float(alpha), float(beta), bptr, ACT[act], DTYPE[dt], stream)
    if check and st != 0:
        raise TTCError(st)
    return out


def _row_pitch(t, what):
    """Pitch of a 2-D tensor that must be row-major."""
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions")
    rows, cols = t.shape
    if (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError(f"{what} must be row-major")
    return max(t.stride(0), cols, 1)


def _group_pitch(t, what):
    """(stride, pitch) of a 3-D tensor of row-major matrices."""
    if t.dim() != 3:
        raise ValueError(f"{what} must have three dimensions")
    return (t.stride(0), _row_pitch(t[0], what)) if t.shape[0] else (0, max(t.shape[2], 1))


def _same(device, dtypes, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}")
        if t is not None and t.dtype not in dtypes:
            raise ValueError(f"{name} must be of {' or '.join(str(d) for d in dtypes)}")


def _check_offsets(offsets, groups, device):
    import torch

    _same(device, (torch.int32,), offsets=offsets)
    if offsets.dim() != 1 or offsets.numel() != groups + 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be groups + 1 contiguous int32")


def _finish(f, device, check, *args):
    status = _call(f, device, *args)
    if check and status != 0:
        raise TTCError(status, f.__name__)


def _half(t, what):
    import torch

    if t.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"{what} must be of torch.float16 or torch.bfloat16")
    return "f16" if t.dtype == torch.float16 else "bf16"


def gemm_grouped(a, b, offsets, out=None, *, alpha=1.0, bias=None, act="none", stream=None, check=True):
    """out[i] = act(alpha * a[i] @ b[g] + bias[g]) for the rows i of every group g
    (offsets[g] <= i < offsets[g + 1]); other rows of out are left as they are.

    a: M x K row-major, b: groups x K x N, each matrix row- or column-major
    (fp16/bf16 CUDA tensors; b.transpose(1, 2) of the weights gives the gradient
    of the rows), offsets: groups + 1 int32 on the device, bias: groups x N fp32.
    Returns out (M x N; a new one is not initialised where no group has rows)."""
    import torch

    dt = _half(a, "a")
    lda = _row_pitch(a, "a")
    if b.dim() != 3 or b.shape[1] != a.shape[1]:
        raise ValueError("b must be groups x K x N with a's K")
    (M, K), (groups, _, N) = a.shape, b.shape
    _same(a.device, (a.dtype,), b=b, out=out)
    _same(a.device, (torch.float32,), bias=bias)
    _check_offsets(offsets, groups, a.device)
    if out is None:
        out = _result((M, N), a.dtype, a.device, stream)
    if out.shape != (M, N):
        raise ValueError("out must be M x N")
    ldd = _row_pitch(out, "out")
    lb, ldb = _matrix_layout(b[0], K, N) if groups else (ROW_MAJOR, max(N, 1))
    stride_bias = 0
    if bias is not None:
        if bias.shape != (groups, N) or (N > 1 and bias.stride(1) != 1):
            raise ValueError("bias must be groups x N, its rows contiguous")
        stride_bias = bias.stride(0)
    stream = _stream_of(stream, a.device)
    _finish(ttc_gemm_grouped, a.device, check, groups, M, N, K, a.data_ptr(), lda, offsets.data_ptr(), b.data_ptr(),
            ldb, b.stride(0), lb, out.data_ptr(), ldd, float(alpha), None if bias is None else bias.data_ptr(),
            stride_bias, ACT[act], DTYPE[dt], stream)
    return out


def gemm_grouped_wgrad(a, b, offsets, c=None, out=None, *, alpha=1.0, beta=0.0, out_dtype=None, stream=None, check=True):
    """out[g] = alpha * a_g.T @ b_g + beta * c[g], a_g and b_g the rows of group g:
    the gradient of gemm_grouped's weights.

    a: M x K, b: M x N row-major (fp16/bf16 CUDA tensors), offsets: groups + 1
    int32 on the device; c, out: groups x K x N, row-major, of a's type or fp32
    (out_dtype, for a new out: fp32).  c may be out itself.  Returns out."""
    import torch

    dt = _half(a, "a")
    lda, ldb = _row_pitch(a, "a"), _row_pitch(b, "b")
    (M, K), N, groups = a.shape, b.shape[1], offsets.numel() - 1
    if b.shape[0] != M:
        raise ValueError("a and b must have the same rows")
    _same(a.device, (a.dtype,), b=b)
    _check_offsets(offsets, groups, a.device)
    if out is None:
        out = _result((groups, K, N), out_dtype or torch.float32, a.device, stream)
    _same(a.device, (a.dtype, torch.float32), out=out)
    _same(a.device, (out.dtype,), c=c)
    if out.shape != (groups, K, N) or (c is not None and c.shape != out.shape):
        raise ValueError("c and out must be groups x K x N")
    stride_d, ldd = _group_pitch(out, "out")
    stride_c, ldc = (0, max(N, 1)) if c is None else _group_pitch(c, "c")
    odt = "f32" if out.dtype == torch.float32 else dt
    stream = _stream_of(stream, a.device)
    _finish(ttc_gemm_grouped_wgrad, a.device, check, groups, M, N, K, a.data_ptr(), lda, b.data_ptr(), ldb,
            offsets.data_ptr(), None if c is None else c.data_ptr(), ldc, stride_c, out.data_ptr(), ldd, stride_d,
            float(alpha), float(beta), DTYPE[dt], DTYPE[odt], stream)
    return out


def quantize_rows(x, out=None, scale=None, *, stream=None, check=True):
    """(q, scale): int8 rows and their fp32 scales, x[i] near scale[i] * q[i].

    x: rows x cols row-major CUDA tensor (fp16/bf16/fp32).  A new q has rows on
    16-byte boundaries, which gemm_i8_scaled reads fastest."""
    import torch

    _same(x.device, (torch.float16, torch.bfloat16, torch.float32), x=x)
    ldx = _row_pitch(x, "x")
    rows, cols = x.shape
    if out is None:
        out = _result((rows, -(-cols // 16) * 16), torch.int8, x.device, stream)[:, :cols]
    if scale is None:
        scale = _result((rows,), torch.float32, x.device, stream)
    _same(x.device, (torch.int8,), out=out)
    _same(x.device, (torch.float32,), scale=scale)
    if out.shape != x.shape or scale.shape != (rows,) or not scale.is_contiguous():
        raise ValueError("out must have x's shape and scale its rows")
    ldq = _row_pitch(out, "out")
    dt = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}[x.dtype]
    stream = _stream_of(stream, x.device)
    _finish(ttc_quantize_rows, x.device, check, rows, cols, x.data_ptr(), ldx, DTYPE[dt], out.data_ptr(), ldq,
            scale.data_ptr(), stream)
    return out, scale


def gemm_i8_scaled(a, scale_a, b, scale_b, out=None, *, out_dtype=None, bias=None, act="none", workspace=None,
                   stream=None, check=True):
    """out = act((a @ b.T) * scale_a[:, None] * scale_b + bias), the int8 product exact.

    a: M x K, b: N x K int8 row-major CUDA tensors as quantize_rows makes them,
    scale_a: M, scale_b and bias: N fp32.  out: M x N row-major, of out_dtype
    (fp16, bf16 or fp32; a new out: bf16).  workspace: uint8 tensor of
    ttc_gemm_i8_scaled_workspace_size() bytes; None takes one from torch's
    allocator where the sizes want one.  Returns out."""
    import torch

    _same(a.device, (torch.int8,), a=a, b=b)
    _same(a.device, (torch.float32,), scale_a=scale_a, scale_b=scale_b, bias=bias)
    lda, ldb = _row_pitch(a, "a"), _row_pitch(b, "b")
    (M, K), N = a.shape, b.shape[0]
    if b.shape[1] != K:
        raise ValueError("inner dimensions differ")
    for name, t, n in (("scale_a", scale_a, M), ("scale_b", scale_b, N), ("bias", bias, N)):
        if t is not None and (t.shape != (n,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be {n} contiguous fp32")
    if out is None:
        out = _result((M, N), out_dtype or torch.bfloat16, a.device, stream)
    _same(a.device, (torch.float16, torch.bfloat16, torch.float32), out=out)
    if out.shape != (M, N):
        raise ValueError("out must be M x N")
    ldd = _row_pitch(out, "out")
    odt = DTYPE[{torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}[out.dtype]]
    if workspace is not None and (workspace.device != a.device or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be on {a.device} and contiguous")
    stream = _stream_of(stream, a.device)
    if workspace is None:
        need = _call(ttc_gemm_i8_scaled_workspace_size, a.device, M, N, K, a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(),
                     ldd, odt)
        if need:
            workspace = _scratch((need,), torch.uint8, a.device, stream)
    _finish(ttc_gemm_i8_scaled, a.device, check, M, N, K, a.data_ptr(), lda, scale_a.data_ptr(), b.data_ptr(), ldb,
            scale_b.data_ptr(), out.data_ptr(), ldd, None if bias is None else bias.data_ptr(), ACT[act], odt,
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size(), stream)
    return out


def _weights(b, groups, K, what):
    """(N, layout, pitch, stride) of K x N weights: a matrix, or with groups one each."""
    if b.dim() != (2 if groups is None else 3) or b.shape[-2] != K or (groups is not None and b.shape[0] != groups):
        raise ValueError(f"{what} must be {'K x N' if groups is None else 'groups x K x N'} with a's K")
    N = b.shape[-1]
    if groups == 0:
        return N, ROW_MAJOR, max(N, 1), 0
    layout, ld = _matrix_layout(b if groups is None else b[0], K, N)
    return N, layout, ld, 0 if groups is None else b.stride(0)


def _half_of(t, N, what):
    """The two M x N halves of an M x 2N tensor, their pitch."""
    if t.dim() != 2 or t.shape[1] != 2 * N:
        raise ValueError(f"{what} must be M x 2N")
    return t.data_ptr(), t.data_ptr() + N * t.element_size(), _row_pitch(t, what)


def _groups_of(offsets, device):
    """Number of groups, None without offsets."""
    if offsets is None:
        return None
    _check_offsets(offsets, offsets.numel() - 1, device)
    if offsets.numel() < 1:
        raise ValueError("offsets must be groups + 1 contiguous int32")
    return offsets.numel() - 1


def gemm_gated(a, b_gate, b_up, out=None, *, offsets=None, pre=None, act="silu", stream=None, check=True):
    """out = act(a @ b_gate) * (a @ b_up): a gated feed-forward block up to its last projection.

    a: M x K row-major, b_gate and b_up: K x N, row- or column-major alike (fp16/bf16
    CUDA tensors; halves of one weight matrix are views of it).  With offsets (groups + 1
    int32 on the device) the weights are groups x K x N and group g's rows use the g-th;
    rows of no group are left as they are.  pre: M x 2N row-major, or True for a new one:
    a @ b_gate and a @ b_up are kept side by side in it for gemm_gated_grad.
    Returns out (M x N), with pre True (out, pre)."""
    import torch

    dt = _half(a, "a")
    lda = _row_pitch(a, "a")
    M, K = a.shape
    groups = _groups_of(offsets, a.device)
    N, layout, ldb, stride_b = _weights(b_gate, groups, K, "b_gate")
    if b_up.shape != b_gate.shape or _weights(b_up, groups, K, "b_up") != (N, layout, ldb, stride_b):
        raise ValueError("b_up must have b_gate's shape and strides")
    new = pre is True
    if new:
        pre = _result((M, 2 * N), a.dtype, a.device, stream)
    if out is None:
        out = _result((M, N), a.dtype, a.device, stream)
    _same(a.device, (a.dtype,), b_gate=b_gate, b_up=b_up, out=out, pre=pre)
    if out.shape != (M, N):
        raise ValueError("out must be M x N")
    if pre is not None and pre.shape[0] != M:
        raise ValueError("pre must be M x 2N")
    ldd = _row_pitch(out, "out")
    gate, up, ldp = (None, None, 0) if pre is None else _half_of(pre, N, "pre")
    stream = _stream_of(stream, a.device)
    _finish(ttc_gemm_gated, a.device, check, 1 if groups is None else groups, M, N, K, a.data_ptr(), lda,
            None if offsets is None else offsets.data_ptr(), b_gate.data_ptr(), b_up.data_ptr(), ldb, stride_b, layout,
            out.data_ptr(), ldd, gate, up, ldp, ACT[act], DTYPE[dt], stream)
    return (out, pre) if new else out


def gemm_gated_grad(a, b, pre, dpre=None, out=None, *, offsets=None, act="silu", stream=None, check=True):
    """Gradients of gemm_gated's two products, from the gradient of what follows them.

    a: M x K row-major, the gradient of the block's result; b: K x N, row- or column-major:
    the last projection read backwards, so that a @ b is the gradient of gemm_gated's out
    (with offsets groups x K x N).  pre: M x 2N as gemm_gated kept it.  dpre: M x 2N, may be
    pre itself.  out: M x N, or None: gets act(gate) * up again, for the gradient of b.
    Returns dpre: dpre @ W, W the weights one above the other (2N x K'), is the gradient of
    gemm_gated's a, and dpre.T @ a' that of W."""
    import torch

    dt = _half(a, "a")
    lda = _row_pitch(a, "a")
    M, K = a.shape
    groups = _groups_of(offsets, a.device)
    N, layout, ldb, stride_b = _weights(b, groups, K, "b")
    if dpre is None:
        dpre = _result((M, 2 * N), a.dtype, a.device, stream)
    _same(a.device, (a.dtype,), b=b, pre=pre, dpre=dpre, out=out)
    if pre.shape[0] != M or dpre.shape != pre.shape or (out is not None and out.shape != (M, N)):
        raise ValueError("pre and dpre must be M x 2N, out M x N")
    gate, up, ldp = _half_of(pre, N, "pre")
    dgate, dup, lddp = _half_of(dpre, N, "dpre")
    ldd = N if out is None else _row_pitch(out, "out")
    stream = _stream_of(stream, a.device)
    _finish(ttc_gemm_gated_grad, a.device, check, 1 if groups is None else groups, M, N, K, a.data_ptr(), lda,
            None if offsets is None else offsets.data_ptr(), b.data_ptr(), ldb, stride_b, layout, gate, up, ldp, dgate,
            dup, lddp, None if out is None else out.data_ptr(), ldd, ACT[act], DTYPE[dt], stream)
    return dpre


def _float8(dtype, what):
    import torch

    names = {torch.float8_e4m3fn: "f8_e4m3", torch.float8_e5m2: "f8_e5m2"}
    if dtype not in names:
        raise ValueError(f"{what} must be of torch.float8_e4m3fn or torch.float8_e5m2")
    return names[dtype]


def quantize_blocks(x, out=None, scale=None, *, block_rows=1, transpose=False, dtype=None, stream=None, check=True):
    """(q, scale): 8-bit floats and a fp32 scale for each block of block_rows (1 or 128) x 128.

    x: rows x cols row-major CUDA tensor (fp16/bf16/fp32).  q is x, or with transpose its
    transpose, over the scales: q[i, j] * scale[i // block_rows, j // 128] is near it.
    dtype, for a new q: torch.float8_e4m3fn (default) or torch.float8_e5m2.  A new q has rows
    on 16-byte boundaries, which gemm_f8_blocks reads fastest."""
    import torch

    _same(x.device, (torch.float16, torch.bfloat16, torch.float32), x=x)
    ldx = _row_pitch(x, "x")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    rows, cols = x.shape
    r, c = (cols, rows) if transpose else (rows, cols)
    if out is None:
        out = _result((r, -(-c // 16) * 16), dtype or torch.float8_e4m3fn, x.device, stream)[:, :c]
    q_dtype = _float8(out.dtype, "out")
    shape = (-(-r // block_rows), -(-c // 128))
    if scale is None:
        scale = _result(shape, torch.float32, x.device, stream)
    _same(x.device, (out.dtype,), out=out)
    _same(x.device, (torch.float32,), scale=scale)
    if out.shape != (r, c) or scale.shape != shape:
        raise ValueError("out must have x's (the transpose's) shape and scale one element a block")
    ldq, lds = _row_pitch(out, "out"), _row_pitch(scale, "scale")
    dt = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}[x.dtype]
    stream = _stream_of(stream, x.device)
    _finish(ttc_quantize_blocks, x.device, check, rows, cols, x.data_ptr(), ldx, DTYPE[dt], block_rows, int(transpose),
            out.data_ptr(), ldq, DTYPE[q_dtype], scale.data_ptr(), lds, stream)
    return out, scale


def gemm_f8_blocks(a, scale_a, b, scale_b, out=None, *, offsets=None, c=None, out_dtype=None, bias=None, act="none",
                   stream=None, check=True):
    """out = act((a over its scales) @ (b over its scales).T + c + bias), as quantize_blocks makes a and b.

    a: M x K, b: N x K (torch.float8_e4m3fn or float8_e5m2 row-major CUDA tensors); scale_a: M x
    blocks of 128 of K, scale_b: N x blocks, or blocks of 128 of N x blocks, fp32.  With offsets
    (groups + 1 int32 on the device) b, scale_b and bias have a group dimension in front and group
    g's rows of a use the g-th; rows of no group are left as they are.  out: M x N row-major, of
    out_dtype (fp16, bf16 or fp32; a new out: bf16); c, of out's type, may be out itself; bias: N
    fp32.  Returns out."""
    import torch

    ta, tb = _float8(a.dtype, "a"), _float8(b.dtype, "b")
    lda = _row_pitch(a, "a")
    M, K = a.shape
    groups = _groups_of(offsets, a.device)
    dims = 2 if groups is None else 3
    if b.dim() != dims or b.shape[-1] != K or scale_b.dim() != dims or (groups is not None and (b.shape[0] != groups or scale_b.shape[0] != groups)):
        raise ValueError("b and scale_b must be N x K and its blocks, with offsets one of each a group")
    N, blocks = b.shape[-2], -(-K // 128)
    if scale_a.shape != (M, blocks):
        raise ValueError("scale_a must be M x blocks of 128 of K")
    if scale_b.shape[-2:] == (N, blocks):
        block_rows = 1
    elif scale_b.shape[-2:] == (-(-N // 128), blocks):
        block_rows = 128
    else:
        raise ValueError("scale_b must have N rows, or one for 128 of them, and a column for 128 of K")
    if bias is not None and (bias.shape != ((N,) if groups is None else (groups, N)) or (N > 1 and bias.stride(-1) != 1)):
        raise ValueError("bias must be N, with offsets groups x N, its rows contiguous")
    if out is None:
        out = _result((M, N), out_dtype or torch.bfloat16, a.device, stream)
    _same(a.device, (torch.float16, torch.bfloat16, torch.float32), out=out)
    _same(a.device, (b.dtype,), b=b)
    _same(a.device, (torch.float32,), scale_a=scale_a, scale_b=scale_b, bias=bias)
    _same(a.device, (out.dtype,), c=c)
    if out.shape != (M, N) or (c is not None and c.shape != (M, N)):
        raise ValueError("out and c must be M x N")
    ldd, ldc = _row_pitch(out, "out"), N if c is None else _row_pitch(c, "c")
    lds_a = _row_pitch(scale_a, "scale_a")
    if groups is None:
        (stride_b, ldb), (stride_sb, lds_b) = (0, _row_pitch(b, "b")), (0, _row_pitch(scale_b, "scale_b"))
    else:
        (stride_b, ldb), (stride_sb, lds_b) = _group_pitch(b, "b"), _group_pitch(scale_b, "scale_b")
    odt = DTYPE[{torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}[out.dtype]]
    stream = _stream_of(stream, a.device)
    _finish(ttc_gemm_f8_blocks, a.device, check, 1 if groups is None else groups, M, N, K, a.data_ptr(), lda, DTYPE[ta],
            scale_a.data_ptr(), lds_a, None if offsets is None else offsets.data_ptr(), b.data_ptr(), ldb, stride_b,
            DTYPE[tb], scale_b.data_ptr(), lds_b, stride_sb, block_rows, None if c is None else c.data_ptr(), ldc,
            out.data_ptr(), ldd, None if bias is None else bias.data_ptr(),
            0 if groups is None or bias is None else bias.stride(0), ACT[act], odt, stream)
    return out
