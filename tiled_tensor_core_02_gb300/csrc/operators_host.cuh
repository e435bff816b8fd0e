// What the entry points of the grouped, gated, int8 and fp8 operators share on the
// host: checks of arguments, extents, parameters and tensor maps of grouped products.
#pragma once
#include <cstring>

#include "gemm_kernel.cuh"
#include "grouped.cuh"
#include "host.cuh"
#include "ttc.h"

namespace ttc {

inline bool is_16bit(ttc_dtype t) { return t == TTC_F16 || t == TTC_BF16; }
inline bool is_dtype(ttc_dtype t) { return t == TTC_F16 || t == TTC_BF16 || t == TTC_I8 || t == TTC_F32; }
inline bool is_act(ttc_act a) { return a == TTC_ACT_NONE || a == TTC_ACT_RELU || a == TTC_ACT_GELU_TANH; }
inline bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
inline int64_t at_least_1(int64_t x) { return x > 1 ? x : 1; }
inline int64_t blocks_of(int64_t x, int64_t b) { return (x + b - 1) / b; }

// Largest distance between two groups' matrices (elements).
constexpr int64_t kStrideLimit = 1ll << 40;

// Bytes from the first to the last element of `count` matrices `stride`
// elements apart, each rows x cols with pitch ld; capped well inside int64.
inline int64_t span_bytes(int64_t count, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int esize) {
  const __int128 n = ((__int128)(count - 1) * stride + (__int128)(rows - 1) * ld + cols) * esize;
  return n > ((__int128)1 << 60) ? 1ll << 60 : (int64_t)n;
}

// The walk over the tiles: bands of 2^shift row blocks.
inline void set_walk(GroupedParams& p, int64_t row_blocks, int64_t col_blocks, int shift) {
  p.row_blocks = (int)row_blocks;
  p.col_blocks = (int)col_blocks;
  p.group_shift = shift;
  p.by_band = fast_div((uint32_t)(col_blocks << shift));
  if (row_blocks > 0) {
    p.by_group = fast_div((uint32_t)(row_blocks * col_blocks));
    const int64_t rest = row_blocks & ((1ll << shift) - 1);
    p.by_rest = fast_div(rest > 0 ? (uint32_t)rest : 1u);
  }
}

// Parameters both grouped products share.
inline void common_params(GroupedParams& p, const HostEnv& env, int64_t groups, int64_t M, int64_t N, int64_t K, const void* A,
                   int64_t lda, const void* B, int64_t ldb, const int32_t* offsets) {
  std::memset(&p, 0, sizeof p);
  p.A = A;
  p.lda = lda;
  p.B = B;
  p.ldb = ldb;
  p.offsets = offsets;
  p.groups = (int)groups;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.err = env.err;
  p.timeout_ns = env.timeout_ns;
  p.inject_stall = env.inject_stall;
}

// Tensor maps of the pair kernel's operands; false where TMA cannot read them.
inline bool pair_maps(GroupedParams& p, bool wgrad, ttc_dtype dtype, const HostEnv& env) {
  if (env.plain_loads || p.M == 0 || p.K == 0) return false;
  if (!tma_rows_ok(p.A, p.lda, 2) || !tma_rows_ok(p.B, p.ldb, 2)) return false;
  if (!wgrad && !tma_stride_ok(p.groups, p.strideB, 2)) return false;
  const CUtensorMapDataType dt = dtype == TTC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  // K contiguous: boxes of 64 k by 128 rows; rows contiguous: 64 rows by the 128 k of a stage
  if (wgrad)
    return encode_matrices(&p.tmA, dt, 2, p.A, p.K, p.M, p.lda, 1, 0, 64, 128, sw) &&
           encode_matrices(&p.tmB, dt, 2, p.B, p.N, p.M, p.ldb, 1, 0, 64, 128, sw);
  const int64_t mats = p.strideB != 0 ? p.groups : 1;
  return encode_matrices(&p.tmA, dt, 2, p.A, p.K, p.M, p.lda, 1, 0, kBK, 128, sw) &&
         (p.b_mn ? encode_matrices(&p.tmB, dt, 2, p.B, p.N, p.K, p.ldb, mats, p.strideB, 64, 128, sw)
                 : encode_matrices(&p.tmB, dt, 2, p.B, p.K, p.N, p.ldb, mats, p.strideB, kBK, 128, sw));
}

}  // namespace ttc
