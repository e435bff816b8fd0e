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

// Output columns of a few-token tile: as few, in steps of 8 up to 128, as let the
// tiles of `blocks` blocks of tokens fill whole waves of SMs (of more than three
// waves the last one costs less than narrower tiles do: 64 groups, 4099 x 1536 x 2048
// 79.6 us with 128 columns, 84.8 with 112); with the columns contiguous in memory
// (TMA boxes of 64) 64 or 128.  `blocks` is an estimate, so the second and third wave
// may miss: over 48 random cases of up to 64 rows a group they took 0.88 (8 groups,
// 34 rows, 2944 x 1728: 15.7 us against 18.0) to 1.36 times (7 groups, 33 rows,
// 2752 x 2432: 17.0 against 12.5) what one wave, else 128 columns, takes.
inline int few_tile_cols(int64_t blocks, int64_t n, int sm_count, bool cols_contiguous, int most) {
  int64_t c = most;
  for (int64_t waves = 1; waves <= 3; ++waves) {
    const int64_t room = waves * sm_count / blocks;  // tiles of a block of tokens
    if (room < 1 || blocks_of(n, room) > most) continue;
    c = blocks_of(blocks_of(n, room), 8) * 8;
    break;
  }
  if (cols_contiguous) return c > 64 ? most : 64;
  return (int)c;
}

// Blocks of tokens that `rows` rows of `matrices` groups are likely to make.  Groups near
// the mean take one block more as often as not (256 rows of 4 groups, 1088 x 1040: tiles for
// four blocks 16.0 us, for six 11.1).
inline int64_t few_blocks(int64_t rows, int tokens, int64_t matrices) {
  const int64_t whole = blocks_of(blocks_of(rows, matrices), tokens) * matrices;
  if (matrices == 1) return whole;  // no groups to differ
  const int64_t half_more = blocks_of(2 * rows + tokens * matrices, 2 * tokens);
  return whole > half_more ? whole : half_more;
}

// Sets up the few-token kernel's tiles and tensor maps; false where TMA cannot
// read the operands or no pipeline fits.  `matrices`: how many weight matrices
// are likely to be read.
// `pair`: columns of two weight matrices lie in a stage (p.tmB is the first's map; the
// other's, alike, is the caller's).
inline bool few_maps(GroupedParams& p, ttc_dtype dtype, int tokens, int64_t matrices, const HostEnv& env, bool pair = false) {
  if (env.plain_loads || p.M == 0 || p.K == 0) return false;
  if (!tma_rows_ok(p.A, p.lda, 2) || !tma_rows_ok(p.B, p.ldb, 2) || !tma_stride_ok(p.groups, p.strideB, 2)) return false;
  p.tile_cols = few_tile_cols(few_blocks(p.M, tokens, matrices), p.N, env.sm_count, p.b_mn != 0, pair ? 64 : 128);
  p.col_blocks = (int)blocks_of(p.N, p.tile_cols);
  if ((blocks_of(p.M, tokens) + p.groups) * p.col_blocks > kSizeLimit) return false;
  p.b_stream = p.M <= matrices * tokens;
  p.stages = few_tokens_stages(tokens, (pair ? 2 : 1) * p.tile_cols, p.groups);
  if (p.stages < 2) return false;
  const CUtensorMapDataType dt = dtype == TTC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const int64_t mats = p.strideB != 0 ? p.groups : 1;
  return encode_matrices(&p.tmA, dt, 2, p.A, p.K, p.M, p.lda, 1, 0, kBK, few_tokens_box(tokens), sw) &&
         (p.b_mn ? encode_matrices(&p.tmB, dt, 2, p.B, p.N, p.K, p.ldb, mats, p.strideB, 64, 128, sw)
                 : encode_matrices(&p.tmB, dt, 2, p.B, p.K, p.N, p.ldb, mats, p.strideB, kBK, p.tile_cols, sw));
}

// Block of tokens for `rows` rows of `groups` groups; 0: not few.  Up to 64 rows a
// group on the average blocks of 64 are the faster where groups are alike: 64 rows of
// 8, 16, 32 and 64 groups, 4096 x 4096, 8192 x 1024, 1024 x 4096 and 1536 x 2048, 46, 50, 47
// and 74 us against the CTA-pair kernel's 52, 51, 51 and 76.  Uneven groups, of which the
// larger read their weights again, come out on either side (53, 58, 53 and 73 against 52,
// 51, 51 and 77).  Above, even ones need a second block: 72 rows 65, 85, 70 and 95 against
// 52, 51, 52 and 76.  (Blocks of 128 leave shared memory for three stages of the
// pipeline only: 87 to 94 us in the case above.)
inline int few_block(int64_t rows, int64_t groups) {
  const int64_t mean = blocks_of(rows, groups);
  if (rows <= 16 || mean <= 8) return 16;
  if (rows <= 32 || mean <= 16) return 32;
  return rows / groups <= 64 ? 64 : 0;
}

}  // namespace ttc
