// Host side of the block-scaled 8-bit floats: argument checks, the choice of a kernel,
// tensor maps, launch.  See include/ttc.h for the contract of each entry point.
#include "f8_blocks.cuh"
#include "operators_host.cuh"

using namespace ttc;

namespace {

bool is_f8(ttc_dtype t) { return t == TTC_F8_E4M3 || t == TTC_F8_E5M2; }
bool is_any_dtype(ttc_dtype t) { return is_dtype(t) || is_f8(t); }

// Tensor maps of the operands, a block of 128 k by so many rows a box; false where TMA
// cannot read them.
bool f8_maps(F8Params& p, int rows_a, int rows_b, const HostEnv& env) {
  if (env.plain_loads || p.K == 0) return false;
  if (!tma_rows_ok(p.A, p.lda, 1) || !tma_rows_ok(p.B, p.ldb, 1) || !tma_stride_ok(p.groups, p.strideB, 1)) return false;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  return encode_matrices(&p.tmA, u8, 1, p.A, p.K, p.M, p.lda, 1, 0, kF8Block, rows_a, sw) &&
         encode_matrices(&p.tmB, u8, 1, p.B, p.K, p.N, p.ldb, p.strideB != 0 ? p.groups : 1, p.strideB, kF8Block, rows_b, sw);
}

// Block of tokens of the few-token kernel, 0 for CTA pairs: as for 16-bit operands up to 64
// rows a group, and with more wherever blocks of 64 make one wave of tiles, whose narrow
// tiles keep all SMs at work (rows x 4096 x 4096: 65 to 256 12.4 to 12.7 us against 18.9 to 20.8;
// 128 x 8192 x 8192 24.2 against 35.6, 256 x 1024 x 4096 13.8 against 18.5; two waves, 320 x
// 4096 x 4096, 24.1 against 20.8; 1024 rows of 8 groups, 4096 x 4096, four waves, 50.9 against 41.5).
int f8_few_block(int64_t rows, int64_t n, int64_t groups, int sm_count) {
  const int block = few_block(rows, groups);
  if (block != 0) return block;
  return few_blocks(rows, 64, groups) * blocks_of(n, 128) <= sm_count ? 64 : 0;
}

// The few-token kernel's tiles; false where no pipeline fits.  `matrices`: how many groups
// are likely to have rows.
bool f8_few_tiles(F8Params& p, int tokens, int64_t matrices, const HostEnv& env) {
  p.tile_cols = few_tile_cols(few_blocks(p.M, tokens, matrices), p.N, env.sm_count, false, 128);
  p.col_blocks = (int)blocks_of(p.N, p.tile_cols);
  p.stages = f8_tokens_stages(tokens, p.tile_cols, p.groups);
  p.b_stream = p.M <= matrices * tokens;
  return p.stages >= 2 && (blocks_of(p.M, tokens) + p.groups) * p.col_blocks <= kSizeLimit;
}

}  // namespace

extern "C" {

ttc_status ttc_quantize_blocks(int64_t rows, int64_t cols, const void* X, int64_t ldx, ttc_dtype dtype, int block_rows,
                               int transpose, void* Q, int64_t ldq, ttc_dtype q_dtype, float* scale, int64_t lds,
                               void* stream) {
  if (rows < 0 || cols < 0 || !is_any_dtype(dtype) || !is_any_dtype(q_dtype)) return TTC_ERR_INVALID_ARG;
  if ((block_rows != 1 && block_rows != kF8Block) || (transpose != 0 && transpose != 1)) return TTC_ERR_INVALID_ARG;
  if (!(is_16bit(dtype) || dtype == TTC_F32) || !is_f8(q_dtype)) return TTC_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return TTC_OK;
  const int64_t q_rows = transpose ? cols : rows, q_cols = transpose ? rows : cols;
  const int64_t s_rows = blocks_of(q_rows, block_rows), s_cols = blocks_of(q_cols, kF8Block);
  const int esize = dtype == TTC_F32 ? 4 : 2;
  if (X == nullptr || Q == nullptr || scale == nullptr || !aligned(X, esize) || !aligned(scale, 4)) return TTC_ERR_INVALID_ARG;
  if (ldx < cols || ldq < q_cols || lds < s_cols) return TTC_ERR_INVALID_ARG;
  if (rows > kSizeLimit || cols > kSizeLimit || ldx > kSizeLimit || ldq > kSizeLimit || lds > kSizeLimit)
    return TTC_ERR_UNSUPPORTED;
  const int64_t x_bytes = span_bytes(1, 0, rows, ldx, cols, esize), q_bytes = span_bytes(1, 0, q_rows, ldq, q_cols, 1),
                s_bytes = span_bytes(1, 0, s_rows, lds, s_cols, 4);
  if (byte_ranges_overlap(X, x_bytes, Q, q_bytes) || byte_ranges_overlap(scale, s_bytes, Q, q_bytes) ||
      byte_ranges_overlap(scale, s_bytes, X, x_bytes))
    return TTC_ERR_INVALID_ARG;
  HostEnv env;
  const ttc_status st = host_env(env);
  if (st != TTC_OK) return st;
  const F8QuantParams p{X, ldx, static_cast<uint8_t*>(Q), ldq, scale, lds, (int)rows, (int)cols};
  const F8QuantIn in = dtype == TTC_F32 ? kF8QuantF32 : dtype == TTC_BF16 ? kF8QuantBF16 : kF8QuantF16;
  if (launch_f8_quantize(p, in, q_dtype == TTC_F8_E5M2, block_rows != 1, transpose != 0, env.sm_count,
                         static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return TTC_ERR_CUDA;
  count_launches(1);
  return TTC_OK;
}

ttc_status ttc_gemm_f8_blocks(int64_t groups, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, ttc_dtype typeA,
                              const float* scaleA, int64_t ldsa, const int32_t* offsets, const void* B, int64_t ldb,
                              int64_t strideB, ttc_dtype typeB, const float* scaleB, int64_t ldsb, int64_t strideSB,
                              int block_rows_b, const void* C, int64_t ldc, void* D, int64_t ldd, const float* bias,
                              int64_t strideBias, ttc_act act, ttc_dtype out_dtype, void* stream) {
  if (groups < 0 || M < 0 || N < 0 || K < 0 || strideB < 0 || strideSB < 0 || strideBias < 0) return TTC_ERR_INVALID_ARG;
  if (!is_any_dtype(typeA) || !is_any_dtype(typeB) || !is_any_dtype(out_dtype) || !is_act(act)) return TTC_ERR_INVALID_ARG;
  if (block_rows_b != 1 && block_rows_b != kF8Block) return TTC_ERR_INVALID_ARG;
  if (!is_f8(typeA) || !is_f8(typeB) || !(is_16bit(out_dtype) || out_dtype == TTC_F32)) return TTC_ERR_UNSUPPORTED;
  if (groups == 0 || M == 0 || N == 0) return TTC_OK;
  if (offsets == nullptr && groups != 1) return TTC_ERR_INVALID_ARG;
  const int64_t k_blocks = blocks_of(K, kF8Block), sb_rows = blocks_of(N, block_rows_b);
  const int esize = out_dtype == TTC_F32 ? 4 : 2;
  if (D == nullptr || ldd < N || !aligned(D, esize) || !aligned(offsets, 4) || !aligned(bias, 4)) return TTC_ERR_INVALID_ARG;
  if (C != nullptr && (ldc < N || !aligned(C, esize))) return TTC_ERR_INVALID_ARG;
  if (K > 0 && (A == nullptr || B == nullptr || scaleA == nullptr || scaleB == nullptr || !aligned(scaleA, 4) ||
                !aligned(scaleB, 4) || lda < K || ldb < K || ldsa < k_blocks || ldsb < k_blocks))
    return TTC_ERR_INVALID_ARG;
  if (groups > kMaxGroups || M > kSizeLimit || N > kSizeLimit || K > kSizeLimit || ldd > kSizeLimit ||
      (C != nullptr && ldc > kSizeLimit) || strideB > kStrideLimit || strideSB > kStrideLimit || strideBias > kStrideLimit ||
      (K > 0 && (lda > kSizeLimit || ldb > kSizeLimit || ldsa > kSizeLimit || ldsb > kSizeLimit)))
    return TTC_ERR_UNSUPPORTED;
  const int64_t col_blocks = blocks_of(N, kF8PlainTile);
  if ((blocks_of(M, kF8PlainTile) + groups) * col_blocks > kSizeLimit) return TTC_ERR_UNSUPPORTED;
  const int64_t d_bytes = span_bytes(1, 0, M, ldd, N, esize);
  if (K > 0 && (byte_ranges_overlap(D, d_bytes, A, span_bytes(1, 0, M, lda, K, 1)) ||
                byte_ranges_overlap(D, d_bytes, B, span_bytes(groups, strideB, N, ldb, K, 1)) ||
                byte_ranges_overlap(D, d_bytes, scaleA, span_bytes(1, 0, M, ldsa, k_blocks, 4)) ||
                byte_ranges_overlap(D, d_bytes, scaleB, span_bytes(groups, strideSB, sb_rows, ldsb, k_blocks, 4))))
    return TTC_ERR_INVALID_ARG;
  if (C != nullptr && !(C == D && ldc == ldd) && byte_ranges_overlap(D, d_bytes, C, span_bytes(1, 0, M, ldc, N, esize)))
    return TTC_ERR_INVALID_ARG;
  if (offsets != nullptr && byte_ranges_overlap(D, d_bytes, offsets, (groups + 1) * 4)) return TTC_ERR_INVALID_ARG;
  if (bias != nullptr && byte_ranges_overlap(D, d_bytes, bias, span_bytes(groups, strideBias, 1, N, N, 4)))
    return TTC_ERR_INVALID_ARG;

  HostEnv env;
  const ttc_status st = host_env(env);
  if (st != TTC_OK) return st;
  F8Params p;
  std::memset(&p, 0, sizeof p);
  common_params(p, env, groups, M, N, K, A, lda, B, ldb, offsets);
  p.strideB = strideB;
  p.k_blocks = (int)k_blocks;
  p.alpha = 1.0f;
  p.a_e5m2 = typeA == TTC_F8_E5M2;
  p.b_e5m2 = typeB == TTC_F8_E5M2;
  p.scale_a = scaleA;
  p.lds_a = ldsa;
  p.scale_b = scaleB;
  p.lds_b = ldsb;
  p.stride_sb = strideSB;
  p.b_shift = block_rows_b == 1 ? 0 : 7;
  p.sa_vec = aligned(scaleA, 16) && ldsa % 4 == 0;
  p.sb_vec = aligned(scaleB, 16) && ldsb % 4 == 0 && (groups == 1 || strideSB % 4 == 0);
  p.bias = bias;
  p.stride_bias = strideBias;
  p.act = (int)act;
  p.C = C;
  p.ldc = ldc;
  p.D = D;
  p.ldd = ldd;
  p.out_f32 = out_dtype == TTC_F32;
  p.d_vec = aligned(D, 16) && ldd * esize % 16 == 0;
  p.c_vec = C != nullptr && aligned(C, 16) && ldc * esize % 16 == 0;
  const F8Result out = out_dtype == TTC_F32 ? kF8ResultF32 : out_dtype == TTC_BF16 ? kF8ResultBF16 : kF8ResultF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t likely = groups < M ? groups : M;  // groups with rows, as far as the host knows
  const int block = f8_few_block(M, N, likely, env.sm_count);
  if (block != 0 && f8_few_tiles(p, block, likely, env) && f8_maps(p, few_tokens_box(block), p.tile_cols, env)) {
    const int64_t tiles = (blocks_of(M, block) + likely) * p.col_blocks;
    if (launch_f8_tokens(p, out, block, (int)(tiles < env.sm_count ? tiles : env.sm_count), s) != cudaSuccess)
      return TTC_ERR_CUDA;
    count_launches(1);
    return TTC_OK;
  }
  if (f8_maps(p, 128, 128, env)) {
    const int clusters = f8_pair_clusters();
    if (clusters <= 0) return TTC_ERR_CUDA;
    set_walk(p, 0, blocks_of(N, kGroupedPairTile), 3);
    p.b_stream = M <= groups * kGroupedPairTile;
    const int64_t tiles = (blocks_of(M, kGroupedPairTile) + likely) * p.col_blocks;
    if (launch_f8_pair(p, out, (int)(2 * tiles < clusters ? 2 * tiles : clusters), s) != cudaSuccess) return TTC_ERR_CUDA;
    count_launches(1);
    return TTC_OK;
  }
  set_walk(p, 0, col_blocks, 4);
  const int64_t tiles = (blocks_of(M, kF8PlainTile) + likely) * col_blocks, room = env.sm_count;
  if (launch_f8_plain(p, out, (int)(tiles < room ? tiles : room), s) != cudaSuccess) return TTC_ERR_CUDA;
  count_launches(1);
  return TTC_OK;
}

}  // extern "C"
