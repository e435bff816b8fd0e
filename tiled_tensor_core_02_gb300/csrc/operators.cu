// Host side of the grouped products, the quantization of rows and the scaled
// int8 product: argument checks, the choice of a kernel, tensor maps, launch.
// See include/ttc.h for the contract of each entry point.
#include <cstring>

#include "gemm_kernel.cuh"
#include "grouped.cuh"
#include "host.cuh"
#include "i8_rows.cuh"
#include "quantize.cuh"
#include "repack.cuh"
#include "ttc.h"

using namespace ttc;

namespace {

bool is_16bit(ttc_dtype t) { return t == TTC_F16 || t == TTC_BF16; }
bool is_dtype(ttc_dtype t) { return t == TTC_F16 || t == TTC_BF16 || t == TTC_I8 || t == TTC_F32; }
bool is_act(ttc_act a) { return a == TTC_ACT_NONE || a == TTC_ACT_RELU || a == TTC_ACT_GELU_TANH; }
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
int64_t at_least_1(int64_t x) { return x > 1 ? x : 1; }
int64_t blocks_of(int64_t x, int64_t b) { return (x + b - 1) / b; }

// Largest distance between two groups' matrices (elements).
constexpr int64_t kStrideLimit = 1ll << 40;

// Bytes from the first to the last element of `count` matrices `stride`
// elements apart, each rows x cols with pitch ld; capped well inside int64.
int64_t span_bytes(int64_t count, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int esize) {
  const __int128 n = ((__int128)(count - 1) * stride + (__int128)(rows - 1) * ld + cols) * esize;
  return n > ((__int128)1 << 60) ? 1ll << 60 : (int64_t)n;
}

// The walk over the tiles: bands of 2^shift row blocks.
void set_walk(GroupedParams& p, int64_t row_blocks, int64_t col_blocks, int shift) {
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
void common_params(GroupedParams& p, const HostEnv& env, int64_t groups, int64_t M, int64_t N, int64_t K, const void* A,
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
bool pair_maps(GroupedParams& p, bool wgrad, ttc_dtype dtype, const HostEnv& env) {
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
int few_tile_cols(int64_t blocks, int64_t n, int sm_count, bool cols_contiguous) {
  int64_t c = 128;
  for (int64_t waves = 1; waves <= 3; ++waves) {
    const int64_t room = waves * sm_count / blocks;  // tiles of a block of tokens
    if (room < 1 || blocks_of(n, room) > 128) continue;
    c = blocks_of(blocks_of(n, room), 8) * 8;
    break;
  }
  if (cols_contiguous) return c > 64 ? 128 : 64;
  return (int)c;
}

// Sets up the few-token kernel's tiles and tensor maps; false where TMA cannot
// read the operands or no pipeline fits.  `matrices`: how many weight matrices
// are likely to be read.  Groups near the mean take one block more as often as not
// (256 rows of 4 groups, 1088 x 1040: tiles for four blocks 16.0 us, for six 11.1).
bool few_maps(GroupedParams& p, ttc_dtype dtype, int tokens, int64_t matrices, const HostEnv& env) {
  if (env.plain_loads || p.M == 0 || p.K == 0) return false;
  if (!tma_rows_ok(p.A, p.lda, 2) || !tma_rows_ok(p.B, p.ldb, 2) || !tma_stride_ok(p.groups, p.strideB, 2)) return false;
  const int64_t whole = blocks_of(blocks_of(p.M, matrices), tokens) * matrices;
  const int64_t half_more = blocks_of(2 * p.M + tokens * matrices, 2 * tokens);
  p.tile_cols = few_tile_cols(whole > half_more ? whole : half_more, p.N, env.sm_count, p.b_mn != 0);
  p.col_blocks = (int)blocks_of(p.N, p.tile_cols);
  if ((blocks_of(p.M, tokens) + p.groups) * p.col_blocks > kSizeLimit) return false;
  p.b_stream = p.M <= matrices * tokens;
  p.stages = few_tokens_stages(tokens, p.tile_cols, p.groups);
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
int few_block(int64_t rows, int64_t groups) {
  const int64_t mean = blocks_of(rows, groups);
  if (rows <= 16 || mean <= 8) return 16;
  if (rows <= 32 || mean <= 16) return 32;
  return rows / groups <= 64 ? 64 : 0;
}

// The tensor-core kernel that widens the weights on its way: the tile's channels
// and the split of K whose CTAs are done soonest, and an estimate of its time in
// microseconds.  A stage takes 0.4 or HBM's share of an SM its bytes, whichever is
// more, a tile six besides and an exchange of sums 1.5 (measured within a tenth
// from 128 x 4096 x 4096, 13.8 us, to 1024 x 14336 x 4096, 219; blocks of 128 tokens
// took longer: 46 us against 38 for 128 x 14336 x 4096).  Clusters that do not fit next
// to the others wait for a whole wave, so the rounds are counted in clusters that
// the device holds (of eight CTAs 15, not 19: 256 x 512 x 2048 took 18 us instead
// of 10 where that was overlooked).  False where TMA cannot read the operands or K
// is too long for its accumulators.
bool i8_tokens_plan(I8TokensParams& q, int block, const HostEnv& env, double& cost_us) {
  I8ScaledParams& p = q.p;
  if (env.plain_loads || p.K == 0 || !tma_rows_ok(p.A, p.lda, 1) || !tma_rows_ok(p.B, p.ldb, 1)) return false;
  const int64_t stages = blocks_of(p.K, kI8TokenStage), most = kI8TokenCols / block * (1024 / kI8TokenStage);
  const int64_t blocks = blocks_of(p.M, block);
  if (blocks > 65535) return false;
  double best = 0.0;
  const int splits[6] = {1, 2, 3, 4, 6, 8};
  for (int split : splits) {
    const int64_t per = blocks_of(stages, split);
    if (per > most || split > stages) continue;
    const int64_t clusters = i8_tokens_clusters(split);
    if (clusters < 1) continue;
    for (int64_t waves = 1; waves <= 64; ++waves) {
      const int64_t room = waves * clusters / blocks;  // tiles
      if (room < 1 && waves < 64) continue;
      const int64_t cols = blocks_of(blocks_of(p.N, room < 1 ? 1 : room), 8) * 8;
      if (cols > 128 && waves < 64) continue;
      const int64_t c = cols > 128 ? 128 : cols;
      const double hbm = (double)c * kI8TokenStage / 44500.0, stage = hbm > 0.4 ? hbm : 0.4;
      const double cost = (double)blocks_of(blocks_of(p.N, c) * blocks, clusters) *
                          ((double)per * stage + 6.0 + (split > 1 ? 1.5 : 0.0));
      if (best == 0.0 || cost < best) {
        best = cost;
        q.tile_cols = (int)c;
        p.split = split;
        p.chunks = (int)stages;
        p.chunks_per_cta = (int)per;
      }
      break;
    }
  }
  cost_us = best;
  if (best == 0.0) return false;
  q.stages = i8_tokens_stages(block, q.tile_cols);
  if (q.stages < 1) return false;
  q.err = env.err;
  q.timeout_ns = env.timeout_ns;
  q.inject_stall = env.inject_stall;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return encode_matrices(&q.tmA, u8, 1, p.A, p.K, p.M, p.lda, 1, 0, 128, block, CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_matrices(&q.tmB, u8, 1, p.B, p.K, p.N, p.ldb, 1, 0, 128, q.tile_cols, CU_TENSOR_MAP_SWIZZLE_128B);
}

// int8 products of many tokens run on the CTA-pair kernel over fp16 copies of the
// operands in the workspace, rows padded to 16 elements.  The copies' 16-byte
// pieces and the tiles are counted in 32 bits.  Up to 256 tokens the kernel above
// is the faster (256 x 8192 x 8192 82 us, 260 here 96), where TMA can read the
// operands; else this one from 129 on (x 4416 x 1455: 128 tokens on plain loads
// 21 us, 192 31; 257 here 22).  Beyond 256 the estimates decide: about ten
// microseconds, the copies, and a round of tiles its share of K (measured within
// a tenth from 512 x 512 x 2048, 20 us, to 1024 x 8192 x 8192, 140).
struct I8Copies {
  int64_t ld;
  size_t b_off, bytes;
};
bool takes_i8_pair(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb) {
  const bool tma = tma_rows_ok(A, lda, 1) && tma_rows_ok(B, ldb, 1);
  return M > (tma ? 256 : 128) && N > 0 && K > 0 && blocks_of(K, 16) * (M > N ? M : N) < (1ll << 31) &&
         blocks_of(M, kGroupedPairTile) * blocks_of(N, kGroupedPairTile) < (1ll << 30);
}
double i8_pair_cost_us(int64_t M, int64_t N, int64_t K, int clusters) {
  const int64_t tiles = blocks_of(M, kGroupedPairTile) * blocks_of(N, kGroupedPairTile);
  return 10.0 + (double)(M + N) * (double)K / 1.5e6 + (double)blocks_of(tiles, clusters) * (double)K / 200.0;
}
I8Copies i8_copies(int64_t M, int64_t N, int64_t K) {
  I8Copies c;
  c.ld = blocks_of(K, 16) * 16;
  c.b_off = (size_t)(blocks_of(M * c.ld * 2, 256) * 256);
  c.bytes = c.b_off + (size_t)(blocks_of(N * c.ld * 2, 256) * 256);
  return c;
}

}  // namespace

extern "C" {

ttc_status ttc_gemm_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                            const int32_t* offsets, const void* B, int64_t ldb, int64_t strideB, ttc_layout layoutB,
                            void* D, int64_t ldd, float alpha, const float* bias, int64_t strideBias, ttc_act act,
                            ttc_dtype dtype, void* stream) {
  if (groups < 0 || M < 0 || N < 0 || K < 0 || strideB < 0 || strideBias < 0) return TTC_ERR_INVALID_ARG;
  if (layoutB != TTC_ROW_MAJOR && layoutB != TTC_COL_MAJOR) return TTC_ERR_INVALID_ARG;
  if (!is_act(act) || !is_dtype(dtype)) return TTC_ERR_INVALID_ARG;
  if (!is_16bit(dtype)) return TTC_ERR_UNSUPPORTED;
  if (groups == 0 || M == 0 || N == 0) return TTC_OK;
  if (lda < at_least_1(K) || ldb < at_least_1(layoutB == TTC_ROW_MAJOR ? N : K) || ldd < N) return TTC_ERR_INVALID_ARG;
  if (offsets == nullptr || D == nullptr || (K > 0 && (A == nullptr || B == nullptr))) return TTC_ERR_INVALID_ARG;
  if (!aligned(offsets, 4) || !aligned(D, 2) || !aligned(bias, 4) || (K > 0 && (!aligned(A, 2) || !aligned(B, 2))))
    return TTC_ERR_INVALID_ARG;
  if (groups > kMaxGroups || M > kSizeLimit || N > kSizeLimit || K > kSizeLimit || lda > kSizeLimit ||
      ldb > kSizeLimit || ldd > kSizeLimit || strideB > kStrideLimit || strideBias > kStrideLimit)
    return TTC_ERR_UNSUPPORTED;
  const int64_t d_bytes = span_bytes(1, 0, M, ldd, N, 2);
  if (K > 0) {
    const int64_t b_rows = layoutB == TTC_ROW_MAJOR ? K : N, b_cols = layoutB == TTC_ROW_MAJOR ? N : K;
    if (byte_ranges_overlap(D, d_bytes, A, span_bytes(1, 0, M, lda, K, 2)) ||
        byte_ranges_overlap(D, d_bytes, B, span_bytes(groups, strideB, b_rows, ldb, b_cols, 2)))
      return TTC_ERR_INVALID_ARG;
  }
  const int64_t col_blocks = blocks_of(N, kGroupedPlainTile);
  if ((blocks_of(M, kGroupedPlainTile) + groups) * col_blocks > kSizeLimit) return TTC_ERR_UNSUPPORTED;

  HostEnv env;
  const ttc_status st = host_env(env);
  if (st != TTC_OK) return st;
  GroupedParams p;
  common_params(p, env, groups, M, N, K, A, lda, B, ldb, offsets);
  p.strideB = strideB;
  p.b_mn = layoutB == TTC_ROW_MAJOR;
  p.k_blocks = (int)blocks_of(K, kBK);
  p.alpha = alpha;
  p.bias = bias;
  p.stride_bias = strideBias;
  p.act = (int)act;
  p.D = D;
  p.ldd = ldd;
  p.d_vec = aligned(D, 16) && ldd % 8 == 0;
  const int64_t likely = groups < M ? groups : M;  // groups with rows, as far as the host knows
  const int block = few_block(M, likely);
  if (block != 0 && few_maps(p, dtype, block, likely, env)) {
    const int64_t tiles = (blocks_of(M, block) + likely) * p.col_blocks;
    if (launch_few_tokens(dtype == TTC_BF16, block, p, (int)(tiles < env.sm_count ? tiles : env.sm_count),
                          static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return TTC_ERR_CUDA;
    count_launches(1);
    return TTC_OK;
  }
  if (pair_maps(p, false, dtype, env)) {
    const int clusters = grouped_pair_clusters();
    if (clusters <= 0) return TTC_ERR_CUDA;
    set_walk(p, 0, blocks_of(N, kGroupedPairTile), 3);
    p.b_stream = M <= groups * kGroupedPairTile;
    const int64_t tiles = (blocks_of(M, kGroupedPairTile) + (groups < M ? groups : M)) * p.col_blocks;
    if (launch_grouped_pair(dtype == TTC_BF16, false, p, (int)(2 * tiles < clusters ? 2 * tiles : clusters),
                            static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return TTC_ERR_CUDA;
    count_launches(1);
    return TTC_OK;
  }
  set_walk(p, 0, col_blocks, 4);
  const int64_t tiles = (blocks_of(M, kGroupedPlainTile) + (groups < M ? groups : M)) * col_blocks;
  const int ctas = (int)(tiles < env.sm_count ? tiles : env.sm_count);
  if (launch_grouped_plain(dtype == TTC_BF16, false, p, ctas, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return TTC_ERR_CUDA;
  count_launches(1);
  return TTC_OK;
}

ttc_status ttc_gemm_grouped_wgrad(int64_t groups, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                                  const void* B, int64_t ldb, const int32_t* offsets, const void* C, int64_t ldc,
                                  int64_t strideC, void* D, int64_t ldd, int64_t strideD, float alpha, float beta,
                                  ttc_dtype dtype, ttc_dtype out_dtype, void* stream) {
  if (groups < 0 || M < 0 || N < 0 || K < 0 || strideC < 0 || strideD < 0) return TTC_ERR_INVALID_ARG;
  if (!is_dtype(dtype) || !is_dtype(out_dtype)) return TTC_ERR_INVALID_ARG;
  if (!is_16bit(dtype) || (out_dtype != dtype && out_dtype != TTC_F32)) return TTC_ERR_UNSUPPORTED;
  if (groups == 0 || N == 0 || K == 0) return TTC_OK;
  if (lda < K || ldb < N || ldd < N || (beta != 0.0f && (C == nullptr || ldc < N))) return TTC_ERR_INVALID_ARG;
  if (offsets == nullptr || D == nullptr || (M > 0 && (A == nullptr || B == nullptr))) return TTC_ERR_INVALID_ARG;
  const int esize = out_dtype == TTC_F32 ? 4 : 2;
  if (!aligned(offsets, 4) || !aligned(D, esize) || (beta != 0.0f && !aligned(C, esize)) ||
      (M > 0 && (!aligned(A, 2) || !aligned(B, 2))))
    return TTC_ERR_INVALID_ARG;
  // the groups' D may not overlap
  if (groups > 1 && (__int128)strideD < (__int128)(K - 1) * ldd + N) return TTC_ERR_INVALID_ARG;
  if (groups > kMaxGroups || M > kSizeLimit || N > kSizeLimit || K > kSizeLimit || lda > kSizeLimit ||
      ldb > kSizeLimit || ldd > kSizeLimit || strideD > kStrideLimit ||
      (beta != 0.0f && (ldc > kSizeLimit || strideC > kStrideLimit)))
    return TTC_ERR_UNSUPPORTED;
  const int64_t d_bytes = span_bytes(groups, strideD, K, ldd, N, esize);
  if (beta != 0.0f && !(C == D && ldc == ldd && (strideC == strideD || groups == 1)) &&
      byte_ranges_overlap(D, d_bytes, C, span_bytes(groups, strideC, K, ldc, N, esize)))
    return TTC_ERR_INVALID_ARG;
  if (M > 0 && (byte_ranges_overlap(D, d_bytes, A, span_bytes(1, 0, M, lda, K, 2)) ||
                byte_ranges_overlap(D, d_bytes, B, span_bytes(1, 0, M, ldb, N, 2))))
    return TTC_ERR_INVALID_ARG;
  const int64_t row_blocks = blocks_of(K, kGroupedPlainTile), col_blocks = blocks_of(N, kGroupedPlainTile);
  if (row_blocks * col_blocks > kSizeLimit / groups) return TTC_ERR_UNSUPPORTED;

  HostEnv env;
  const ttc_status st = host_env(env);
  if (st != TTC_OK) return st;
  GroupedParams p;
  common_params(p, env, groups, M, N, K, A, lda, B, ldb, offsets);
  p.b_mn = 1;
  set_walk(p, row_blocks, col_blocks, 4);
  p.alpha = alpha;
  p.beta = beta;
  p.out_f32 = out_dtype == TTC_F32;
  if (beta != 0.0f) {
    p.C = C;
    p.ldc = ldc;
    p.strideC = strideC;
    p.c_vec = aligned(C, 16) && ldc * esize % 16 == 0 && (groups == 1 || strideC * esize % 16 == 0);
  }
  p.D = D;
  p.ldd = ldd;
  p.strideD = strideD;
  p.d_vec = aligned(D, 16) && ldd * esize % 16 == 0 && (groups == 1 || strideD * esize % 16 == 0);
  if (pair_maps(p, true, dtype, env)) {
    const int clusters = grouped_pair_clusters();
    if (clusters <= 0) return TTC_ERR_CUDA;
    set_walk(p, blocks_of(K, kGroupedPairTile), blocks_of(N, kGroupedPairTile), 3);
    const int64_t tiles = groups * p.row_blocks * p.col_blocks;
    if (launch_grouped_pair(dtype == TTC_BF16, true, p, (int)(2 * tiles < clusters ? 2 * tiles : clusters),
                            static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return TTC_ERR_CUDA;
    count_launches(1);
    return TTC_OK;
  }
  const int64_t tiles = groups * row_blocks * col_blocks;
  const int ctas = (int)(tiles < env.sm_count ? tiles : env.sm_count);
  if (launch_grouped_plain(dtype == TTC_BF16, true, p, ctas, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return TTC_ERR_CUDA;
  count_launches(1);
  return TTC_OK;
}

ttc_status ttc_quantize_rows(int64_t rows, int64_t cols, const void* X, int64_t ldx, ttc_dtype dtype, int8_t* Q,
                             int64_t ldq, float* scale, void* stream) {
  if (rows < 0 || cols < 0 || !is_dtype(dtype)) return TTC_ERR_INVALID_ARG;
  if (dtype == TTC_I8) return TTC_ERR_UNSUPPORTED;
  if (rows == 0) return TTC_OK;
  const int esize = dtype == TTC_F32 ? 4 : 2;
  if (scale == nullptr || !aligned(scale, 4)) return TTC_ERR_INVALID_ARG;
  if (cols > 0 && (X == nullptr || Q == nullptr || !aligned(X, esize))) return TTC_ERR_INVALID_ARG;
  if (ldx < cols || ldq < cols) return TTC_ERR_INVALID_ARG;
  if (rows > kSizeLimit || cols > kSizeLimit || ldx > kSizeLimit || ldq > kSizeLimit) return TTC_ERR_UNSUPPORTED;
  if (cols > 0) {
    const int64_t x_bytes = span_bytes(1, 0, rows, ldx, cols, esize), q_bytes = span_bytes(1, 0, rows, ldq, cols, 1);
    if (byte_ranges_overlap(X, x_bytes, Q, q_bytes) || byte_ranges_overlap(scale, rows * 4, Q, q_bytes) ||
        byte_ranges_overlap(scale, rows * 4, X, x_bytes))
      return TTC_ERR_INVALID_ARG;
  }
  HostEnv env;
  const ttc_status st = host_env(env);
  if (st != TTC_OK) return st;
  QuantParams p{X, ldx, Q, ldq, scale, (int)rows, (int)cols};
  const QuantIn in = dtype == TTC_F32 ? kQuantF32 : dtype == TTC_BF16 ? kQuantBF16 : kQuantF16;
  if (launch_quantize_rows(p, in, env.sm_count, static_cast<cudaStream_t>(stream)) != cudaSuccess) return TTC_ERR_CUDA;
  count_launches(1);
  return TTC_OK;
}

size_t ttc_gemm_i8_scaled_workspace_size(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const int8_t* B,
                                         int64_t ldb, const void* D, int64_t ldd, ttc_dtype out_dtype) {
  (void)D;
  if (M <= 0 || N <= 0 || K <= 0 || K > TTC_I8_SCALED_MAX_K || lda < K || ldb < K || ldd < N || M > kSizeLimit ||
      N > kSizeLimit || !(is_16bit(out_dtype) || out_dtype == TTC_F32))
    return 0;
  return takes_i8_pair(M, N, K, A, lda, B, ldb) ? i8_copies(M, N, K).bytes : 0;
}

ttc_status ttc_gemm_i8_scaled(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda, const float* scaleA,
                              const int8_t* B, int64_t ldb, const float* scaleB, void* D, int64_t ldd,
                              const float* bias, ttc_act act, ttc_dtype out_dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || !is_act(act) || !is_dtype(out_dtype)) return TTC_ERR_INVALID_ARG;
  if (out_dtype == TTC_I8) return TTC_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return TTC_OK;
  if (lda < at_least_1(K) || ldb < at_least_1(K) || ldd < N) return TTC_ERR_INVALID_ARG;
  if (scaleA == nullptr || scaleB == nullptr || D == nullptr || (K > 0 && (A == nullptr || B == nullptr)))
    return TTC_ERR_INVALID_ARG;
  const int esize = out_dtype == TTC_F32 ? 4 : 2;
  if (!aligned(scaleA, 4) || !aligned(scaleB, 4) || !aligned(bias, 4) || !aligned(D, esize)) return TTC_ERR_INVALID_ARG;
  if (M > kSizeLimit || N > kSizeLimit || lda > kSizeLimit || ldb > kSizeLimit || ldd > kSizeLimit ||
      K > TTC_I8_SCALED_MAX_K)
    return TTC_ERR_UNSUPPORTED;
  const int64_t d_bytes = span_bytes(1, 0, M, ldd, N, esize);
  if (K > 0 && (byte_ranges_overlap(D, d_bytes, A, span_bytes(1, 0, M, lda, K, 1)) ||
                byte_ranges_overlap(D, d_bytes, B, span_bytes(1, 0, N, ldb, K, 1))))
    return TTC_ERR_INVALID_ARG;

  HostEnv env;
  const ttc_status st = host_env(env);
  if (st != TTC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const I8ResultType out = out_dtype == TTC_F32 ? kI8ResultF32 : out_dtype == TTC_BF16 ? kI8ResultBF16 : kI8ResultF16;
  I8TokensParams q;
  std::memset(&q, 0, sizeof q);
  I8ScaledParams& p = q.p;
  p.A = A;
  p.lda = lda;
  p.B = B;
  p.ldb = ldb;
  p.scaleA = scaleA;
  p.scaleB = scaleB;
  p.bias = bias;
  p.D = D;
  p.ldd = ldd;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.act = (int)act;
  p.a_vec = aligned(A, 16) && lda % 16 == 0;
  p.b_vec = aligned(B, 16) && ldb % 16 == 0;
  const int block = M <= 32 ? 32 : 64;
  double few_us = 0.0;
  const bool few = M > 16 && i8_tokens_plan(q, block, env, few_us);
  if (workspace != nullptr && aligned(workspace, 256) && takes_i8_pair(M, N, K, A, lda, B, ldb) && !env.plain_loads) {
    const I8Copies copies = i8_copies(M, N, K);
    const int clusters = grouped_pair_clusters();
    if (clusters <= 0) return TTC_ERR_CUDA;
    if (workspace_bytes >= copies.bytes && !(few && few_us < i8_pair_cost_us(M, N, K, clusters))) {
      uint8_t* ws = static_cast<uint8_t*>(workspace);
      const WidenSpec specs[2] = {{A, lda, M, K, ws, copies.ld}, {B, ldb, N, K, ws + copies.b_off, copies.ld}};
      GroupedParams f;
      common_params(f, env, 1, M, N, K, ws, copies.ld, ws + copies.b_off, copies.ld, nullptr);
      if (!pair_maps(f, false, TTC_F16, env)) return TTC_ERR_CUDA;
      set_walk(f, 0, blocks_of(N, kGroupedPairTile), 3);
      f.k_blocks = (int)blocks_of(K, kBK);
      f.alpha = 1.0f;
      f.bias = bias;
      f.act = (int)act;
      f.scale_a = scaleA;
      f.scale_b = scaleB;
      f.out_f32 = out == kI8ResultF32;
      f.D = D;
      f.ldd = ldd;
      f.d_vec = aligned(D, 16) && ldd * esize % 16 == 0;
      const int64_t tiles = blocks_of(M, kGroupedPairTile) * f.col_blocks;
      if (launch_widen_i8(specs, 2, env.sm_count, s) != cudaSuccess ||
          launch_pair_i8_scaled(out == kI8ResultBF16, f, (int)(2 * tiles < clusters ? 2 * tiles : clusters), s) != cudaSuccess)
        return TTC_ERR_CUDA;
      count_launches(2);
      return TTC_OK;
    }
  }
  if (few) {
    if (launch_i8_tokens(q, block, out, s) != cudaSuccess) return TTC_ERR_CUDA;
    count_launches(1);
    return TTC_OK;
  }
  // CTAs for two on each SM, where a cluster of up to eight leaves each CTA two
  // chunks of K at least.
  p.chunks = (int)blocks_of(K, kI8RowsChunk);
  const int64_t blocks = blocks_of(N, kI8RowsFeatures) * blocks_of(M, kI8RowsTokens);
  int64_t split = 2ll * env.sm_count / blocks;
  if (split > p.chunks / 2) split = p.chunks / 2;
  p.split = (int)(split < 1 ? 1 : split > 8 ? 8 : split);
  p.chunks_per_cta = (int)blocks_of(p.chunks, p.split);
  if (launch_i8_rows(p, out, s) != cudaSuccess) return TTC_ERR_CUDA;
  count_launches(1);
  return TTC_OK;
}

}  // extern "C"
