// int8 products with a scale for each token and output channel (i8_rows.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace ttc {

// Types of a scaled int8 product.
enum I8ResultType : int { kI8ResultF16 = 0, kI8ResultBF16 = 1, kI8ResultF32 = 2 };

// D[i, j] = act(scaleA[i] scaleB[j] sum_k A[i, k] B[j, k] + bias[j])
struct I8ScaledParams {
  const int8_t* A;  // M x K, K contiguous
  int64_t lda;
  const int8_t* B;  // N x K, K contiguous
  int64_t ldb;
  const float* scaleA;
  const float* scaleB;
  const float* bias;
  void* D;
  int64_t ldd;
  int M, N, K;
  int act;
  int a_vec, b_vec;  // rows start on 16-byte boundaries
  int chunks;         // 256-wide chunks of K
  int split;          // CTAs of a cluster that share an output block's chunks, 1 to 8,
  int chunks_per_cta;  // and how many each takes
};

constexpr int kI8RowsFeatures = 128;  // output channels of a CTA
constexpr int kI8RowsTokens = 32;     // tokens of a CTA at most
constexpr int kI8RowsChunk = 256;     // of K

cudaError_t launch_i8_rows(const I8ScaledParams& p, I8ResultType out, cudaStream_t stream);

// The tensor-core kernel for some hundred tokens (i8_tokens.cu): token
// blocks of 32 and 64, tiles of 8 to 128 output channels, K shared by the
// `split` CTAs of a cluster.  A CTA holds an accumulator for every 1024 of its K,
// 256 columns of them: at most kI8TokenCols / block * 1024 of K a CTA.
struct I8TokensParams {
  CUtensorMap tmA;  // boxes of 128 bytes by `block` tokens
  CUtensorMap tmB;  // boxes of 128 bytes by tile_cols channels
  I8ScaledParams p;  // split, and K in stages of 128: chunks, chunks_per_cta
  int tile_cols, stages;
  uint32_t* err;
  uint64_t timeout_ns;
  int inject_stall;
};
constexpr int kI8TokenCols = 256;
constexpr int kI8TokenStage = 128;
int i8_tokens_stages(int block, int tile_cols);
int i8_tokens_clusters(int split);  // clusters of `split` CTAs that the device holds (0 on error)
cudaError_t launch_i8_tokens(const I8TokensParams& p, int block, I8ResultType out, cudaStream_t stream);

}  // namespace ttc
