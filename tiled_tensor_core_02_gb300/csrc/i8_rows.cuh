// int8 products with a scale for each token and output channel (i8_rows.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace ttc {

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

enum I8Out : int { kI8OutF16 = 0, kI8OutBF16 = 1, kI8OutF32 = 2 };

constexpr int kI8RowsFeatures = 128;  // output channels of a CTA
constexpr int kI8RowsTokens = 32;     // tokens of a CTA at most
constexpr int kI8RowsChunk = 256;     // of K

cudaError_t launch_i8_rows(const I8ScaledParams& p, I8Out out, cudaStream_t stream);

}  // namespace ttc
