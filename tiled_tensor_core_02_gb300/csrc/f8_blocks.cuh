// Products of 8-bit floats with a fp32 scale for each block of 128: what the kernels
// and their launchers share.
//
//   D[i, j] = act(sum over b of sA[i, b] sB_g[j / r, b] P_b[i, j] + C[i, j] + bias_g[j]),
//   P_b[i, j] = sum of A[i, k] B_g[j, k] over the k of block b (128 of them),
//
// r = 1 or 128 rows of B a scale.  Rows are grouped as in ttc_gemm_grouped, or all one
// group's (offsets null).  P_b is the tensor cores' fp32 sum; the scales' product is rounded to
// nearest, one fused multiply-add a block, in order, adds P_b times it to the sum; C, bias and the
// activation are fp32.
#pragma once
#include "grouped.cuh"

namespace ttc {

constexpr int kF8Block = 128;

enum F8Result : int { kF8ResultF16 = 0, kF8ResultBF16 = 1, kF8ResultF32 = 2 };

// A, B: bytes; pitches and strideB in elements of them.  C and D have the result's type.
struct F8Params : GroupedParams {
  int a_e5m2, b_e5m2;  // else e4m3
  int64_t lds_a, lds_b, stride_sb;  // scale_a, scale_b: pitches, and from one group's to the next
  int b_shift;  // rows of B a scale: 2^0 or 2^7
  int sa_vec, sb_vec;  // rows of scales start on 16-byte boundaries
};

// Any pitch and alignment: tiles of 128 x 128, warp-level products of fp16 copies.
constexpr int kF8PlainTile = 128;
cudaError_t launch_f8_plain(const F8Params& p, F8Result out, int ctas, cudaStream_t stream);

// Few tokens: blocks of 16, 32 and 64 of a group's, tiles of 8 to 128 output columns.  tmA
// has boxes of few_tokens_box tokens.  Stages that fit:
int f8_tokens_stages(int tokens, int tile_cols, int groups);
cudaError_t launch_f8_tokens(const F8Params& p, F8Result out, int tokens, int ctas, cudaStream_t stream);

// CTA pairs: tiles of 256 x 256 (kGroupedPairTile) of operands TMA can read.
int f8_pair_clusters();
cudaError_t launch_f8_pair(const F8Params& p, F8Result out, int clusters, cudaStream_t stream);

// Rows (or blocks of 128 rows) of 8-bit floats from 16- or 32-bit ones.
struct F8QuantParams {
  const void* x;
  int64_t ldx;
  uint8_t* q;
  int64_t ldq;
  float* scale;
  int64_t lds;
  int rows, cols;  // of x
};
enum F8QuantIn : int { kF8QuantF16 = 0, kF8QuantBF16 = 1, kF8QuantF32 = 2 };
cudaError_t launch_f8_quantize(const F8QuantParams& p, F8QuantIn in, bool e5m2, bool square, bool turn, int sm_count,
                               cudaStream_t stream);

}  // namespace ttc
