// Products grouped by expert: what the kernels and their launchers share.
//
//   forward   D[i, :] = act(alpha A[i, :] B_g + bias_g)   for every row i of group g
//   wgrad     D_g     = alpha A[rows of g]^T B[rows of g] + beta C_g
//
// Group g's rows are offsets[g] .. offsets[g + 1] - 1 of A (and of D, or B).
// The offsets live on the device and are read there, so that the host need
// not wait for the router that wrote them: the kernels count the tiles
// themselves.  Offsets out of [0, M] are clamped to it and a group that ends
// before it starts is empty, so no offset leads out of the operands.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

namespace ttc {

// Largest number of groups: their tables fit in the shared memory that the
// widest kernel has left.
constexpr int kMaxGroups = 1024;

// Division by a number that the host knows, by Granlund and Montgomery's multiplication
// ("Division by invariant integers using multiplication", 1994):
// n / d = (n mul / 2^32 + n) / 2^shift for 0 <= n < 2^31, with shift = ceil(log2 d) and mul = 2^32 (2^shift - d) / d + 1.  A
// tile's place takes three of them; as integer divisions they were 0.4 us of a short
// tile's 2.3 in the epilogue.
struct FastDiv {
  uint32_t mul, shift;
};
constexpr FastDiv fast_div(uint32_t d) {
  FastDiv f{0, 0};
  while (((uint64_t)1 << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((((uint64_t)1 << f.shift) - d) << 32) / d) + 1);
  return f;
}

struct GroupedParams {
  CUtensorMap tmA;  // the kernels that load with TMA
  CUtensorMap tmB;
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb, strideB;
  const int32_t* offsets;  // null: all rows are one group's
  int groups;
  int M;  // rows of all groups together: the bound of every offset
  int N, K;
  int b_mn;          // forward: B_g is stored K x N (its columns contiguous)
  // tiles: blocks of D's columns, blocks of its rows (wgrad: per group; forward:
  // counted on the device), and how many row blocks share one column block
  // before the walk moves on (2^group_shift)
  int col_blocks, row_blocks, group_shift;
  int k_blocks;  // forward: 64-wide blocks of K
  float alpha, beta;
  const float* bias;
  int64_t stride_bias;
  int act;
  const void* C;
  int64_t ldc, strideC;
  void* D;
  int64_t ldd, strideD;
  int out_f32;  // wgrad: C and D are fp32
  int c_vec, d_vec;  // rows of C, D start on 16-byte boundaries
  int b_stream;  // forward: a group's weights are read by one block of rows as a rule
  int tile_cols, stages;  // few-token kernel: output columns of a tile, its pipeline's stages
  const float* scale_a;  // int8 products: a scale for each row of A and each column of B
  const float* scale_b;
  uint32_t* err;
  uint64_t timeout_ns;
  int inject_stall;
  // tiles of 2^group_shift row blocks; wgrad: tiles of a group, row blocks of its last band
  FastDiv by_band, by_group, by_rest;
};

// Gated feed-forward blocks run on the grouped kernels too (offsets null: dense).
//
//   forward  D = act(A B) * (A U): B and U the gate's and the other projection's
//            weights, alike in layout, pitch and stride; both products are kept
//            where gate and up are given.
//   grad     with dH = A B: dgate = dH * up * act'(gate), dup = dH * act(gate), and
//            D = act(gate) * up where D is given.
struct GatedParams : GroupedParams {
  CUtensorMap tmU;  // forward: the kernels that load with TMA
  const void* U;
  void* gate;  // M x N; forward: written (or null), grad: read
  void* up;
  int64_t ldp;
  int p_vec;
  void* dgate;  // grad: written; may be gate and up themselves
  void* dup;
  int64_t lddp;
  int dp_vec;
};
// The two as types of their own: kernels take one or the other.
struct GatedForward : GatedParams {};
struct GatedGrad : GatedParams {};
template <typename P>
constexpr bool kIsGatedForward = std::is_same<P, GatedForward>::value;
template <typename P>
constexpr bool kIsGatedGrad = std::is_same<P, GatedGrad>::value;
template <typename P>
constexpr bool kIsGated = kIsGatedForward<P> || kIsGatedGrad<P>;

// Tile of the kernel of CTA pairs: 256 x 256.
constexpr int kGroupedPairTile = 256;
int grouped_pair_clusters();
cudaError_t launch_grouped_pair(bool bf16, bool wgrad, const GroupedParams& p, int clusters, cudaStream_t stream);
// The same kernel for gated blocks: 256 x 128 tiles of D forward, 256 x 256 of its gradient.
constexpr int kGatedPairCols = 128;
cudaError_t launch_gated_pair(bool bf16, const GatedForward& p, int clusters, cudaStream_t stream);
cudaError_t launch_gated_pair(bool bf16, const GatedGrad& p, int clusters, cudaStream_t stream);
// The same kernel for int8 products: fp16 copies of the operands, all rows one
// group (no offsets), exact int32 sums, a scaled result (p.out_f32, or fp16 / bf16).
cudaError_t launch_pair_i8_scaled(bool bf16_out, const GroupedParams& p, int clusters, cudaStream_t stream);

// The kernel for few tokens: token tiles of 16, 32 and 64, tiles of 8 to 128
// output columns (gated forward: 64, as many rows of either weights a stage).  tmA
// has boxes of few_tokens_box tokens.  Stages that fit:
constexpr int few_tokens_box(int tokens) { return tokens < 32 ? tokens : 32; }
int few_tokens_stages(int tokens, int weight_rows, int groups);
cudaError_t launch_few_tokens(bool bf16, int tokens, const GroupedParams& p, int ctas, cudaStream_t stream);
cudaError_t launch_few_tokens(bool bf16, int tokens, const GatedForward& p, int ctas, cudaStream_t stream);
cudaError_t launch_few_tokens(bool bf16, int tokens, const GatedGrad& p, int ctas, cudaStream_t stream);

// Tile of the kernels that load with plain loads: 128 x 128.
constexpr int kGroupedPlainTile = 128;
cudaError_t launch_grouped_plain(bool bf16, bool wgrad, const GroupedParams& p, int ctas, cudaStream_t stream);
// Gated blocks: tiles of 128 rows by 64 columns of D forward, of 128 by 128 of its gradient.
constexpr int kGatedPlainCols = 64;
cudaError_t launch_gated_plain(bool bf16, const GatedForward& p, int ctas, cudaStream_t stream);
cudaError_t launch_gated_plain(bool bf16, const GatedGrad& p, int ctas, cudaStream_t stream);

}  // namespace ttc
