// Block-scaled fp8 products for operands of any pitch and alignment: the kernel that
// is right for every case.  A CTA takes 64 x 64 of D; a block of 128 k of both
// operands is widened to fp16 (exact for both 8-bit formats) on its way into shared
// memory, eight warps multiply it with mma.sync into fresh fp32 sums, and those are
// added, scaled, to the tile's.  What is outside the group's rows and the operands'
// extents is zero and not loaded.
//
// Bound by the loads of single bytes.  Operands TMA can read take the other kernels.
#include <cuda_fp8.h>

#include "f8_blocks.cuh"
#include "grouped_common.cuh"

namespace ttc {

namespace {

constexpr int kTile = kF8PlainTile;
constexpr int kThreads = 256;  // eight warps: four of 16 rows by two of 32 columns
constexpr int kPitch = kF8Block + 8;  // halves; rows 16 bytes on from a multiple of all banks

__device__ __forceinline__ __half widen(uint8_t v, int e5m2) {
  return __half(__nv_cvt_fp8_to_halfraw(v, e5m2 ? __NV_E5M2 : __NV_E4M3));
}

// 64 rows of 128 k from (row0, k0) on.
__device__ __forceinline__ void load_tile(__half* dst, const uint8_t* src, int64_t ld, int row0, int row_end, int k0, int k_end,
                                          int e5m2) {
#pragma unroll 8
  for (int i = threadIdx.x; i < kTile * kF8Block; i += kThreads) {
    const int r = i / kF8Block, k = i % kF8Block;
    const bool in = row0 + r < row_end && k0 + k < k_end;
    dst[r * kPitch + k] = in ? widen(__ldg(src + (int64_t)(row0 + r) * ld + k0 + k), e5m2) : __float2half(0.0f);
  }
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

template <int OUT>
__device__ __forceinline__ float load_result(const void* c, int64_t i) {
  if constexpr (OUT == kF8ResultF32) return static_cast<const float*>(c)[i];
  return half_bits_to_float<OUT == kF8ResultBF16>(static_cast<const uint16_t*>(c)[i]);
}
template <int OUT>
__device__ __forceinline__ void store_result(void* d, int64_t i, float v) {
  if constexpr (OUT == kF8ResultF32)
    static_cast<float*>(d)[i] = v;
  else
    static_cast<uint16_t*>(d)[i] = (uint16_t)(pack2<OUT == kF8ResultBF16>(v, 0.0f) & 0xFFFFu);
}

template <int OUT>
__global__ void __launch_bounds__(kThreads) f8_plain_kernel(const __grid_constant__ F8Params p) {
  __shared__ __align__(16) __half sa[kTile * kPitch];
  __shared__ __align__(16) __half sb[kTile * kPitch];
  __shared__ int start[kMaxGroups / 8 + 2];
  __shared__ int dense[2];
  grid_dependency_wait();
  grid_dependents_launch();
  const GroupTable tb{p.offsets == nullptr ? dense : nullptr, start, 8, p.col_blocks};
  build_group_table<kTile>(p, tb);
  const int tiles = table_tiles(p, tb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp & 3, wc = warp >> 2, gid = lane >> 2, tig = lane & 3;
  const int blocks = (p.K + kF8Block - 1) / kF8Block;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const GroupedTile x = grouped_tile<kTile, false>(p, tb, t);
    const int row0 = x.lo + x.rb * kTile, col0 = x.cb * kTile;
    const uint8_t* b = static_cast<const uint8_t*>(p.B) + (int64_t)x.g * p.strideB;
    const float* scale_b = p.scale_b + (int64_t)x.g * p.stride_sb;
    // this thread's: rows row0 + wr * 16 + gid (+ 8), columns col0 + wc * 32 + n * 8 + tig * 2 (+ 1)
    float sums[4][4] = {};
    for (int kb = 0; kb < blocks; ++kb) {
      __syncthreads();
      load_tile(sa, static_cast<const uint8_t*>(p.A), p.lda, row0, x.hi, kb * kF8Block, p.K, p.a_e5m2);
      load_tile(sb, b, p.ldb, col0, p.N, kb * kF8Block, p.K, p.b_e5m2);
      __syncthreads();
      float c[4][4] = {};
#pragma unroll
      for (int k = 0; k < kF8Block; k += 16) {
        uint32_t a[4];
        const __half* ar = sa + (wr * 16 + gid) * kPitch + k + tig * 2;
        a[0] = *reinterpret_cast<const uint32_t*>(ar);
        a[1] = *reinterpret_cast<const uint32_t*>(ar + 8 * kPitch);
        a[2] = *reinterpret_cast<const uint32_t*>(ar + 8);
        a[3] = *reinterpret_cast<const uint32_t*>(ar + 8 * kPitch + 8);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const __half* br = sb + (wc * 32 + n * 8 + gid) * kPitch + k + tig * 2;
          const uint32_t bw[2] = {*reinterpret_cast<const uint32_t*>(br), *reinterpret_cast<const uint32_t*>(br + 8)};
          mma_16816(c[n], a, bw);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + wr * 16 + gid + h * 8;
        const float s = row < x.hi ? __ldg(p.scale_a + (int64_t)row * p.lds_a + kb) : 0.0f;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = col0 + wc * 32 + n * 8 + tig * 2 + e;
            const float w = col < p.N ? __ldg(scale_b + (int64_t)(col >> p.b_shift) * p.lds_b + kb) : 0.0f;
            sums[n][h * 2 + e] = fmaf(s * w, c[n][h * 2 + e], sums[n][h * 2 + e]);
          }
      }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = row0 + wr * 16 + gid + (e >> 1) * 8, col = col0 + wc * 32 + n * 8 + tig * 2 + (e & 1);
        if (row >= x.hi || col >= p.N) continue;
        float v = sums[n][e];
        if (p.C != nullptr) v += load_result<OUT>(p.C, (int64_t)row * p.ldc + col);
        if (p.bias != nullptr) v += __ldg(p.bias + (int64_t)x.g * p.stride_bias + col);
        store_result<OUT>(p.D, (int64_t)row * p.ldd + col, act_value(p.act, v));
      }
  }
}

template <int OUT>
cudaError_t launch(const F8Params& p, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f8_plain_kernel<OUT>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_f8_plain(const F8Params& p, F8Result out, int ctas, cudaStream_t stream) {
  switch (out) {
    case kF8ResultF16: return launch<kF8ResultF16>(p, ctas, stream);
    case kF8ResultBF16: return launch<kF8ResultBF16>(p, ctas, stream);
    case kF8ResultF32: return launch<kF8ResultF32>(p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ttc
