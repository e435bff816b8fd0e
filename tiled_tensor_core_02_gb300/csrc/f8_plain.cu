// Block-scaled fp8 products for operands of any pitch and alignment: the kernel that
// is right for every case, K == 0 among them.  A CTA takes 128 x 128 of D; a block of 128 k of
// both operands is widened to fp16 (exact for both 8-bit formats) on its way into shared
// memory, sixteen warps multiply it with mma.sync into fresh fp32 sums, and those are
// added, scaled, to the tile's.
//
// Sixteen bytes that start anywhere lie in one or two aligned 16-byte blocks; a thread
// loads those, the next block of K's while the MMAs run, and shifts them into place.  Only blocks
// that hold a byte of the row are read; what is outside the group's rows and the
// operands' extents is zero and not loaded.
//
// Bound by the loads and the widening, 4 us a block of K and tile: 8192 x 14336 x 4096 6.85 ms, 140
// TFLOP/s; 16 x 4096 x 4095 131 us.  Operands TMA can read take the other kernels.
#include <cuda_fp8.h>

#include <atomic>

#include "f8_blocks.cuh"
#include "grouped_common.cuh"

namespace ttc {

namespace {

constexpr int kTile = kF8PlainTile;
constexpr int kThreads = 512;         // sixteen warps: four of 32 rows by four of 32 columns
constexpr int kPitch = kF8Block + 8;  // halves: rows 16 bytes on from a multiple of all banks
constexpr int kOperandBytes = kTile * kPitch * 2;
constexpr int kTableInts = kMaxGroups / 8 + 2;
constexpr int kSmemBytes = 2 * kOperandBytes + (kTableInts + 2) * 4;
static_assert(kTile == 128, "pieces and warps cover the tile");

// A thread's pieces of 16 bytes of 128 rows by 128 k.
struct Pieces {
  static constexpr int kCount = kTile * kF8Block / 16 / kThreads;
  uint4 lo[kCount], hi[kCount];
  uint32_t phase[kCount];
  int n[kCount];  // bytes inside the operand

  __device__ __forceinline__ void load(const void* src, int64_t ld, int row0, int row_end, int k0, int k_end) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const int piece = threadIdx.x + i * kThreads;
      const int row = row0 + piece / (kF8Block / 16), k = k0 + piece % (kF8Block / 16) * 16;
      n[i] = row < row_end ? max(0, min(16, k_end - k)) : 0;
      const uintptr_t at = reinterpret_cast<uintptr_t>(src) + (int64_t)row * ld + k;
      phase[i] = (uint32_t)(at & 15);
      const uint4* blk = reinterpret_cast<const uint4*>(at - phase[i]);
      lo[i] = n[i] > 0 ? __ldg(blk) : make_uint4(0u, 0u, 0u, 0u);
      hi[i] = (int)phase[i] + n[i] > 16 ? __ldg(blk + 1) : make_uint4(0u, 0u, 0u, 0u);
    }
  }

  __device__ __forceinline__ void store(__half* dst, int e5m2) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      uint32_t x[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
      // bytes down by the phase: words by 2 and 1, then the rest
      const bool s8 = phase[i] & 8, s4 = phase[i] & 4;
#pragma unroll
      for (int k = 0; k < 6; ++k) x[k] = s8 ? x[k + 2] : x[k];
#pragma unroll
      for (int k = 0; k < 5; ++k) x[k] = s4 ? x[k + 1] : x[k];
      uint32_t y[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w = __funnelshift_r(x[k], x[k + 1], (phase[i] & 3) * 8);
        const int left = n[i] - k * 4;
        w = left >= 4 ? w : left <= 0 ? 0u : w & ((1u << (left * 8)) - 1u);
        y[2 * k] = widen2(w & 0xFFFFu, e5m2);
        y[2 * k + 1] = widen2(w >> 16, e5m2);
      }
      const int piece = threadIdx.x + i * kThreads;
      uint4* out = reinterpret_cast<uint4*>(dst + piece / (kF8Block / 16) * kPitch + piece % (kF8Block / 16) * 16);
      out[0] = make_uint4(y[0], y[1], y[2], y[3]);
      out[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }

  static __device__ __forceinline__ uint32_t widen2(uint32_t v, int e5m2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, e5m2 ? __NV_E5M2 : __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
  }
};

__device__ __forceinline__ void load_matrices(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__global__ void __launch_bounds__(kThreads, 1) f8_plain_kernel(const __grid_constant__ F8Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __half* sa = reinterpret_cast<__half*>(smem);
  __half* sb = reinterpret_cast<__half*>(smem + kOperandBytes);
  int* start = reinterpret_cast<int*>(smem + 2 * kOperandBytes);
  grid_dependency_wait();
  grid_dependents_launch();
  const GroupTable tb{p.offsets == nullptr ? start + kTableInts : nullptr, start, 8, p.col_blocks};
  build_group_table<kTile>(p, tb);
  const int tiles = table_tiles(p, tb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = (warp & 3) * 32, wc = (warp >> 2) * 32, gid = lane >> 2, tig = lane & 3;
  // ldmatrix: lanes 0 to 15 name A's rows, B's 16 rows come as two matrices of 8 by 8 k each
  const uint32_t a_at = smem_u32(sa + (wr + (lane & 15)) * kPitch + (lane >> 4) * 8);
  const uint32_t b_at = smem_u32(sb + (wc + (lane & 7) + (lane >> 4) * 8) * kPitch + ((lane >> 3) & 1) * 8);
  const int blocks = (p.K + kF8Block - 1) / kF8Block;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const GroupedTile x = grouped_tile<kTile, false>(p, tb, t);
    const int row0 = x.lo + x.rb * kTile, col0 = x.cb * kTile;
    const uint8_t* b = static_cast<const uint8_t*>(p.B) + (int64_t)x.g * p.strideB;
    const float* scale_b = p.scale_b + (int64_t)x.g * p.stride_sb;
    // this thread's: rows row0 + wr + m * 16 + gid (+ 8), columns col0 + wc + n * 8 + tig * 2 (+ 1)
    float sums[2][4][4] = {};
    Pieces pa, pb;
    if (blocks > 0) {
      pa.load(p.A, p.lda, row0, x.hi, 0, p.K);
      pb.load(b, p.ldb, col0, p.N, 0, p.K);
    }
    for (int kb = 0; kb < blocks; ++kb) {
      __syncthreads();
      pa.store(sa, p.a_e5m2);
      pb.store(sb, p.b_e5m2);
      __syncthreads();
      if (kb + 1 < blocks) {
        pa.load(p.A, p.lda, row0, x.hi, (kb + 1) * kF8Block, p.K);
        pb.load(b, p.ldb, col0, p.N, (kb + 1) * kF8Block, p.K);
      }
      float c[2][4][4] = {};
#pragma unroll
      for (int k = 0; k < kF8Block; k += 16) {
        uint32_t a[2][4], w[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) load_matrices(a_at + (m * 16 * kPitch + k) * 2, a[m]);
#pragma unroll
        for (int n = 0; n < 2; ++n) load_matrices(b_at + (n * 16 * kPitch + k) * 2, w[n]);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < 4; ++n) mma_16816(c[m][n], a[m], w[n / 2][n % 2 * 2], w[n / 2][n % 2 * 2 + 1]);
      }
      float by_column[4][2];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = col0 + wc + n * 8 + tig * 2 + e;
          by_column[n][e] = col < p.N ? __ldg(scale_b + (int64_t)(col >> p.b_shift) * p.lds_b + kb) : 0.0f;
        }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = row0 + wr + m * 16 + gid + h * 8;
          const float s = row < x.hi ? __ldg(p.scale_a + (int64_t)row * p.lds_a + kb) : 0.0f;
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              sums[m][n][h * 2 + e] = fmaf(s * by_column[n][e], c[m][n][h * 2 + e], sums[m][n][h * 2 + e]);
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = row0 + wr + m * 16 + gid + (e >> 1) * 8, col = col0 + wc + n * 8 + tig * 2 + (e & 1);
          if (row >= x.hi || col >= p.N) continue;
          float v = sums[m][n][e];
          if (p.C != nullptr) v += load_result<OUT>(p.C, (int64_t)row * p.ldc + col);
          if (p.bias != nullptr) v += __ldg(p.bias + (int64_t)x.g * p.stride_bias + col);
          store_result<OUT>(p.D, (int64_t)row * p.ldd + col, act_value(p.act, v));
        }
  }
}

template <int OUT>
cudaError_t launch(const F8Params& p, int ctas, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(f8_plain_kernel<OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, f8_plain_kernel<OUT>, p);
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
