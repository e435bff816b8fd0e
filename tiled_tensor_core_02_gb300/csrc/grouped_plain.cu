// Grouped products for operands of any pitch and alignment: the kernel that is
// right for every case.  One CTA per 128 x 128 tile, persistent; four warps
// bring the operands into 128-byte-swizzled shared memory with plain loads
// (generic_load_tile: vectors of 8 elements where rows are aligned, elements
// otherwise, zeros outside the group's rows and the operand's extents), one
// thread issues tcgen05.mma, four warps drain the accumulator.  In the
// gradient of the weights the reduction runs over the group's rows, so both
// operands lie with the reduction outermost, as the MMA takes them too.
//
// It is bound by the plain loads' latency; operands TMA can read take the
// other kernels.
#include "grouped_common.cuh"

#include <atomic>

namespace ttc {

namespace {

constexpr int kTile = kGroupedPlainTile;
constexpr int kStages = 4;
constexpr int kThreads = 32 * (4 + 1 + 4);  // producers, MMA issuer, epilogue
constexpr int kOperandBytes = kTile * kBK * 2;
constexpr int kTableBytes = 2 * (kMaxGroups + 4) * 4;
constexpr int kSmemBytes = 1024 + kStages * 2 * kOperandBytes + 256 + kTableBytes;

template <bool BF16, bool WGRAD>
__global__ void __launch_bounds__(kThreads, 1) grouped_plain_kernel(const __grid_constant__ GroupedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + kStages * kOperandBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sB + kStages * kOperandBytes);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* tmem_full = bars + 2 * kStages;
  uint64_t* tmem_empty = bars + 2 * kStages + 2;
  uint64_t* stall_bar = bars + 2 * kStages + 4;
  uint64_t* drain_bar = bars + 2 * kStages + 5;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 6);
  int* offs = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 256);
  int* start = offs + kMaxGroups + 4;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{p.err, p.timeout_ns};
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 128);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tmem_full[a], 1);
      mbar_init(&tmem_empty[a], 4);
    }
    mbar_init(stall_bar, 1);
    mbar_init(drain_bar, 1);
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();
  const GroupTable tb{offs, WGRAD ? nullptr : start, 1, p.col_blocks};
  build_group_table<kTile>(p, tb);
  const int tiles = WGRAD ? p.groups * p.row_blocks * p.col_blocks : table_tiles(p, tb);

  if (warp < 4) {
    // ---------------------------------------------------------------- producers
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const GroupedTile x = grouped_tile<kTile, WGRAD>(p, tb, t);
      const int nkb = WGRAD ? (x.hi - x.lo + kBK - 1) / kBK : p.k_blocks;
      const int n0 = x.cb * kTile;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) {
          ok = false;
          break;
        }
        uint8_t* a = sA + stage * kOperandBytes;
        uint8_t* b = sB + stage * kOperandBytes;
        if constexpr (WGRAD) {
          const int r0 = x.lo + kb * kBK;
          generic_load_tile<kBK, kTile, false>(a, p.A, p.lda, r0, x.rb * kTile, x.hi, p.K, p.a_vec != 0, threadIdx.x);
          generic_load_tile<kBK, kTile, false>(b, p.B, p.ldb, r0, n0, x.hi, p.N, p.b_vec != 0, threadIdx.x);
        } else {
          const uint16_t* bg = static_cast<const uint16_t*>(p.B) + (int64_t)x.g * p.strideB;
          generic_load_tile<kTile, kBK, false>(a, p.A, p.lda, x.lo + x.rb * kTile, kb * kBK, x.hi, p.K, p.a_vec != 0,
                                               threadIdx.x);
          if (p.b_mn)
            generic_load_tile<kBK, kTile, false>(b, bg, p.ldb, kb * kBK, n0, p.K, p.N, p.b_vec != 0, threadIdx.x);
          else
            generic_load_tile<kTile, kBK, false>(b, bg, p.ldb, n0, kb * kBK, p.N, p.K, p.b_vec != 0, threadIdx.x);
        }
        fence_proxy_async_smem();
        mbar_arrive(&full[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 4) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const bool b_mn = WGRAD || p.b_mn != 0;
      const uint32_t idesc = idesc_f16(BF16, WGRAD, b_mn, kTile, kTile);
      const uint64_t a0 = smem_desc_sw128(smem_u32(sA), WGRAD ? 8192u : 16u, 1024);
      const uint64_t b0 = smem_desc_sw128(smem_u32(sB), b_mn ? 8192u : 16u, 1024);
      const uint64_t a_step = WGRAD ? 2048u >> 4 : 32u >> 4, b_step = b_mn ? 2048u >> 4 : 32u >> 4;
      bool ok = true, any = false;
      if (p.inject_stall) ok = mbar_wait(stall_bar, 0, wc);  // nothing arrives here
      int stage = 0, it = 0;
      uint32_t phase = 0;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++it) {
        const GroupedTile x = grouped_tile<kTile, WGRAD>(p, tb, t);
        const int nkb = WGRAD ? (x.hi - x.lo + kBK - 1) / kBK : p.k_blocks;
        const int acc = it & 1;
        if (!mbar_wait(&tmem_empty[acc], ((it >> 1) & 1) ^ 1u, wc)) break;
        tc_fence_after();
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&full[stage], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = a0 + (uint32_t)(stage * (kOperandBytes >> 4));
          const uint64_t bd = b0 + (uint32_t)(stage * (kOperandBytes >> 4));
#pragma unroll
          for (int k = 0; k < kBK / kUmmaK; ++k)
            mma_f16(tmem_base + acc * kTile, ad + k * a_step, bd + k * b_step, idesc, (kb | k) != 0);
          any = true;
          mma_commit(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (nkb == 0)
          mbar_arrive(&tmem_full[acc]);
        else
          mma_commit(&tmem_full[acc]);
      }
      if (any) {
        mma_commit(drain_bar);
        drain_wait(drain_bar, 0, 100000000ull);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int esize = p.out_f32 ? 4 : 2;
    int it = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
      const GroupedTile x = grouped_tile<kTile, WGRAD>(p, tb, t);
      const bool has_k = WGRAD ? x.hi > x.lo : p.k_blocks > 0;
      const int acc = it & 1;
      // D's row of this thread, and the group's first element of C and D
      const int r = x.rb * kTile + q * 32 + lane;
      const int64_t row = WGRAD ? r : (int64_t)x.lo + r;
      const bool row_ok = WGRAD ? r < p.K : row < x.hi;
      char* d_row = static_cast<char*>(p.D) + ((WGRAD ? (int64_t)x.g * p.strideD : 0) + row * p.ldd) * esize;
      const char* c_row =
          p.C != nullptr ? static_cast<const char*>(p.C) + ((int64_t)x.g * p.strideC + row * p.ldc) * esize : nullptr;
      const float* bias = p.bias != nullptr ? p.bias + (int64_t)x.g * p.stride_bias : nullptr;
      if (!mbar_wait(&tmem_full[acc], (it >> 1) & 1, wc)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kTile / 32; ++c) {
        const int col0 = x.cb * kTile + c * 32;
        uint32_t w[32];
        if (has_k) {
          tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(q * 32) << 16) + acc * kTile + c * 32, w);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = 0u;
        }
        if (c == kTile / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tmem_empty[acc]);
        }
        const int n = min(32, p.N - col0);
        if (row_ok && n > 0) {
          float v[32];
          grouped_values<BF16>(p, w, c_row != nullptr ? c_row + (int64_t)col0 * esize : nullptr,
                               bias != nullptr ? bias + col0 : nullptr, n, v);
          store_row<BF16>(p, v, d_row + (int64_t)col0 * esize, n);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 256);
  }
}

template <bool BF16, bool WGRAD>
cudaError_t launch(const GroupedParams& p, int ctas, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(grouped_plain_kernel<BF16, WGRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
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
  e = cudaLaunchKernelEx(&cfg, grouped_plain_kernel<BF16, WGRAD>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_plain(bool bf16, bool wgrad, const GroupedParams& p, int ctas, cudaStream_t stream) {
  if (wgrad) return bf16 ? launch<true, true>(p, ctas, stream) : launch<false, true>(p, ctas, stream);
  return bf16 ? launch<true, false>(p, ctas, stream) : launch<false, false>(p, ctas, stream);
}

}  // namespace ttc
