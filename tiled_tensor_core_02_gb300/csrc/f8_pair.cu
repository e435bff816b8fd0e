// Block-scaled fp8 products on CTA pairs: 256 x 256 tiles by tcgen05.mma.cta_group::2
// (kind::f8f6f4), operands by TMA.
//
// The scales change with every 128 of K, so the tensor cores add up one such block at
// a time: each goes into one of two accumulators in tensor memory, and the epilogue warps
// add it, scaled, to the tile's sums in their registers (a thread has one row and 128
// columns) while the tensor cores fill the other.  For that they have 512 clocks, the
// MMAs' time at fp8's rate; a warp takes its four loads of 32 columns one ahead of the
// additions, two columns an instruction.  The sums take most of a thread's registers, so the
// four warps that load and issue hand theirs over.
//
// Scales of A come a block of four of K ahead, one row a lane.  B's are one for all of
// a warp's columns (blocks of 128 rows), or one a column: then a lane fetches four
// columns' and hands them round through the warp's staging block.
#include <atomic>
#include <type_traits>

#include "f8_blocks.cuh"
#include "grouped_common.cuh"

namespace ttc {

namespace {

constexpr int kTile = kGroupedPairTile;
constexpr int kShareBytes = 128 * kF8Block;  // a CTA's share of one operand's block
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarpCount = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarpCount);
constexpr int kStagingBytes = kEpiWarpCount * 4096;
constexpr int kBarBytes = 256;
constexpr int kTableInts = 384;
// Scales by column take 4 KB an epilogue warp: a stage less.
template <bool BY_COLUMN>
constexpr int kStagesOf = BY_COLUMN ? 5 : 6;
constexpr int kSmemBytes = 1024 + 6 * 2 * kShareBytes + kStagingBytes + kBarBytes + kTableInts * 4;
static_assert(kEpiWarpCount * 4096 <= 2 * kShareBytes, "a stage has room for the scales");
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert((kMaxGroups + 3) / 4 + 1 <= kTableInts, "a table of every fourth group's tiles has room");
// Registers a thread: at launch, of the first four warps, of the epilogue's.
constexpr int kRegsLaunch = 168, kRegsFew = 72, kRegsMany = 216;
static_assert(128 * kRegsFew + (kThreads - 128) * kRegsMany <= kThreads * kRegsLaunch, "the shares fit the launch's registers");
constexpr int kLoad = 32;  // columns of an accumulator a load
constexpr int kAhead = 4;  // blocks of K whose scales are fetched together

// Where an epilogue warp's part of a tile lies.
struct Part {
  int g, col0, at, width;  // group; first column of D and of the accumulator; columns (128, of half a tile 64)
  int64_t row;
  int rows;
};
__device__ __forceinline__ Part part_of(const F8Params& p, const GroupTable& tb, const PairWalk& walk, int t, uint32_t rank, int q,
                                        int half) {
  const PairItem item = pair_item<false>(p, tb, walk, t);
  const GroupedTile& x = item.x;
  const int r0 = x.rb * kTile + (int)rank * 128 + q * 32;
  Part e;
  e.g = x.g;
  e.width = item.half < 0 ? kTile / 2 : kTile / 4;
  e.at = half * e.width;
  e.col0 = x.cb * kTile + max(item.half, 0) * (kTile / 2) + e.at;
  e.row = (int64_t)x.lo + r0;
  e.rows = max(0, min(32, x.hi - x.lo - r0));
  return e;
}

// Scales of kAhead blocks of K from kb0 on: this lane's row of A, and B's for the warp's
// columns where that is one.
template <bool BY_COLUMN>
struct Scales {
  float a[kAhead], b[BY_COLUMN ? 1 : kAhead];

  __device__ __forceinline__ void load(const F8Params& p, const Part& e, int lane, int kb0) {
    const float* sa = p.scale_a + (e.row + lane) * p.lds_a + kb0;
    const float* sb = p.scale_b + (int64_t)e.g * p.stride_sb + (int64_t)(e.col0 >> 7) * p.lds_b + kb0;
    const int n = p.k_blocks - kb0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      a[i] = lane < e.rows && i < n ? __ldg(sa + i) : 0.0f;
      if constexpr (!BY_COLUMN) b[i] = e.col0 < p.N && i < n ? __ldg(sb + i) : 0.0f;
    }
  }
};

// The same of B by column into shared memory, [block][128 columns], without a register;
// copy_async_wait and a __syncwarp come before their use.
__device__ __forceinline__ void fetch_columns(const F8Params& p, const Part& e, int lane, int kb0, float* dst) {
  const float* sb = p.scale_b + (int64_t)e.g * p.stride_sb + kb0;
  const int n = p.k_blocks - kb0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int at = c * 32 + lane, col = e.col0 + at;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (col < p.N && i < n)
        copy_async_4(dst + i * 128 + at, sb + (int64_t)col * p.lds_b + i);
      else
        dst[i * 128 + at] = 0.0f;
    }
  }
}

// C's 32 rows of 128 bytes into the staging block, zeros outside; a __syncwarp comes
// before their use and before the block is written again.
template <typename T>
__device__ __forceinline__ void stage_c(const F8Params& p, const T* c0, int rows, int n, int lane, uint8_t* sb) {
  constexpr int kElems = 16 / (int)sizeof(T), kCols = 128 / (int)sizeof(T);
  n = max(0, min(n, kCols));
  const int whole = p.c_vec ? n & ~(kElems - 1) : 0;
  const int piece = lane & 7, r0 = lane >> 3;
  if (piece * kElems < whole) {
    const T* src = c0 + (int64_t)r0 * p.ldc + piece * kElems;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = i * 4 + r0 < rows ? *reinterpret_cast<const uint4*>(src + (int64_t)(i * 4) * p.ldc) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(sb + staged<32>(i * 4 + r0, piece)) = v[i];
  }
  for (int c = whole + lane; c < n; c += 32) {
#pragma unroll 4
    for (int r = 0; r < 32; ++r)
      *reinterpret_cast<T*>(sb + staged<32>(r, c / kElems) + (c % kElems) * sizeof(T)) = r < rows ? c0[(int64_t)r * p.ldc + c] : T{};
  }
}

__device__ __forceinline__ void load_columns(uint32_t taddr, uint32_t (&w)[32]) { tmem_ld_32x32b_x32(taddr, w); }
__device__ __forceinline__ void load_columns(uint32_t taddr, uint32_t (&w)[16]) { tmem_ld_32x32b_x16<0>(taddr, w); }

// OUT: F8Result; BY_COLUMN: B has a scale for each row (a column of D).
template <int OUT, bool BY_COLUMN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) f8_pair_kernel(const __grid_constant__ F8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kStages = kStagesOf<BY_COLUMN>;
  uint8_t* sA = smem;
  uint8_t* sB = sA + kStages * kShareBytes;
  uint8_t* staging = smem + 6 * 2 * kShareBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStagingBytes);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* tmem_full = bars + 2 * kStages;
  uint64_t* tmem_empty = bars + 2 * kStages + 2;
  uint64_t* stall_bar = bars + 2 * kStages + 4;
  uint64_t* drain_bar = bars + 2 * kStages + 5;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 6);
  // what the producer tells the MMA issuer about a stage: whether the tile is half a tile
  int* stage_info = reinterpret_cast<int*>(bars + 2 * kStages + 7);
  static_assert((2 * kStages + 7) * 8 + kStages * 4 <= kBarBytes, "barrier area");
  int* table = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);
  // the whole table where it has room, else only every fourth group's first tile
  GroupTable tb{nullptr, nullptr, 1, p.col_blocks};
  if (2 * (p.groups + 1) <= kTableInts) {
    tb.offs = table;
    tb.start = table + p.groups + 1;
  } else {
    tb.start = table;
    tb.step = 4;
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
  const WaitCtx wc{p.err, p.timeout_ns};

  if (warp == 0) {
    if (lane < kStages) {
      mbar_init(&full[lane], 1);
      mbar_init(&empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&tmem_full[lane], 1);
      mbar_init(&tmem_empty[lane], 2 * kEpiWarpCount);
    }
    if (lane == 0) {
      mbar_init(stall_bar, 1);
      mbar_init(drain_bar, 1);
      prefetch_tmap(&p.tmA);
      prefetch_tmap(&p.tmB);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();
  build_group_table<kTile>(p, tb);
  const PairWalk walk = pair_walk(table_tiles(p, tb), num_pairs);

  if (warp < kEpiWarp0) {
    registers_down<kRegsFew>();
    if (warp == 0) {
      // ---------------------------------------------------------------- producer (both CTAs)
      if (lane == 0) {
        const uint64_t keep = policy_evict_last();
        const uint64_t pol_b = p.b_stream ? policy_evict_first() : keep;
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;  // stages armed on `full` (even CTA)
        bool ok = true;
        for (int t = pair; ok && t < walk.items; t += num_pairs) {
          const PairItem item = pair_item<false>(p, tb, walk, t);
          const GroupedTile& x = item.x;
          // of half a tile the MMA reads 64 columns, the first of the 128 that are loaded
          const int n0 = x.cb * kTile + (item.half < 0 ? (int)rank * 128 : item.half * 128 + (int)rank * 64);
          const int m0 = x.lo + x.rb * kTile + (int)rank * 128;
          // whether this CTA's, and the other's, rows of A hold any of the group
          const bool a_on = m0 < x.hi;
          const int shares = (x.lo + x.rb * kTile + 128 < x.hi ? 2 : 1) + 2;
          const int zb = p.strideB != 0 ? x.g : 0;
          for (int kb = 0; kb < p.k_blocks; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) {
              ok = false;
              break;
            }
            const uint32_t full_leader = mapa_shared(smem_u32(&full[stage]), 0);
            if (leader) {
              stage_info[stage] = item.half >= 0;
              mbar_arrive_expect_tx(full + stage, shares * kShareBytes);
              armed |= 1u << stage;
              armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            }
            if (a_on) tma_load_3d_pair(sA + stage * kShareBytes, &p.tmA, kb * kF8Block, m0, 0, full_leader, keep);
            tma_load_3d_pair(sB + stage * kShareBytes, &p.tmB, kb * kF8Block, n0, zb, full_leader, pol_b);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // a stage completes once both CTAs' loads for it have landed
        if (leader)
          drain_ring(full, kStages, armed, armed_parity);
        else
          drain_odd_cta(wc);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer (even CTA)
      if (leader && lane == 0) {
        const uint32_t idesc_whole = idesc_f8(p.a_e5m2 != 0, p.b_e5m2 != 0, kTile, kTile);
        const uint32_t idesc_half = idesc_f8(p.a_e5m2 != 0, p.b_e5m2 != 0, kTile, kTile / 2);
        const uint64_t a0 = smem_desc_sw128(smem_u32(sA), 16u, 1024);
        const uint64_t b0 = smem_desc_sw128(smem_u32(sB), 16u, 1024);
        bool ok = true, any = false;
        if (p.inject_stall) ok = mbar_wait(stall_bar, 0, wc);  // nothing arrives here
        int stage = 0, it = 0;
        uint32_t phase = 0;
        for (int t = pair; ok && t < walk.items; t += num_pairs) {
          for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
            const int acc = it & 1;
            // the first use of each accumulator passes at once
            if (!mbar_wait_cluster(&tmem_empty[acc], ((it >> 1) & 1) ^ 1u, wc) || !mbar_wait(&full[stage], phase, wc)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t idesc = stage_info[stage] != 0 ? idesc_half : idesc_whole;
            const uint64_t ad = a0 + (uint32_t)stage * (kShareBytes >> 4), bd = b0 + (uint32_t)stage * (kShareBytes >> 4);
#pragma unroll
            for (int k = 0; k < kF8Block / 32; ++k) mma_f8_pair(tmem_base + acc * kTile, ad + k * 2, bd + k * 2, idesc, k != 0);
            any = true;
            mma_commit_pair(&empty[stage], 0x3);
            mma_commit_pair(&tmem_full[acc], 0x3);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (any) {
          // every MMA must have finished with both CTAs' TMEM before it is freed
          mma_commit_pair(drain_bar, 0x1);
          drain_wait(drain_bar, 0, 100000000ull);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    registers_up<kRegsMany>();
    using T = typename std::conditional<OUT == kF8ResultF32, float, uint16_t>::type;
    constexpr int kUnit = 128 / (int)sizeof(T);  // columns that 128 bytes hold
    constexpr int kElems = 16 / (int)sizeof(T);
    const int ew = warp - kEpiWarp0, q = warp & 3, half = ew >> 2;  // quarter of the rows, half of the columns
    uint8_t* sb = staging + ew * 4096;
    const uint32_t tmem_mine = tmem_base + ((uint32_t)(q * 32) << 16);
    int it = 0;
    bool ok = true;
    Part e{};
    Scales<BY_COLUMN> next;
    // the scales of this chunk of K and of the next
    float* columns = reinterpret_cast<float*>(smem + kStages * 2 * kShareBytes + ew * 4096);
    int buffer = 0;
    const auto fetch = [&](int kb0) {
      next.load(p, e, lane, kb0);
      if constexpr (BY_COLUMN) {
        buffer ^= kAhead * 128;
        fetch_columns(p, e, lane, kb0, columns + buffer);
      }
    };
    if (pair < walk.items) {
      e = part_of(p, tb, walk, pair, rank, q, half);
      fetch(0);
    }
    for (int t = pair; ok && t < walk.items; t += num_pairs) {
      uint64_t sums[kTile / 4];  // pairs of columns
#pragma unroll
      for (int j = 0; j < kTile / 4; ++j) sums[j] = 0ull;
      const Part me = e;
      for (int kb0 = 0; ok && kb0 < p.k_blocks; kb0 += kAhead) {
        float s[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s[i] = BY_COLUMN ? next.a[i] : next.a[i] * next.b[BY_COLUMN ? 0 : i];
        const float* by_column = columns + buffer;
        if constexpr (BY_COLUMN) {
          copy_async_wait();
          __syncwarp();
        }
        if (kb0 + kAhead < p.k_blocks) {
          fetch(kb0 + kAhead);
        } else if (t + num_pairs < walk.items) {
          e = part_of(p, tb, walk, t + num_pairs, rank, q, half);
          fetch(0);
        }
        const int blocks = min(kAhead, p.k_blocks - kb0);
#pragma unroll 1
        for (int i = 0; i < blocks; ++i) {
          const int acc = it & 1;
          if (!mbar_wait_warp(&tmem_full[acc], (it >> 1) & 1, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t from = tmem_mine + me.at + acc * kTile;
          const float scale = s[0];
#pragma unroll
          for (int k = 0; k + 1 < kAhead; ++k) s[k] = s[k + 1];
          const uint64_t scale2 = pair_of(scale, scale);
          // two loads of kLoad columns in turn
          uint32_t w[2][kLoad];
          load_columns(from, w[0]);
#pragma unroll
          for (int c = 0; c < kTile / 2 / kLoad; ++c) {
            tmem_ld_wait_for(w[c & 1]);
            if (c + 1 < kTile / 2 / kLoad) {
              load_columns(from + (c + 1) * kLoad, w[(c + 1) & 1]);
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
            }
#pragma unroll
            for (int j = 0; j < kLoad / 2; j += 2) {
              uint64_t f0 = scale2, f1 = scale2;
              if constexpr (BY_COLUMN) {
                const float4 v = *reinterpret_cast<const float4*>(by_column + i * 128 + c * kLoad + j * 2);
                f0 = mul_pair(pair_of(v.x, v.y), scale2);
                f1 = mul_pair(pair_of(v.z, v.w), scale2);
              }
              const uint32_t* v = w[c & 1] + 2 * j;
              fma_pair(pair_of(__uint_as_float(v[0]), __uint_as_float(v[1])), f0, sums[c * (kLoad / 2) + j]);
              fma_pair(pair_of(__uint_as_float(v[2]), __uint_as_float(v[3])), f1, sums[c * (kLoad / 2) + j + 1]);
            }
          }
          ++it;
        }
      }
      if (!ok) break;
      const int cols = min(me.width, p.N - me.col0);
      float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.bias != nullptr) bias = four_columns(p.bias + (int64_t)me.g * p.stride_bias + me.col0, lane, cols);
      T* d = static_cast<T*>(p.D) + me.row * p.ldd + me.col0;
      const T* c0 = static_cast<const T*>(p.C) + me.row * p.ldc + me.col0;
#pragma unroll
      for (int u = 0; u < kTile / 2 / kUnit; ++u) {
        if (cols <= u * kUnit || me.rows <= 0) continue;
        if (p.C != nullptr) {
          stage_c(p, c0 + u * kUnit, me.rows, cols - u * kUnit, lane, sb);
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kUnit / kElems; ++i) {
          uint4* piece = reinterpret_cast<uint4*>(sb + staged<32>(lane, i));
          float v[kElems];
#pragma unroll
          for (int k = 0; k < kElems / 2; ++k) halves_of(sums[(u * kUnit + i * kElems) / 2 + k], v[2 * k], v[2 * k + 1]);
          if (p.C != nullptr) {
            const uint4 old = *piece;
            const uint32_t cw[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (OUT == kF8ResultF32) {
                v[k] += __uint_as_float(cw[k]);
              } else {
                v[2 * k] += half_bits_to_float<OUT == kF8ResultBF16>((uint16_t)(cw[k] & 0xFFFFu));
                v[2 * k + 1] += half_bits_to_float<OUT == kF8ResultBF16>((uint16_t)(cw[k] >> 16));
              }
            }
          }
          if (p.bias != nullptr) {
#pragma unroll
            for (int k = 0; k < kElems / 4; ++k) {
              const int src = (u * kUnit + i * kElems) / 4 + k;
              v[4 * k] += __shfl_sync(0xFFFFFFFFu, bias.x, src);
              v[4 * k + 1] += __shfl_sync(0xFFFFFFFFu, bias.y, src);
              v[4 * k + 2] += __shfl_sync(0xFFFFFFFFu, bias.z, src);
              v[4 * k + 3] += __shfl_sync(0xFFFFFFFFu, bias.w, src);
            }
          }
          if (p.act != kActNone) {
#pragma unroll
            for (int k = 0; k < kElems; ++k) v[k] = act_value(p.act, v[k]);
          }
          if constexpr (OUT == kF8ResultF32)
            *piece = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
          else
            *piece = make_uint4(pack2<OUT == kF8ResultBF16>(v[0], v[1]), pack2<OUT == kF8ResultBF16>(v[2], v[3]),
                                pack2<OUT == kF8ResultBF16>(v[4], v[5]), pack2<OUT == kF8ResultBF16>(v[6], v[7]));
        }
        __syncwarp();
        copy_out<T, 4>(p, sb, d + u * kUnit, me.rows, cols - u * kUnit, lane);
        __syncwarp();
      }
    }
    if constexpr (BY_COLUMN) copy_async_wait();  // after an error some may be on their way
  }

  __syncthreads();
  cluster_sync();  // the pair's MMAs, remote arrivals and loads are all finished
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int OUT, bool BY_COLUMN>
cudaError_t prepare() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, f8_pair_kernel<OUT, BY_COLUMN>);
    if (e != cudaSuccess) return e;
    if (a.numRegs != kRegsLaunch) return cudaErrorInvalidKernelImage;  // the warps would wait for registers that there are not
    e = cudaFuncSetAttribute(f8_pair_kernel<OUT, BY_COLUMN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  return cudaSuccess;
}

template <int OUT, bool BY_COLUMN>
cudaError_t launch(const F8Params& p, int clusters, cudaStream_t stream) {
  cudaError_t e = prepare<OUT, BY_COLUMN>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, f8_pair_kernel<OUT, BY_COLUMN>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Pairs that can be resident at once (0 on error): one CTA fits an SM whatever the variant.
int f8_pair_clusters() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load();
  if (n > 0) return n;
  if (prepare<kF8ResultBF16, false>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaOccupancyMaxActiveClusters(&n, f8_pair_kernel<kF8ResultBF16, false>, &cfg) != cudaSuccess) return 0;
  known[dev].store(n);
  return n;
}

cudaError_t launch_f8_pair(const F8Params& p, F8Result out, int clusters, cudaStream_t stream) {
#define TTC_F8(O) (p.b_shift == 0 ? launch<O, true>(p, clusters, stream) : launch<O, false>(p, clusters, stream))
  switch (out) {
    case kF8ResultF16: return TTC_F8(kF8ResultF16);
    case kF8ResultBF16: return TTC_F8(kF8ResultBF16);
    case kF8ResultF32: return TTC_F8(kF8ResultF32);
  }
#undef TTC_F8
  return cudaErrorInvalidValue;
}

}  // namespace ttc
