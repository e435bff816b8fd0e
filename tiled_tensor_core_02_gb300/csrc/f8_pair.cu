// Block-scaled fp8 products on CTA pairs: 256 x 256 tiles by tcgen05.mma.cta_group::2
// (kind::f8f6f4), operands by TMA.
//
// The scales change with every 128 of K, so the tensor cores add up one such block at
// a time: each goes into one of two accumulators in tensor memory, and sixteen epilogue warps
// add it, scaled, to the tile's sums in their registers (a thread has one row and 64 columns,
// read 16 at a time) while the tensor cores fill the other.  What has to be short is the way
// from an accumulator's last MMA to its being free again, two crossings between SMs and the
// reads: 8192 x 14336 x 4096 takes 441 us, 401 without the results' way out, 255 by the MMAs
// alone.  Eight warps of 128 columns, which read twice as long, took 751; four accumulators of
// 128 columns 464, where an MMA of half the width costs more than half (313 us alone); loads of
// 32 columns a fifth more, of 8 a twentieth.
//
// Two warps bring the scales of four blocks of K at a time into shared memory: A's by row, B's
// one for 128 columns or one a column, and where the tile lies.  In the epilogue's own hands
// they took registers that the sums need, and what is spilled goes to L2, nearly all of L1
// being shared memory here.  For the same reason the four warps that load and issue hand
// registers over.  The MMAs are issued by a converged warp: by one thread of it, which moves
// descriptors to uniform registers each time, four of them took 0.38 us instead of 0.22.  One
// commit after a block's MMAs says both that its accumulator is full and that its operands' place
// is free (two, and loads by a single thread: 447 us).
//
// Bound by the epilogue: 0.52 us a block of K and tile, and at a tile's end 1.9 us, with GELU
// 3.7 (its exponentials and quotients), during which the tensor cores get two blocks ahead.
// 8192 x 14336 x 4096: 2.18 PFLOP/s, with GELU 2.01; by columns, fp32 sums added to,
// 4096 x 4096 x 8192 203 us.
#include <atomic>
#include <type_traits>

#include "f8_blocks.cuh"
#include "grouped_common.cuh"

namespace ttc {

namespace {

constexpr int kTile = kGroupedPairTile;
constexpr int kShareBytes = 128 * kF8Block;  // a CTA's share of one operand's block
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarpCount = 16;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarpCount);
constexpr int kLoaders = 64;  // threads that load scales: warps 2 and 3
constexpr int kStagingBytes = kEpiWarpCount * 4096;
constexpr int kBarBytes = 256;
constexpr int kTableInts = 384;
constexpr int kStages = 4;
// Scales of a chunk of K: A's of 128 rows, four each, then B's.
constexpr int kAhead = 4;       // blocks of K of a chunk
constexpr int kScaleSlots = 2;  // chunks on their way
constexpr int kScaleBytes = 128 * kAhead * 4 + kTile * kAhead * 4 + 32;
constexpr int kSmemBytes =
    1024 + kStages * 2 * kShareBytes + kStagingBytes + kScaleSlots * kScaleBytes + kBarBytes + kTableInts * 4;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert((kMaxGroups + 3) / 4 + 1 <= kTableInts, "a table of every fourth group's tiles has room");
// Registers a thread: at launch, of the first four warps, of the epilogue's.
constexpr int kRegsLaunch = 96, kRegsFew = 64, kRegsMany = 104;
static_assert(128 * kRegsFew + (kThreads - 128) * kRegsMany <= kThreads * kRegsLaunch, "the shares fit the launch's registers");
constexpr int kLoad = 16;  // columns a load
constexpr int kAccs = 2, kAccCols = kTile;  // accumulators; columns of each

// What the loaders of scales tell the epilogue about a chunk's tile.
struct TileInfo {
  int parts;            // 2, of half a tile 1
  int g, col0;          // group; first column of D
  int row0, row_end;    // first row of the CTA, the group's last
};

// Four scales in a row of which `n` exist (zeros behind them); volatile, so that they are
// asked for here and not where they are used.
__device__ __forceinline__ float4 four_scales(const float* p, bool vec, int n) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (vec && n >= 4) {
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  } else {
    if (n > 0) asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v.x) : "l"(p));
    if (n > 1) asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v.y) : "l"(p + 1));
    if (n > 2) asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v.z) : "l"(p + 2));
    if (n > 3) asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v.w) : "l"(p + 3));
  }
  return v;
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


// Shared memory by its 32-bit address.
__device__ __forceinline__ uint32_t shared_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ float shared_f32(uint32_t at) { return __uint_as_float(shared_u32(at)); }
__device__ __forceinline__ float4 shared_f32x4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void arrive_at(uint32_t at) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(at) : "memory");
}
__device__ __forceinline__ bool try_wait_at(uint32_t at, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(at), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait_warp.
__device__ __forceinline__ bool wait_warp_at(uint32_t at, uint32_t parity, const WaitCtx& w) {
  bool ok = try_wait_at(at, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t spins = 1;; ++spins) {
      if (try_wait_at(at, parity)) {
        ok = true;
        break;
      }
      if ((spins & 63u) != 0u) continue;
      if (error_raised(w)) break;
      if (globaltimer_ns() - t0 > w.timeout_ns) {
        record_error(w, kDevTimeout);
        break;
      }
    }
  }
  return __all_sync(0xFFFFFFFFu, ok) != 0;
}

// Two columns at a time: half the instructions, though no faster in the FMA pipe.
__device__ __forceinline__ void add_pair(float* sum, const uint32_t* w, float2 scale) {
  const float2 v = __ffma2_rn(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), scale, make_float2(sum[0], sum[1]));
  sum[0] = v.x;
  sum[1] = v.y;
}

// OUT: F8Result; BY_COLUMN: B has a scale for each row (a column of D).
template <int OUT, bool BY_COLUMN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) f8_pair_kernel(const __grid_constant__ F8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + kStages * kShareBytes;
  uint8_t* staging = sB + kStages * kShareBytes;
  uint8_t* scales = staging + kStagingBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(scales + kScaleSlots * kScaleBytes);
  uint64_t* full = bars;
  uint64_t* done = bars + kStages;  // a stage's MMAs: its accumulator is full and its place free
  uint64_t* tmem_empty = done + kStages;
  uint64_t* scale_full = tmem_empty + kAccs;
  uint64_t* scale_empty = scale_full + kScaleSlots;
  uint64_t* stall_bar = scale_empty + kScaleSlots;
  uint64_t* drain_bar = stall_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  // what the producer tells the MMA issuer about a stage: 2, of half a tile 1
  int* stage_info = reinterpret_cast<int*>(drain_bar + 2);

  static_assert((2 * kStages + 2 * kAccs + 2 * kScaleSlots + 3) * 8 + kStages * 4 <= kBarBytes, "barrier area");
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
      mbar_init(&done[lane], 1);
    }
    if (lane < kAccs) {
      mbar_init(&tmem_empty[lane], 2 * kEpiWarpCount);
    }
    if (lane < kScaleSlots) {
      mbar_init(&scale_full[lane], kLoaders);
      mbar_init(&scale_empty[lane], kEpiWarpCount);
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
  grid_dependency_wait();
  grid_dependents_launch();
  build_group_table<kTile>(p, tb);
  // Each role finds the walk and the accumulators for itself: what is live where the roles
  // part is spilled in the one that is short of registers.
  const auto find_walk = [&] { return pair_walk(table_tiles(p, tb), num_pairs); };
  const auto find_tmem = [&] { return *const_cast<volatile uint32_t*>(tmem_slot); };

  if (warp < kEpiWarp0) {
    registers_down<kRegsFew>();
    if (warp == 0) {
      // ---------------------------------------------------------------- producer (both CTAs)
      const uint32_t lead = elect_lead();  // a converged warp, one lane of which loads
      const PairWalk walk = find_walk();
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
          if (!mbar_wait_warp(&done[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          const uint32_t full_leader = mapa_shared(smem_u32(&full[stage]), 0);
          if (leader) {
            if (lead) {
              stage_info[stage] = item.half < 0 ? 2 : 1;
              mbar_arrive_expect_tx(full + stage, shares * kShareBytes);
            }
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          }
          if (a_on) tma_load_3d_pair_lead(lead, sA + stage * kShareBytes, &p.tmA, kb * kF8Block, m0, 0, full_leader, keep);
          tma_load_3d_pair_lead(lead, sB + stage * kShareBytes, &p.tmB, kb * kF8Block, n0, zb, full_leader, pol_b);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // a stage completes once both CTAs' loads for it have landed
      if (leader)
        drain_ring_lanes(full, armed, armed_parity);
      else
        drain_odd_cta(wc);
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer (even CTA)
      if (leader) {
        const uint32_t lead = elect_lead(), tmem_base = find_tmem();
        const PairWalk walk = find_walk();
        const uint32_t idesc_whole = idesc_f8(p.a_e5m2 != 0, p.b_e5m2 != 0, kTile, kTile);
        const uint32_t idesc_half = idesc_f8(p.a_e5m2 != 0, p.b_e5m2 != 0, kTile, kTile / 2);
        const uint64_t a0 = smem_desc_sw128(smem_u32(sA), 16u, 1024);
        const uint64_t b0 = smem_desc_sw128(smem_u32(sB), 16u, 1024);
        const uint32_t a_hi = (uint32_t)(a0 >> 32), b_hi = (uint32_t)(b0 >> 32);
        bool ok = true, any = false;
        if (p.inject_stall) ok = mbar_wait_warp(stall_bar, 0, wc);  // nothing arrives here
        int stage = 0;
        uint32_t it = 0, phase = 0;
        for (int t = pair; ok && t < walk.items; t += num_pairs) {
          for (int kb = 0; ok && kb < p.k_blocks; ++kb) {
            if (!mbar_wait_warp(&full[stage], phase, wc)) {
              ok = false;
              break;
            }
            const uint32_t idesc = stage_info[stage] == 2 ? idesc_whole : idesc_half;
            const uint32_t a_lo = (uint32_t)a0 + (uint32_t)stage * (kShareBytes >> 4);
            const uint32_t b_lo = (uint32_t)b0 + (uint32_t)stage * (kShareBytes >> 4);
            const uint32_t acc = it & (kAccs - 1);
            // the first use of each accumulator passes at once
            if (!mbar_wait_warp(&tmem_empty[acc], ((it / kAccs) & 1) ^ 1u, wc)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kF8Block / 32; ++k)
              mma_f8_pair_lead(lead, tmem_base + acc * kAccCols, a_lo + k * 2, a_hi, b_lo + k * 2, b_hi, idesc, k != 0);
            any = true;
            ++it;
            mma_commit_pair_lead(lead, &done[stage], 0x3);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (any) {
          // every MMA must have finished with both CTAs' TMEM before it is freed
          mma_commit_pair_lead(lead, drain_bar, 0x1);
          drain_wait(drain_bar, 0, 100000000ull);
        }
      }
    } else {
      // ---------------------------------------------------------------- scales (both CTAs)
      const PairWalk walk = find_walk();
      const int i0 = threadIdx.x - 64;
      uint32_t chunk = 0;
      bool ok = true;
      for (int t = pair; ok && t < walk.items; t += num_pairs) {
        const PairItem item = pair_item<false>(p, tb, walk, t);
        const GroupedTile& x = item.x;
        const int row0 = x.lo + x.rb * kTile + (int)rank * 128;
        const int col0 = x.cb * kTile + max(item.half, 0) * (kTile / 2);
        const int width = item.half < 0 ? kTile : kTile / 2;
        const float* sb = p.scale_b + (int64_t)x.g * p.stride_sb;
        for (int kb0 = 0; kb0 < p.k_blocks; kb0 += kAhead, ++chunk) {
          const int slot = chunk % kScaleSlots, n = p.k_blocks - kb0;
          if (!mbar_wait(&scale_empty[slot], (chunk / kScaleSlots & 1) ^ 1u, wc)) {
            ok = false;
            break;
          }
          float4* a_out = reinterpret_cast<float4*>(scales + slot * kScaleBytes);
          float* b_out = reinterpret_cast<float*>(a_out + 128);
          float4 a[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = row0 + i * kLoaders + i0;
            a[i] = four_scales(p.scale_a + (int64_t)row * p.lds_a + kb0, p.sa_vec != 0, row < x.hi ? n : 0);
          }
          if constexpr (BY_COLUMN) {  // [block][column]
            float4 v[kTile / kLoaders];
#pragma unroll
            for (int i = 0; i < kTile / kLoaders; ++i) {
              const int col = col0 + i * kLoaders + i0;
              v[i] = four_scales(sb + (int64_t)col * p.lds_b + kb0, p.sb_vec != 0,
                                 col < p.N && i * kLoaders < width ? n : 0);
            }
#pragma unroll
            for (int i = 0; i < kTile / kLoaders; ++i) {
              float* o = b_out + i * kLoaders + i0;
              o[0] = v[i].x;
              o[kTile] = v[i].y;
              o[2 * kTile] = v[i].z;
              o[3 * kTile] = v[i].w;
            }
          } else if (i0 < 2) {  // one for either half's columns
            const int col = col0 + i0 * (width / 2);
            reinterpret_cast<float4*>(b_out)[i0] =
                four_scales(sb + (int64_t)(col >> 7) * p.lds_b + kb0, p.sb_vec != 0, col < p.N ? n : 0);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) a_out[i * kLoaders + i0] = a[i];
          if (i0 == 0) *reinterpret_cast<TileInfo*>(b_out + kTile * kAhead) = TileInfo{width / 128, x.g, col0, row0, x.hi};
          mbar_arrive(&scale_full[slot]);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    registers_up<kRegsMany>();
    using T = typename std::conditional<OUT == kF8ResultF32, float, uint16_t>::type;
    constexpr int kUnit = 128 / (int)sizeof(T);  // columns that 128 bytes hold
    constexpr int kElems = 16 / (int)sizeof(T);
    // quarter of the rows; which CTA's weights the columns are of, and which half of those (of
    // half a tile they have 64 columns, and the second warps nothing)
    const int ew = warp - kEpiWarp0, q = warp & 3, half = (ew >> 2) & 1, second = ew >> 3;
    const PairWalk walk = find_walk();
    const uint32_t from = find_tmem() + ((uint32_t)(q * 32) << 16) ;
    // shared memory by 32-bit addresses: the accumulators' barriers here and in the even CTA, this lane's scales
    const uint32_t full_at = smem_u32(done), release = mapa_shared(smem_u32(tmem_empty), 0);
    const uint32_t scales_at = smem_u32(scales);
    uint32_t it = 0;  // accumulators so far
    uint32_t chunk = 0;
    bool ok = true;
    for (int t = pair; ok && t < walk.items; t += num_pairs) {
      float sums[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) sums[j] = 0.0f;
      for (int kb0 = 0; ok && kb0 < p.k_blocks; kb0 += kAhead, ++chunk) {
        const uint32_t slot = chunk % kScaleSlots;
        if (!wait_warp_at(full_at + (kStages + kAccs + slot) * 8, chunk / kScaleSlots & 1, wc)) {
          ok = false;
          break;
        }
        uint32_t a_at = scales_at + slot * kScaleBytes, b_at = a_at + 128 * kAhead * 4;
        const uint32_t parts = shared_u32(b_at + kTile * kAhead * 4);
        a_at += (q * 32 + lane) * kAhead * 4;
        b_at += BY_COLUMN ? (half * (parts * 64) + second * 64) * 4 : half * kAhead * 4;
        const uint32_t at = from + (parts == 2 ? half * 128 + second * 64 : half * 64);
        const int blocks = min(kAhead, p.k_blocks - kb0);
#pragma unroll 1
        for (int i = 0; i < blocks; ++i, ++it, a_at += 4, b_at += BY_COLUMN ? kTile * 4 : 4) {
          float scale = shared_f32(a_at);
          if constexpr (!BY_COLUMN) scale *= shared_f32(b_at);
          const uint32_t acc = it & (kAccs - 1);
          if (!wait_warp_at(full_at + (it % kStages) * 8, (it / kStages) & 1, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 64 / kLoad; ++c) {
            uint32_t w[kLoad];
            tmem_ld_32x32b_x16<0>(at + acc * kAccCols + c * kLoad, w);
            tmem_ld_wait_for(w);
            if (c + 1 == 64 / kLoad) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster_relaxed(release + acc * 8);
            }
#pragma unroll
            for (int j = 0; j < kLoad; j += 4) {
              float2 f0 = make_float2(scale, scale), f1 = f0;
              if constexpr (BY_COLUMN) {
                const float4 v = shared_f32x4(b_at + (c * kLoad + j) * 4);
                f0 = __fmul2_rn(f0, make_float2(v.x, v.y));
                f1 = __fmul2_rn(f1, make_float2(v.z, v.w));
              }
              add_pair(sums + c * kLoad + j, w + j, f0);
              add_pair(sums + c * kLoad + j + 2, w + j + 2, f1);
            }
          }
        }
        if (kb0 + kAhead < p.k_blocks) {
          __syncwarp();
          if (lane == 0) arrive_at(full_at + (kStages + kAccs + kScaleSlots + slot) * 8);
        }
      }
      if (!ok) break;
      // where the tile lies, from its last chunk
      const uint32_t slot = (chunk - 1) % kScaleSlots;
      const TileInfo x = *reinterpret_cast<const TileInfo*>(scales + slot * kScaleBytes + 128 * kAhead * 4 + kTile * kAhead * 4);
      __syncwarp();
      if (lane == 0) arrive_at(full_at + (kStages + kAccs + kScaleSlots + slot) * 8);
      const int r0 = x.row0 + q * 32, rows = max(0, min(32, x.row_end - r0));
      const int col0 = x.col0 + (x.parts == 2 ? half * 128 + second * 64 : half * 64);
      const int cols = x.parts == 1 && second != 0 ? 0 : min(64, p.N - col0);
      uint8_t* sb = staging + ew * 4096;
      float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.bias != nullptr) bias = four_columns(p.bias + (int64_t)x.g * p.stride_bias + col0, lane, cols);
      T* d = static_cast<T*>(p.D) + (int64_t)r0 * p.ldd + col0;
      const T* c0 = static_cast<const T*>(p.C) + (int64_t)r0 * p.ldc + col0;
#pragma unroll
      for (int u = 0; u < 64 / kUnit; ++u) {
        if (cols <= u * kUnit || rows <= 0) continue;
        if (p.C != nullptr) {
          stage_c(p, c0 + u * kUnit, rows, cols - u * kUnit, lane, sb);
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kUnit / kElems; ++i) {
          uint4* piece = reinterpret_cast<uint4*>(sb + staged<32>(lane, i));
          float v[kElems];
#pragma unroll
          for (int k = 0; k < kElems; ++k) v[k] = sums[u * kUnit + i * kElems + k];
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
          if (p.act == kActGelu) {
#pragma unroll
            for (int k = 0; k < kElems; ++k) v[k] = act_value(kActGelu, v[k]);
          } else if (p.act == kActRelu) {
#pragma unroll
            for (int k = 0; k < kElems; ++k) v[k] = act_value(kActRelu, v[k]);
          }
          if constexpr (OUT == kF8ResultF32)
            *piece = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
          else
            *piece = make_uint4(pack2<OUT == kF8ResultBF16>(v[0], v[1]), pack2<OUT == kF8ResultBF16>(v[2], v[3]),
                                pack2<OUT == kF8ResultBF16>(v[4], v[5]), pack2<OUT == kF8ResultBF16>(v[6], v[7]));
        }
        __syncwarp();
        copy_out<T, 4>(p, sb, d + u * kUnit, rows, cols - u * kUnit, lane);
        __syncwarp();
      }
    }
  }

  __syncthreads();
  cluster_sync();  // the pair's MMAs, remote arrivals and loads are all finished
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(find_tmem(), 512);
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
