// Grouped products on CTA pairs: 256 x 256 tiles by tcgen05.mma.cta_group::2,
// operands by TMA, both directions.
//
//   forward   rows of D: 256 of one group's tokens; reduction: K
//   wgrad     rows of D: 256 of A's columns; reduction: the group's tokens, so
//             both operands lie with the reduction outermost ("MN-major")
//
// The pipeline is gemm_pair_kernel's: each CTA stages its 128 rows of A and 128
// columns of B, three stages of two 64-deep k-blocks, two accumulators in
// tensor memory, eight epilogue warps.  What ragged groups add:
//
// * A tile's rows start at the group's first row wherever that is, which TMA
//   allows (only the contiguous coordinate has an alignment).  The box of the
//   last tile reaches into the next group's rows; they fill accumulator rows
//   that are not stored.  A warp whose 32 rows all belong to the group stores
//   them with TMA, the others row by row.  A half tile with no row in the group
//   loads no A.
// * In wgrad the next group's rows would be added to the sums.  The last
//   k-block therefore issues MMAs for ceil(rows / 16) steps of 16 only, and where
//   the group ends inside a step the rows behind it are set to zero in shared
//   memory, in both operands (a NaN times zero would still be one).  A warp of
//   its own does that in each CTA: the stage's loads complete on a barrier of
//   its CTA, it waits there, writes the zeros, and then arrives on the even
//   CTA's `full` barrier, as the producers do for every other stage.  The
//   producer goes on with the next tile meanwhile.
// * fp32 results (wgrad): the tensor cores cut, not round, each addition to the
//   accumulator, an error that grows with the number of tokens (measured 4.5e-6
//   of the result after 2000 to 5600 tokens).  Every kChunkKBlocks k-blocks a fresh
//   accumulator is started and the epilogue warps add up the partial sums in
//   registers, rounded to nearest.
#include <atomic>

#include "gemm2sm_kernel.cuh"
#include "grouped_common.cuh"

namespace ttc {

namespace {

constexpr int kTile = kGroupedPairTile;
constexpr int kKPS = 2;  // k-blocks of a stage
constexpr int kStages = 3;
constexpr int kHalfBytes = 128 * kBK * 2;             // a CTA's share of one operand's k-block
constexpr int kKBlockBytes = 2 * kHalfBytes;          // of both
constexpr int kEpiWarps8 = 8;
constexpr int kStagingBytes = kEpiWarps8 * 4096;      // 2 x 2 KB a warp (16-bit), or 4 KB (fp32)
constexpr int kBarBytes = 256;
constexpr int kSmemBytes = 1024 + kStages * kKPS * kKBlockBytes + kStagingBytes + kBarBytes + kPairTableBytes;
constexpr int kChunkKBlocks = 8;                      // fp32 results: 512 tokens to an accumulator
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert(kChunkKBlocks % kKPS == 0, "accumulator chunks hold whole stages");

// threads: producer, MMA issuer, eight epilogue warps, and in wgrad the warp
// that clears the rows behind a group's end
template <bool WGRAD>
constexpr int kThreadsOf = 32 * (2 + kEpiWarps8 + (WGRAD ? 1 : 0));

struct PairLoop {
  int k_blocks;  // of the tile
  int fix_rows;  // wgrad: rows of the last k-block inside the group where that is no multiple of 16, else 0
  int last_steps;  // steps of 16 in the last k-block
};

template <bool WGRAD>
__device__ __forceinline__ PairLoop pair_loop(const GroupedParams& p, const GroupedTile& x) {
  PairLoop l;
  if constexpr (WGRAD) {
    const int rows = x.hi - x.lo;
    l.k_blocks = (rows + kBK - 1) / kBK;
    const int last = rows - (l.k_blocks - 1) * kBK;
    l.last_steps = (last + kUmmaK - 1) / kUmmaK;
    l.fix_rows = rows > 0 && last % kUmmaK != 0 ? last : 0;
  } else {
    l.k_blocks = p.k_blocks;
    l.last_steps = kBK / kUmmaK;
    l.fix_rows = 0;
  }
  return l;
}

// `boxes` boxes of one operand's share of a k-block: one 64 x 128 box with K
// contiguous, or two 64 x 64 ones of 64 contiguous rows (columns) each.
template <bool PAIR>
__device__ __forceinline__ void load_share(uint8_t* dst, const CUtensorMap* m, bool mn, int r0, int k0, int z,
                                           uint64_t* bar, uint32_t bar_leader, uint64_t pol) {
  const int x = mn ? r0 : k0, y = mn ? k0 : r0;
  if constexpr (PAIR) {
    tma_load_3d_pair(dst, m, x, y, z, bar_leader, pol);
    if (mn) tma_load_3d_pair(dst + kHalfBytes / 2, m, x + 64, y, z, bar_leader, pol);
  } else {
    tma_load_3d(dst, m, x, y, z, bar, pol);
    if (mn) tma_load_3d(dst + kHalfBytes / 2, m, x + 64, y, z, bar, pol);
  }
}

// Stores 32 columns of the warp's 32 rows through the staging buffer by TMA.
template <bool BF16, bool F32>
__device__ __forceinline__ void store_block_tma(const GroupedParams& p, const float (&v)[32], uint8_t* sb, int col0,
                                                int row0, int z, int lane) {
  if constexpr (F32) {
    constexpr layout::SwizzleBytes128 swz{};
#pragma unroll
    for (int ch = 0; ch < 8; ++ch)
      *reinterpret_cast<float4*>(sb + swz((uint32_t)(lane * 128 + ch * 16))) =
          make_float4(v[4 * ch], v[4 * ch + 1], v[4 * ch + 2], v[4 * ch + 3]);
  } else {
    constexpr layout::SwizzleBytes64 swz{};
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
      *reinterpret_cast<uint4*>(sb + swz((uint32_t)(lane * 64 + ch * 16))) =
          make_uint4(pack2<BF16>(v[8 * ch], v[8 * ch + 1]), pack2<BF16>(v[8 * ch + 2], v[8 * ch + 3]),
                     pack2<BF16>(v[8 * ch + 4], v[8 * ch + 5]), pack2<BF16>(v[8 * ch + 6], v[8 * ch + 7]));
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(&p.tmD, col0, row0, z, sb);
    bulk_commit();
  }
}

template <bool BF16, bool WGRAD, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsOf<WGRAD>, 1)
    grouped_pair_kernel(const __grid_constant__ GroupedParams p) {
  static_assert(WGRAD || !F32, "forward results are 16-bit");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;  // [stage][k-block of the stage]
  uint8_t* sB = sA + kStages * kKPS * kHalfBytes;
  uint8_t* staging = sB + kStages * kKPS * kHalfBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStagingBytes);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* fix = bars + 2 * kStages;  // wgrad: a stage's loads by this CTA, where its last rows are to be cleared
  uint64_t* tmem_full = bars + 3 * kStages;
  uint64_t* tmem_empty = bars + 3 * kStages + 2;
  uint64_t* stall_bar = bars + 3 * kStages + 4;
  uint64_t* drain_bar = bars + 3 * kStages + 5;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kStages + 6);
  int* table = reinterpret_cast<int*>(p.table == kTableInStaging ? staging + kStagingBytes / 2
                                                                 : reinterpret_cast<uint8_t*>(bars) + kBarBytes);
  int* offs = p.table == kTableGlobal ? nullptr : table;
  int* start = WGRAD ? nullptr : table + p.groups + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
  const WaitCtx wc{p.err, p.timeout_ns};

  if (warp == 0) {
    if (lane < kStages) {
      mbar_init(&full[lane], WGRAD ? 2 : 1);  // wgrad: both CTAs arrive, the producers or the clearing warps
      mbar_init(&empty[lane], 1);
      mbar_init(&fix[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&tmem_full[lane], 1);
      mbar_init(&tmem_empty[lane], 2 * kEpiWarps8);
    }
    if (lane == 0) {
      mbar_init(stall_bar, 1);
      mbar_init(drain_bar, 1);
      prefetch_tmap(&p.tmA);
      prefetch_tmap(&p.tmB);
      if (p.d_tma) prefetch_tmap(&p.tmD);
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
  if (offs != nullptr) build_group_table<kTile>(p, offs, start);
  const int tiles = WGRAD ? p.groups * p.row_blocks * p.col_blocks : start[p.groups];

  if (warp == 0) {
    // ---------------------------------------------------------------- producer (both CTAs)
    if (lane == 0) {
      const uint64_t keep = policy_evict_last();
      const uint64_t pol_b = !WGRAD && p.b_stream ? policy_evict_first() : keep;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0, armed_parity = 0;          // stages armed on `full` (even CTA)
      uint32_t fixed = 0, fix_parity = 0, fix_phase = 0;  // stages armed on `fix`
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += num_pairs) {
        const GroupedTile x = grouped_tile<kTile, WGRAD>(p, offs, start, t);
        const PairLoop l = pair_loop<WGRAD>(p, x);
        const int n0 = x.cb * kTile + (int)rank * 128;
        const int m0 = (WGRAD ? 0 : x.lo) + x.rb * kTile + (int)rank * 128;
        // forward: whether this CTA's, and the other's, rows of A hold any of the group
        const bool a_on = WGRAD || m0 < x.hi;
        const int halves = WGRAD || x.lo + x.rb * kTile + 128 < x.hi ? 2 : 1;
        const int zb = WGRAD ? 0 : (p.strideB != 0 ? x.g : 0);
        for (int kb0 = 0; kb0 < l.k_blocks; kb0 += kKPS) {
          const int nkb = min(kKPS, l.k_blocks - kb0);
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          const bool clear = WGRAD && l.fix_rows != 0 && kb0 + nkb == l.k_blocks;
          const uint32_t full_leader = mapa_shared(smem_u32(&full[stage]), 0);
          if (clear) {
            mbar_arrive_expect_tx(&fix[stage], nkb * kKBlockBytes);
            fixed |= 1u << stage;
            fix_parity = (fix_parity & ~(1u << stage)) | (fix_phase & (1u << stage));
            fix_phase ^= 1u << stage;
          } else if (leader) {
            mbar_arrive_expect_tx(&full[stage], nkb * (halves + 2) * kHalfBytes);
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          } else if (WGRAD) {
            mbar_arrive_cluster_relaxed(full_leader);
          }
          for (int j = 0; j < nkb; ++j) {
            uint8_t* a = sA + (stage * kKPS + j) * kHalfBytes;
            uint8_t* b = sB + (stage * kKPS + j) * kHalfBytes;
            const int k0 = (WGRAD ? x.lo : 0) + (kb0 + j) * kBK;
            if (clear) {
              load_share<false>(a, &p.tmA, WGRAD, m0, k0, 0, &fix[stage], 0, keep);
              load_share<false>(b, &p.tmB, WGRAD || p.b_mn, n0, k0, zb, &fix[stage], 0, pol_b);
            } else {
              if (a_on) load_share<true>(a, &p.tmA, WGRAD, m0, k0, 0, nullptr, full_leader, keep);
              load_share<true>(b, &p.tmB, WGRAD || p.b_mn, n0, k0, zb, nullptr, full_leader, pol_b);
            }
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        // loads in flight land before the pair may exit
        for (int s = 0; s < kStages; ++s) {
          if (leader && (armed & (1u << s))) drain_wait(&full[s], (armed_parity >> s) & 1u, 100000000ull);
          if (fixed & (1u << s)) drain_wait(&fix[s], (fix_parity >> s) & 1u, 100000000ull);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (even CTA)
    if (leader && lane == 0) {
      const bool b_mn = WGRAD || p.b_mn != 0;
      const uint32_t idesc = idesc_f16(BF16, WGRAD, b_mn, kTile, kTile);
      const uint64_t a0 = smem_desc_sw128(smem_u32(sA), WGRAD ? 8192u : 16u, 1024);
      const uint64_t b0 = smem_desc_sw128(smem_u32(sB), b_mn ? 8192u : 16u, 1024);
      const uint64_t a_step = WGRAD ? 2048u >> 4 : 32u >> 4, b_step = b_mn ? 2048u >> 4 : 32u >> 4;
      bool ok = true, any = false;
      if (p.inject_stall) ok = mbar_wait(stall_bar, 0, wc);  // nothing arrives here
      int stage = 0, it = 0;
      uint32_t phase = 0;
      for (int t = pair; ok && t < tiles; t += num_pairs) {
        const GroupedTile x = grouped_tile<kTile, WGRAD>(p, offs, start, t);
        const PairLoop l = pair_loop<WGRAD>(p, x);
        const int chunk = F32 ? kChunkKBlocks : l.k_blocks;
        int kbeg = 0;
        do {  // once, too, for a tile without k-blocks
          const int kend = min(l.k_blocks, kbeg + chunk);
          const int acc = it & 1;
          if (!mbar_wait_cluster(&tmem_empty[acc], ((it >> 1) & 1) ^ 1u, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * kTile;
          for (int kb0 = kbeg; kb0 < kend; kb0 += kKPS) {
            const int nkb = min(kKPS, kend - kb0);
            // zeros written by the other CTA's threads are behind this barrier in wgrad
            if (!(WGRAD ? mbar_wait_cluster(&full[stage], phase, wc) : mbar_wait(&full[stage], phase, wc))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < kKPS; ++j) {
              if (j < nkb) {
                const uint64_t ad = a0 + (uint32_t)(stage * kKPS + j) * (kHalfBytes >> 4);
                const uint64_t bd = b0 + (uint32_t)(stage * kKPS + j) * (kHalfBytes >> 4);
                const int steps = WGRAD && kb0 + j == l.k_blocks - 1 ? l.last_steps : kBK / kUmmaK;
                mma_f16_pair(d_tmem, ad, bd, idesc, kb0 + j != kbeg);
#pragma unroll
                for (int k = 1; k < kBK / kUmmaK; ++k)
                  if (!WGRAD || k < steps) mma_f16_pair(d_tmem, ad + k * a_step, bd + k * b_step, idesc, 1u);
              }
            }
            any = true;
            mma_commit_pair(&empty[stage], 0x3);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (kend == kbeg) {
            mbar_arrive(&tmem_full[acc]);
            mbar_arrive_cluster(mapa_shared(smem_u32(&tmem_full[acc]), 1));
          } else {
            mma_commit_pair(&tmem_full[acc], 0x3);
          }
          ++it;
          kbeg = kend;
        } while (kbeg < l.k_blocks);
      }
      if (any) {
        // every MMA must have finished with both CTAs' TMEM before it is freed
        mma_commit_pair(drain_bar, 0x1);
        drain_wait(drain_bar, 0, 100000000ull);
      }
    }
  } else if (warp < 2 + kEpiWarps8) {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int ew = warp - 2, q = warp & 3, part = ew >> 2;
    constexpr int esize = F32 ? 4 : 2;
    constexpr int kChunks = kTile / 64;  // 32-column chunks of this warp: one half of the tile's columns
    uint8_t* sbuf = staging + ew * (F32 ? 4096 : 2048);
    const bool two_bufs = !F32 && p.table != kTableInStaging;
    const int gran = 16 / esize;
    int buf = 0, it = 0;
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += num_pairs) {
      const GroupedTile x = grouped_tile<kTile, WGRAD>(p, offs, start, t);
      const PairLoop l = pair_loop<WGRAD>(p, x);
      const int r0 = x.rb * kTile + (int)rank * 128 + q * 32;  // the warp's first row, of the group in forward
      const int64_t row0 = WGRAD ? r0 : (int64_t)x.lo + r0;
      const int64_t row = row0 + lane;
      const bool row_ok = WGRAD ? row < p.K : row < x.hi;
      const int z = WGRAD ? x.g : 0;
      const int colp = x.cb * kTile + part * (kTile / 2);
      char* d_row = static_cast<char*>(p.D) + ((int64_t)z * p.strideD + row * p.ldd) * esize;
      const char* c_row = p.C != nullptr && row_ok
                              ? static_cast<const char*>(p.C) + ((int64_t)z * p.strideC + row * p.ldc) * esize
                              : nullptr;
      const float* bias = p.bias != nullptr ? p.bias + (int64_t)x.g * p.stride_bias : nullptr;
      if (c_row != nullptr && p.c_vec && colp < p.N) {
        // this row's part of C toward L2 while the sums are made
        const int n = min(kTile / 2, p.N - colp) * esize & ~15;
        if (n > 0) prefetch_l2_bulk(c_row + (int64_t)colp * esize, (uint32_t)n);
      }
      auto finish = [&](const uint32_t(&w)[32], int c) {
        const int col0 = colp + c * 32;
        const int n = min(32, p.N - col0);
        float v[32];
        grouped_values<BF16>(p, w, c_row != nullptr && n > 0 ? c_row + (int64_t)col0 * esize : nullptr,
                             bias != nullptr && n > 0 ? bias + col0 : nullptr, n, v);
        // a TMA store ends at whole 16-byte granules of a row: a chunk that
        // holds fewer is stored by its threads
        const bool by_tma = p.d_tma && n > 0 && n % gran == 0 && (WGRAD ? row0 < p.K : row0 + 32 <= x.hi);
        if (by_tma) {
          if (lane == 0) {
            if (two_bufs)
              bulk_wait_read<1>();
            else
              bulk_wait_read<0>();
          }
          __syncwarp();
          store_block_tma<BF16, F32>(p, v, sbuf + (two_bufs ? buf * (kStagingBytes / 2) : 0), col0, (int)row0, z, lane);
          buf ^= 1;
        } else if (row_ok && n > 0) {
          store_row<BF16>(p, v, d_row + (int64_t)col0 * esize, n);
        }
      };
      if constexpr (F32) {
        uint32_t sums[kChunks][32];  // floats
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) sums[c][j] = 0u;
        int kbeg = 0;
        do {
          const int acc = it & 1;
          if (!mbar_wait(&tmem_full[acc], (it >> 1) & 1, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (l.k_blocks > 0) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              uint32_t w[32];
              tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(q * 32) << 16) + acc * kTile + part * (kTile / 2) + c * 32, w);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j)
                sums[c][j] = __float_as_uint(__uint_as_float(sums[c][j]) + __uint_as_float(w[j]));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
          ++it;
          kbeg += kChunkKBlocks;
        } while (kbeg < l.k_blocks);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) finish(sums[c], c);
      } else {
        const int acc = it & 1;
        if (!mbar_wait(&tmem_full[acc], (it >> 1) & 1, wc)) break;
        ++it;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          uint32_t w[32];
          if (l.k_blocks > 0) {
            tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(q * 32) << 16) + acc * kTile + part * (kTile / 2) + c * 32, w);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = 0u;
          }
          if (c == kChunks - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
          }
          finish(w, c);
        }
      }
    }
    if (p.d_tma && lane == 0) bulk_wait_all();
  } else {
    // ---------------------------------------------------------------- wgrad: rows behind a group's end (both CTAs)
    int stage = 0;
    uint32_t fix_phase = 0;
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += num_pairs) {
      const GroupedTile x = grouped_tile<kTile, WGRAD>(p, offs, start, t);
      const PairLoop l = pair_loop<WGRAD>(p, x);
      const int stages = (l.k_blocks + kKPS - 1) / kKPS;
      if (l.fix_rows != 0) {
        const int s = (stage + stages - 1) % kStages;
        if (!mbar_wait(&fix[s], (fix_phase >> s) & 1u, wc)) {
          ok = false;
          break;
        }
        fix_phase ^= 1u << s;
        const int j = (l.k_blocks - 1) % kKPS;  // the last k-block's place in its stage
        const int r_end = (l.fix_rows + kUmmaK - 1) / kUmmaK * kUmmaK;
        const int n16 = (r_end - l.fix_rows) * 8;  // 16-byte pieces of a 64-wide slab's rows
        uint8_t* ops[2] = {sA + (s * kKPS + j) * kHalfBytes, sB + (s * kKPS + j) * kHalfBytes};
#pragma unroll
        for (int o = 0; o < 2; ++o)
          for (int i = lane; i < 2 * n16; i += 32) {
            const int slab = i >= n16 ? 1 : 0;
            *reinterpret_cast<uint4*>(ops[o] + slab * (kHalfBytes / 2) + l.fix_rows * 128 + (i - slab * n16) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&full[s]), 0));
      }
      stage = (stage + stages) % kStages;
    }
  }

  __syncthreads();
  cluster_sync();  // the pair's MMAs, remote arrivals and loads are all finished
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <bool BF16, bool WGRAD, bool F32>
cudaError_t prepare() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(grouped_pair_kernel<BF16, WGRAD, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  return cudaSuccess;
}

template <bool BF16, bool WGRAD, bool F32>
int clusters_of() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load();
  if (n > 0) return n;
  if (prepare<BF16, WGRAD, F32>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreadsOf<WGRAD>, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaOccupancyMaxActiveClusters(&n, grouped_pair_kernel<BF16, WGRAD, F32>, &cfg) != cudaSuccess) return 0;
  known[dev].store(n);
  return n;
}

template <bool BF16, bool WGRAD, bool F32>
cudaError_t launch(const GroupedParams& p, int clusters, cudaStream_t stream) {
  cudaError_t e = prepare<BF16, WGRAD, F32>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreadsOf<WGRAD>, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, grouped_pair_kernel<BF16, WGRAD, F32>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Pairs that can be resident at once (0 on error).
int grouped_pair_clusters(bool bf16, bool wgrad, bool f32) {
  if (!wgrad) return bf16 ? clusters_of<true, false, false>() : clusters_of<false, false, false>();
  if (f32) return bf16 ? clusters_of<true, true, true>() : clusters_of<false, true, true>();
  return bf16 ? clusters_of<true, true, false>() : clusters_of<false, true, false>();
}

cudaError_t launch_grouped_pair(bool bf16, bool wgrad, const GroupedParams& p, int clusters, cudaStream_t stream) {
  if (!wgrad) return bf16 ? launch<true, false, false>(p, clusters, stream) : launch<false, false, false>(p, clusters, stream);
  if (p.out_f32) return bf16 ? launch<true, true, true>(p, clusters, stream) : launch<false, true, true>(p, clusters, stream);
  return bf16 ? launch<true, true, false>(p, clusters, stream) : launch<false, true, false>(p, clusters, stream);
}

}  // namespace ttc
