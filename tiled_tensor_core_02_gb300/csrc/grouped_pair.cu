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
//   that are not stored.  A half tile with no row in the group loads no A.
// * In wgrad the next group's rows would be added to the sums.  The last
//   k-block therefore issues MMAs for ceil(rows / 16) steps of 16 only, and where
//   the group ends inside a step the rows behind it are set to zero in shared
//   memory, in both operands (a NaN times zero would still be one).  A warp of
//   its own does that in each CTA: the stage's loads complete on a barrier of
//   its CTA, it waits there, writes the zeros, and then arrives on the even
//   CTA's `full` barrier, as the producers do for every other stage.  The
//   producer goes on with the next tile meanwhile.
// * fp32 results (wgrad): the tensor cores cut, not round, each addition to the
//   accumulator, an error that grows with the number of tokens (6.4e-6
//   of the result after 8192).  Every kChunkKBlocks k-blocks a fresh
//   accumulator is started and the epilogue warps add up the partial sums in
//   registers, rounded to nearest.
// * C (wgrad) comes while the tile's products do.  16-bit C is read before the
//   accumulator is waited for; fp32 C joins the partial sums 32 columns at a time
//   between the accumulators.  Read at the end, a block at a time, or all of it at
//   the tile's start, it met the next tile's operands on their way from L2, which
//   they fill, and held the tensor cores up: 8 x 4096 x 4096, 16384 tokens in equal
//   groups, 414 and 424 us against 381 in one burst of all (without C 335).
//
// int8 products with scales run here too, on fp16 copies of the operands (every
// int8 value is exact in fp16, every product and sum below 2^24 in fp32): one
// group, an accumulator for every 1024 of K, the partial sums added up as int32.
//
// Gated blocks (see gated_common.cuh) run here too.  Forward an accumulator holds both
// products of 128 columns side by side: the even CTA stages the gate's weights, the odd one the
// other projection's, which the pair's MMA reads as 256 columns.  In the gradient the
// epilogue reads the kept projections of its columns before it waits for the products.
// 8192 x 14336 x 4096 bf16: forward 1032 to 1130 us with both projections kept (1.70 to 1.86
// PFLOP/s, by the power cap), gradient 634 to 670 (20 us a tile for its products, 16 for its
// epilogue, which reads and writes 1.2 GB in all; K = 512 388 us, 3.1 TB/s).
//
// Where two halves of each of the last wave's tiles find a pair, the wave takes them
// as halves of 128 columns: half the MMA's time and half the epilogue (1120 rows of 7
// groups, 896 x 2944 20.7 -> 17.6 us; long walks at capped clocks gain nothing).  A gated
// forward tile's half saves half of the MMAs and stores; its epilogue reads and computes 64 columns
// a warp all the same, the second 32 of them for nothing.
//
// Results leave through a 4 KB block of shared memory per epilogue warp, 32 rows
// of 128 bytes: written a row per lane, read back and stored four whole rows an
// instruction, with no asynchronous copy to wait for and any row left out.
//
// An operand with its rows contiguous ("MN-major") comes as two boxes of 64
// rows by the stage's 128 k, so that a stage takes as few TMA instructions as
// one with K contiguous: with a box per k-block the issuing thread, at about 70 ns
// an instruction, set the pace.
//
// Bound by the tensor cores.  In bursts (replayed; the power cap, which holds longer
// runs to 1.5 to 1.6 GHz, adds a tenth): 16384 x 4096 x 4096 bf16 over 8 equal groups
// 305 us forward, 302 for the weights' gradient in bf16 (331 added to C) and 346 to 372
// in fp32 (399 to 415 added to C); int8 8192 x 14336 x 4096 568 us with its copies.
#include <atomic>
#include <type_traits>

#include "gated_common.cuh"
#include "gemm2sm_kernel.cuh"

namespace ttc {

namespace {

constexpr int kTile = kGroupedPairTile;
constexpr int kKPS = 2;  // k-blocks of a stage
constexpr int kStages = 3;
constexpr int kHalfBytes = 128 * kBK * 2;      // a CTA's share of one operand's k-block
constexpr int kShareBytes = kKPS * kHalfBytes;  // ... of its stage
constexpr int kEpiWarpCount = 8;
constexpr int kStagingBytes = kEpiWarpCount * 4096;
constexpr int kBarBytes = 256;
constexpr int kTableInts = 384;
constexpr int kSmemBytes = 1024 + kStages * 2 * kShareBytes + kStagingBytes + kBarBytes + kTableInts * 4;
// k-blocks of an accumulator where the partial sums are added up in registers:
// fp32 results, or int8, 1024 products
template <bool I8>
constexpr int kChunkKBlocks = I8 ? 16 : kSumKBlocks;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
static_assert(kChunkKBlocks<false> % kKPS == 0 && kChunkKBlocks<true> % kKPS == 0, "accumulator chunks hold whole stages");
static_assert((kMaxGroups + 3) / 4 + 1 <= kTableInts, "a table of every fourth group's tiles has room");

// Warps: producer, MMA issuer, in wgrad the one that clears the rows behind a
// group's end, a spare; then eight of the epilogue.
constexpr int kEpiWarp0 = 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarpCount);

// A stage's k-blocks (0 to 2), the steps of 16 in its last one where that is
// the tile's last, whether it is, and whether the tile is half a tile.
__device__ __forceinline__ int stage_word(int nkb, int last_steps, bool last, bool narrow) {
  return nkb | (last ? last_steps << 4 | 256 : (kBK / kUmmaK) << 4) | (narrow ? 512 : 0);
}

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

// A CTA's share of one operand's stage: with K contiguous a box of 64 k by 128
// rows for each of `nkb` k-blocks, else two boxes of 64 rows by 128 k.
__device__ __forceinline__ int share_bytes(bool mn, int nkb) { return mn ? kShareBytes : nkb * kHalfBytes; }

template <bool PAIR>
__device__ __forceinline__ void load_share(uint8_t* dst, const CUtensorMap* m, bool mn, int nkb, int r0, int k0, int z,
                                           uint64_t* bar, uint32_t bar_leader, uint64_t pol) {
  const int x0 = mn ? r0 : k0, y = mn ? k0 : r0;
  const int x1 = x0 + 64;
  if constexpr (PAIR) {
    tma_load_3d_pair(dst, m, x0, y, z, bar_leader, pol);
    if (mn || nkb > 1) tma_load_3d_pair(dst + kHalfBytes, m, x1, y, z, bar_leader, pol);
  } else {
    tma_load_3d(dst, m, x0, y, z, bar, pol);
    if (mn || nkb > 1) tma_load_3d(dst + kHalfBytes, m, x1, y, z, bar, pol);
  }
}

// A lane's row of the staging block; the block may be written again afterwards.
__device__ __forceinline__ void row_of_block(const uint8_t* sb, int lane, uint32_t (&w)[32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(sb + staged<32>(lane, i));
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
  __syncwarp();
}

// The reverse for C: N units of 32 rows by 128 bytes, all of them on their way
// before the first is used, then one after the other through the staging block to
// a row per lane.  Zeros outside `rows` and `n` columns.
template <int N, typename T>
__device__ __forceinline__ void load_c(const GroupedParams& p, const T* c0, int rows, int n, int lane, uint8_t* sb,
                                       uint32_t (&w)[N][32]) {
  constexpr int kElems = 16 / (int)sizeof(T), kCols = 128 / (int)sizeof(T);
  const int piece = lane & 7, r0 = lane >> 3;
  const T* src = c0 + (int64_t)r0 * p.ldc + piece * kElems;
#pragma unroll
  for (int i = 0; i < 8; ++i, src += 4 * p.ldc)
#pragma unroll
    for (int u = 0; u < N; ++u) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (p.c_vec && n >= (u + 1) * kCols && i * 4 + r0 < rows) v = *reinterpret_cast<const uint4*>(src + u * kCols);
      w[u][4 * i] = v.x;
      w[u][4 * i + 1] = v.y;
      w[u][4 * i + 2] = v.z;
      w[u][4 * i + 3] = v.w;
    }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    if (n <= u * kCols) continue;  // zeros, if they were used
    if (p.c_vec && n >= (u + 1) * kCols) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(sb + staged<32>(i * 4 + r0, piece)) =
            make_uint4(w[u][4 * i], w[u][4 * i + 1], w[u][4 * i + 2], w[u][4 * i + 3]);
    } else {
#pragma unroll 1
      for (int c = lane; c < kCols; c += 32)
#pragma unroll 1
        for (int r = 0; r < 32; ++r)
          *reinterpret_cast<T*>(sb + staged<32>(r, c / kElems) + (c % kElems) * sizeof(T)) =
              r < rows && u * kCols + c < n ? c0[(int64_t)r * p.ldc + u * kCols + c] : T{};
    }
    __syncwarp();
    row_of_block(sb, lane, w[u]);
  }
}

// 32 rows by 32 fp32 columns into the staging block without a register (the sums'
// 128 leave none: any that is spilled goes to L2, nearly all of L1 being shared
// memory here), asynchronously where C allows it; copy_async_wait and a __syncwarp
// come before their use.
__device__ __forceinline__ void stage_rows_async(const GroupedParams& p, const float* c0, int rows, int n, int lane,
                                                 uint8_t* sb) {
  n = max(0, min(n, 32));
  const int whole = p.c_vec ? n & ~3 : 0;
  const int piece = lane & 7, r0 = lane >> 3;
  if (piece * 4 < whole) {
    const float* src = c0 + (int64_t)r0 * p.ldc + piece * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 4 + r0 < rows) copy_async_16(sb + staged<32>(i * 4 + r0, piece), src + (int64_t)(i * 4) * p.ldc);
  }
  if (whole < n) {
#pragma unroll 1
    for (int r = 0; r < rows; ++r)
      if (lane >= whole && lane < n)
        *reinterpret_cast<float*>(sb + staged<32>(r, lane / 4) + (lane & 3) * 4) = c0[(int64_t)r * p.ldc + lane];
  }
}

// What an epilogue warp has of a tile: 32 rows by 128 columns (of half a tile 64).
template <typename T>
struct EpiTile {
  T* d;        // its first element of D, and of C (null without C)
  const T* c;
  int g, col0;
  int at;       // the accumulator's column of col0
  int64_t row;  // its first row of D
  int rows, cols;  // rows inside the group (wgrad: inside D); columns of the tile inside D, from col0 on
  int k_blocks;
};

template <bool WGRAD, typename T>
__device__ __forceinline__ EpiTile<T> epi_tile(const GroupedParams& p, const PairItem& item, uint32_t rank, int q,
                                               int part) {
  const GroupedTile& x = item.x;
  EpiTile<T> e;
  const int r0 = x.rb * kTile + (int)rank * 128 + q * 32;
  const int64_t row0 = WGRAD ? r0 : (int64_t)x.lo + r0;
  e.g = x.g;
  e.at = part * (item.half < 0 ? kTile / 2 : kTile / 4);
  e.col0 = x.cb * kTile + max(item.half, 0) * (kTile / 2) + e.at;
  e.row = row0;
  e.rows = max(0, min(32, WGRAD ? p.K - r0 : x.hi - x.lo - r0));
  e.cols = min(p.N - e.col0, item.half < 0 ? kTile / 2 : kTile / 4);
  e.d = static_cast<T*>(p.D) + (WGRAD ? (int64_t)x.g * p.strideD : 0) + row0 * p.ldd + e.col0;
  e.c = WGRAD && p.C != nullptr ? static_cast<const T*>(p.C) + (int64_t)x.g * p.strideC + row0 * p.ldc + e.col0 : nullptr;
  e.k_blocks = pair_loop<WGRAD>(p, x).k_blocks;
  return e;
}

// Sixteen sums of a row (columns s16 * 16 on), scaled: each lane has four columns'
// scales and biases and hands them round.  Loaded where they are used, they cost
// the epilogue a wait for L2 every sixteen columns (10.5 us a tile of 256 x 256
// x 560 in place of 7).
__device__ __forceinline__ void scaled_values(const GroupedParams& p, const uint32_t* sums, float scale, float4 sc,
                                              float4 bias, int s16, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int src = s16 * 4 + i;
    const float w[4] = {__shfl_sync(0xFFFFFFFFu, sc.x, src), __shfl_sync(0xFFFFFFFFu, sc.y, src),
                        __shfl_sync(0xFFFFFFFFu, sc.z, src), __shfl_sync(0xFFFFFFFFu, sc.w, src)};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * i + k] = __uint_as_float(sums[4 * i + k]) * scale * w[k];
  }
  if (p.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int src = s16 * 4 + i;
      v[4 * i] += __shfl_sync(0xFFFFFFFFu, bias.x, src);
      v[4 * i + 1] += __shfl_sync(0xFFFFFFFFu, bias.y, src);
      v[4 * i + 2] += __shfl_sync(0xFFFFFFFFu, bias.z, src);
      v[4 * i + 3] += __shfl_sync(0xFFFFFFFFu, bias.w, src);
    }
  }
  if (p.act != kActNone) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = act_value(p.act, v[j]);
  }
}

// A gated block's tiles: this warp's 32 rows by 64 columns of D forward (of half a
// tile 32), by 128 (of half a tile 64) of its gradient.
template <bool BF16, typename P>
__device__ __forceinline__ void gated_tiles(const P& p, const GroupTable& tb, const PairWalk& walk, int pair, int num_pairs,
                                            uint32_t rank, int q, int part, uint32_t tmem_mine, uint8_t* sb, int lane,
                                            uint64_t* tmem_full, uint64_t* tmem_empty, const WaitCtx& wc) {
  const bool has_k = p.k_blocks > 0;
  int it = 0;
  for (int t = pair; t < walk.items; t += num_pairs, ++it) {
    const PairItem item = pair_item<false>(p, tb, walk, t);
    const GroupedTile& x = item.x;
    const int r0 = x.rb * kTile + (int)rank * 128 + q * 32;
    const int64_t row = (int64_t)x.lo + r0;
    const int rows = max(0, min(32, x.hi - x.lo - r0));
    const int acc = it & 1;
    const uint32_t at = tmem_mine + acc * kTile;
    const auto wait = [&] {
      const bool ok = mbar_wait_warp(&tmem_full[acc], (it >> 1) & 1, wc);
      tc_fence_after();
      return ok;
    };
    const auto release = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
    };
    if constexpr (kIsGatedForward<P>) {
      const int width = item.half < 0 ? kTile / 4 : kTile / 8;  // of this warp; the tile has twice as many
      const int col = x.cb * (kTile / 2) + max(item.half, 0) * (kTile / 4) + part * width;
      if (!wait()) return;
      gated_forward_unit<BF16>(p, at + part * width, at + (2 + part) * width, has_k, row, rows, col, min(width, p.N - col), sb,
                               lane, release);
    } else {
      const int units = item.half < 0 ? 2 : 1;
      const int col = x.cb * kTile + max(item.half, 0) * (kTile / 2) + part * units * 64;
#pragma unroll 1
      for (int u = 0; u < units; ++u)
        if (!gated_grad_unit<BF16>(p, at + (part * units + u) * 64, has_k, row, rows, col + u * 64, p.N - col - u * 64, sb, lane,
                                   [&] { return u > 0 || wait(); },
                                   [&] {
                                     if (u == units - 1) release();
                                   }))
          return;
    }
  }
}

// ADD: C is read (wgrad); a parameter of its own because the fp32 sums leave
// few registers for it.
// I8: forward with int8 sums, scaled; BF16 then is the type of a 16-bit result.
// P: GroupedParams, or those of a gated block, whose forward tiles are 256 rows by 128
// columns of D: the even CTA stages the gate's 128 columns of weights, the odd one the
// other projection's, so that an accumulator holds both side by side.
template <bool BF16, bool WGRAD, bool F32, bool ADD, bool I8 = false, typename P = GroupedParams>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_pair_kernel(const __grid_constant__ P p) {
  static_assert(WGRAD || ((!F32 || I8) && !ADD), "forward results are 16-bit and added to nothing");
  static_assert(!kIsGated<P> || !(WGRAD || F32 || ADD || I8), "gated blocks are forward products");
  static_assert(!WGRAD || !I8, "int8 products are forward ones");
  constexpr bool kSums = F32 || I8;  // partial sums in registers
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;  // [stage][k-block of the stage, or 64 rows]
  uint8_t* sB = sA + kStages * kShareBytes;
  uint8_t* staging = sB + kStages * kShareBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStagingBytes);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* fix = bars + 2 * kStages;  // wgrad: a stage's loads by this CTA, where its last rows are to be cleared
  uint64_t* tmem_full = bars + 3 * kStages;
  uint64_t* tmem_empty = bars + 3 * kStages + 2;
  uint64_t* stall_bar = bars + 3 * kStages + 4;
  uint64_t* drain_bar = bars + 3 * kStages + 5;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kStages + 6);
  // what the producer tells the MMA issuer about a stage
  int* stage_info = reinterpret_cast<int*>(bars + 3 * kStages + 7);
  int* table = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);
  // the whole table where it has room, else only every fourth group's first tile
  GroupTable tb{nullptr, nullptr, 1, p.col_blocks};
  if constexpr (WGRAD) {
    if (p.groups + 1 <= kTableInts) tb.offs = table;
  } else if (2 * (p.groups + 1) <= kTableInts) {
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
      mbar_init(&full[lane], WGRAD ? 2 : 1);  // wgrad: both CTAs arrive, the producers or the clearing warps
      mbar_init(&empty[lane], 1);
      mbar_init(&fix[lane], 1);
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
      if constexpr (kIsGatedForward<P>) prefetch_tmap(&p.tmU);
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
  const PairWalk walk = pair_walk(WGRAD ? p.groups * p.row_blocks * p.col_blocks : table_tiles(p, tb), num_pairs);

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
      for (int t = pair; ok && t < walk.items; t += num_pairs) {
        const PairItem item = pair_item<WGRAD>(p, tb, walk, t);
        const GroupedTile& x = item.x;
        const PairLoop l = pair_loop<WGRAD>(p, x);
        // of half a tile the MMA reads 64 columns, the first of the 128 that are loaded
        int n0 = x.cb * kTile + (item.half < 0 ? (int)rank * 128 : item.half * 128 + (int)rank * 64);
        const CUtensorMap* map_b = &p.tmB;
        if constexpr (kIsGatedForward<P>) {
          n0 = x.cb * (kTile / 2) + max(item.half, 0) * (kTile / 4);
          if (!leader) map_b = &p.tmU;
        }
        const int m0 = (WGRAD ? 0 : x.lo) + x.rb * kTile + (int)rank * 128;
        // forward: whether this CTA's, and the other's, rows of A hold any of the group
        const bool a_on = WGRAD || m0 < x.hi;
        const int halves = WGRAD || x.lo + x.rb * kTile + 128 < x.hi ? 2 : 1;
        const int zb = WGRAD ? 0 : (p.strideB != 0 ? x.g : 0);
        int kb0 = 0;
        do {  // a tile without k-blocks takes a stage without loads
          const int nkb = min(kKPS, l.k_blocks - kb0);
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          if (leader) stage_info[stage] = stage_word(nkb, l.last_steps, kb0 + nkb >= l.k_blocks, item.half >= 0);
          const bool b_mn = WGRAD || p.b_mn;
          const int bytes_a = nkb > 0 ? share_bytes(WGRAD, nkb) : 0, bytes_b = nkb > 0 ? share_bytes(b_mn, nkb) : 0;
          const bool clear = WGRAD && l.fix_rows != 0 && kb0 + nkb == l.k_blocks;
          const uint32_t full_leader = mapa_shared(smem_u32(&full[stage]), 0);
          if (clear) {
            mbar_arrive_expect_tx(&fix[stage], bytes_a + bytes_b);
            armed &= ~(1u << stage);  // what it held has landed; `full` goes on without the producer
            fixed |= 1u << stage;
            fix_parity = (fix_parity & ~(1u << stage)) | (fix_phase & (1u << stage));
            fix_phase ^= 1u << stage;
          } else if (leader) {
            mbar_arrive_expect_tx(&full[stage], halves * bytes_a + 2 * bytes_b);
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          } else if (WGRAD) {
            mbar_arrive_cluster_relaxed(full_leader);
          }
          uint8_t* a = sA + stage * kShareBytes;
          uint8_t* b = sB + stage * kShareBytes;
          const int k0 = (WGRAD ? x.lo : 0) + kb0 * kBK;
          if (nkb == 0) {
            // nothing to load
          } else if (clear) {
            load_share<false>(a, &p.tmA, WGRAD, nkb, m0, k0, 0, &fix[stage], 0, keep);
            load_share<false>(b, map_b, b_mn, nkb, n0, k0, zb, &fix[stage], 0, pol_b);
          } else {
            if (a_on) load_share<true>(a, &p.tmA, WGRAD, nkb, m0, k0, 0, nullptr, full_leader, keep);
            load_share<true>(b, map_b, b_mn, nkb, n0, k0, zb, nullptr, full_leader, pol_b);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
          kb0 += kKPS;
        } while (kb0 < l.k_blocks);
      }
      // a stage completes once both CTAs' loads for it have landed, one to be cleared with this CTA's
      drain_ring(fix, kStages, fixed, fix_parity);
      if (leader)
        drain_ring(full, kStages, armed, armed_parity);
      else
        drain_odd_cta(wc);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (even CTA)
    if (leader && lane == 0) {
      const bool b_mn = WGRAD || p.b_mn != 0;
      const uint32_t idesc_whole = idesc_f16(BF16 && !I8, WGRAD, b_mn, kTile, kTile);
      const uint32_t idesc_half = idesc_f16(BF16 && !I8, WGRAD, b_mn, kTile, kTile / 2);
      const uint64_t a0 = smem_desc_sw128(smem_u32(sA), WGRAD ? (uint32_t)kHalfBytes : 16u, 1024);
      const uint64_t b0 = smem_desc_sw128(smem_u32(sB), b_mn ? (uint32_t)kHalfBytes : 16u, 1024);
      const uint64_t a_step = WGRAD ? 2048u >> 4 : 32u >> 4, b_step = b_mn ? 2048u >> 4 : 32u >> 4;
      // from one k-block of a stage to the next
      const uint32_t a_kb = (WGRAD ? kHalfBytes / 2 : kHalfBytes) >> 4, b_kb = (b_mn ? kHalfBytes / 2 : kHalfBytes) >> 4;
      bool ok = true, any = false;
      if (p.inject_stall) ok = mbar_wait(stall_bar, 0, wc);  // nothing arrives here
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ready = true;  // whether the next accumulator is known to be free
      // the first use of each accumulator passes at once
      for (int t = pair; ok && t < walk.items; t += num_pairs) {
        bool last = false;
        do {  // an accumulator: the tile's, or a chunk of it
          const int acc = it & 1;
          if (!ready && !mbar_wait_cluster(&tmem_empty[acc], ((it >> 1) & 1) ^ 1u, wc)) {
            ok = false;
            break;
          }
          ready = false;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * kTile;
          int done = 0;  // k-blocks in this accumulator
          do {
            // zeros written by the other CTA's threads are behind this barrier in wgrad
            if (!(WGRAD ? mbar_wait_cluster(&full[stage], phase, wc) : mbar_wait(&full[stage], phase, wc))) {
              ok = false;
              break;
            }
            const int info = stage_info[stage];
            const int nkb = info & 15, steps = (info >> 4) & 15;
            last = (info & 256) != 0;
            const uint32_t idesc = (info & 512) != 0 ? idesc_half : idesc_whole;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < kKPS; ++j) {
              if (j < nkb) {
                const uint64_t ad = a0 + (uint32_t)stage * (kShareBytes >> 4) + j * a_kb;
                const uint64_t bd = b0 + (uint32_t)stage * (kShareBytes >> 4) + j * b_kb;
                mma_f16_pair(d_tmem, ad, bd, idesc, (done | j) != 0);
#pragma unroll
                for (int k = 1; k < kBK / kUmmaK; ++k)
                  if (!WGRAD || k < steps || j + 1 < nkb) mma_f16_pair(d_tmem, ad + k * a_step, bd + k * b_step, idesc, 1u);
              }
            }
            done += nkb;
            any = any || nkb > 0;
            mma_commit_pair(&empty[stage], 0x3);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
            if (!ready) ready = mbar_test_cluster(&tmem_empty[acc ^ 1], (((it + 1) >> 1) & 1) ^ 1u);
          } while (!last && (!kSums || done < kChunkKBlocks<I8>));
          if (!ok) break;
          mma_commit_pair(&tmem_full[acc], 0x3);
          ++it;
        } while (!last);
      }
      if (any) {
        // every MMA must have finished with both CTAs' TMEM before it is freed
        mma_commit_pair(drain_bar, 0x1);
        drain_wait(drain_bar, 0, 100000000ull);
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int ew = warp - kEpiWarp0, q = warp & 3, part = ew >> 2;  // quarter of the rows, half of the columns
    using T = typename std::conditional<F32, float, uint16_t>::type;
    constexpr int kUnit = 128 / (int)sizeof(T);    // columns that 128 bytes hold
    constexpr int kUnits = kTile / 2 / kUnit;      // of this warp
    uint8_t* sb = staging + ew * 4096;
    const uint32_t tmem_mine = tmem_base + ((uint32_t)(q * 32) << 16);
    int it = 0;
    bool ok = true;
    if constexpr (kIsGated<P>) {
      gated_tiles<BF16>(p, tb, walk, pair, num_pairs, rank, q, part, tmem_mine, sb, lane, tmem_full, tmem_empty, wc);
      ok = false;
    }
    for (int t = pair; ok && t < walk.items; t += num_pairs) {
      const EpiTile<T> e0 = epi_tile<WGRAD, T>(p, pair_item<WGRAD>(p, tb, walk, t), rank, q, part);
      if constexpr (kSums) {
        // floats (int8 with more than one accumulator: int32): this thread's row of the
        // warp's 128 columns
        uint32_t sums[kTile / 64][32];
#pragma unroll
        for (int c = 0; c < kTile / 64; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) sums[c][j] = 0u;
        const int k_blocks = e0.k_blocks;
        int kbeg = 0;
        // C joins the sums 32 columns at a time while the products are on their way,
        // as many before each partial sum that all have before the last
        const float* cf = reinterpret_cast<const float*>(e0.c);
        const int chunks = max(1, (k_blocks + kChunkKBlocks<I8> - 1) / kChunkKBlocks<I8>);
        int joined = 0, chunk = 0;
        if constexpr (ADD) stage_rows_async(p, cf, e0.rows, e0.cols, lane, sb);
        do {
          if constexpr (ADD) {
            const int due = min(kTile / 64, kTile / 64 * ++chunk / chunks);
#pragma unroll
            for (int u = 0; u < kTile / 64; ++u) {
              if (u < joined || u >= due) continue;
              copy_async_wait();
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 c = *reinterpret_cast<const float4*>(sb + staged<32>(lane, i));
                sums[u][4 * i] = __float_as_uint(fmaf(p.beta, c.x, __uint_as_float(sums[u][4 * i])));
                sums[u][4 * i + 1] = __float_as_uint(fmaf(p.beta, c.y, __uint_as_float(sums[u][4 * i + 1])));
                sums[u][4 * i + 2] = __float_as_uint(fmaf(p.beta, c.z, __uint_as_float(sums[u][4 * i + 2])));
                sums[u][4 * i + 3] = __float_as_uint(fmaf(p.beta, c.w, __uint_as_float(sums[u][4 * i + 3])));
              }
              __syncwarp();
              if (u + 1 < kTile / 64) stage_rows_async(p, cf + u * 32 + 32, e0.rows, e0.cols - u * 32 - 32, lane, sb);
            }
            joined = due;
          }
          const int acc = it & 1;
          if (!mbar_wait(&tmem_full[acc], (it >> 1) & 1, wc)) {
            if constexpr (ADD) copy_async_wait();
            ok = false;
            break;
          }
          tc_fence_after();
          if (I8 && k_blocks <= kChunkKBlocks<I8>) {
            // one accumulator: its values are the sums, whole numbers in fp32
#pragma unroll
            for (int c = 0; c < kTile / 64; ++c) tmem_ld_32x32b_x32(tmem_mine + e0.at + acc * kTile + c * 32, sums[c]);
            tmem_ld_wait();
          } else if (k_blocks > 0) {
#pragma unroll
            for (int c = 0; c < kTile / 32; ++c) {
              uint32_t w[16];
              tmem_ld_32x32b_x16<0>(tmem_mine + e0.at + acc * kTile + c * 16, w);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                uint32_t& sum = sums[c / 2][c % 2 * 16 + j];
                if constexpr (I8)
                  sum += (uint32_t)__float2int_rn(__uint_as_float(w[j]));  // an integer of at most 2^24
                else if constexpr (ADD)
                  sum = __float_as_uint(fmaf(p.alpha, __uint_as_float(w[j]), __uint_as_float(sum)));
                else
                  sum = __float_as_uint(__uint_as_float(sum) + __uint_as_float(w[j]));
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
          ++it;
          kbeg += kChunkKBlocks<I8>;
        } while (kbeg < k_blocks);
        if (!ok) break;
        // found again rather than kept: the sums leave no registers for it
        int t_again = t;
        asm volatile("" : "+r"(t_again));
        const EpiTile<T> e = epi_tile<WGRAD, T>(p, pair_item<WGRAD>(p, tb, walk, t_again), rank, q, part);
        if constexpr (I8) {
          const float scale = lane < e.rows ? __ldg(p.scale_a + e.row + lane) : 0.0f;
          const float4 sc = four_columns(p.scale_b + e.col0, lane, e.cols);
          const float4 bias =
              p.bias != nullptr ? four_columns(p.bias + e.col0, lane, e.cols) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (k_blocks > kChunkKBlocks<I8>) {
#pragma unroll
            for (int c = 0; c < kTile / 64; ++c)
#pragma unroll
              for (int j = 0; j < 32; ++j) sums[c][j] = __float_as_uint(__int2float_rn((int32_t)sums[c][j]));
          }
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
#pragma unroll
            for (int h = 0; h < kUnit / 16; ++h) {
              const int s16 = u * (kUnit / 16) + h;
              float v[16];
              scaled_values(p, sums[s16 / 2] + s16 % 2 * 16, scale, sc, bias, s16, v);
              if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  *reinterpret_cast<float4*>(sb + staged<32>(lane, h * 4 + i)) =
                      make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
              } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  *reinterpret_cast<uint4*>(sb + staged<32>(lane, h * 2 + i)) =
                      make_uint4(pack2<BF16>(v[8 * i], v[8 * i + 1]), pack2<BF16>(v[8 * i + 2], v[8 * i + 3]),
                                 pack2<BF16>(v[8 * i + 4], v[8 * i + 5]), pack2<BF16>(v[8 * i + 6], v[8 * i + 7]));
              }
            }
            __syncwarp();
            copy_out<T, 4>(p, sb, e.d + u * kUnit, e.rows, e.cols - u * kUnit, lane);
            __syncwarp();
          }
          continue;
        }
        float* df = reinterpret_cast<float*>(e.d);
#pragma unroll
        for (int c = 0; c < kTile / 64; ++c) {
          const float scale = ADD ? 1.0f : p.alpha;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(sb + staged<32>(lane, i)) =
                make_float4(scale * __uint_as_float(sums[c][4 * i]), scale * __uint_as_float(sums[c][4 * i + 1]),
                            scale * __uint_as_float(sums[c][4 * i + 2]), scale * __uint_as_float(sums[c][4 * i + 3]));
          __syncwarp();
          copy_out<float, 4>(p, sb, df + c * 32, e.rows, e.cols - c * 32, lane);
          __syncwarp();
        }
      } else {
        const int acc = it & 1;
        float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!WGRAD && p.bias != nullptr)
          bias = four_columns(p.bias + (int64_t)e0.g * p.stride_bias + e0.col0, lane, e0.cols);
        uint32_t cw[ADD ? kUnits : 1][32];
        if constexpr (ADD) load_c(p, e0.c, e0.rows, e0.cols, lane, sb, cw);
        if (!mbar_wait(&tmem_full[acc], (it >> 1) & 1, wc)) break;
        ++it;
        tc_fence_after();
#pragma unroll (ADD ? kUnits : 1)
        for (int u = 0; u < kUnits; ++u) {
          uint32_t w[2][32];
          if (e0.k_blocks > 0) {
            tmem_ld_32x32b_x32(tmem_mine + e0.at + acc * kTile + u * kUnit, w[0]);
            tmem_ld_32x32b_x32(tmem_mine + e0.at + acc * kTile + u * kUnit + 32, w[1]);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) w[0][j] = w[1][j] = 0u;
          }
          if (u == kUnits - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tmem_empty[acc]), 0));
          }
          if (e0.cols <= u * kUnit) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            grouped_values(p, w[h], bias, u * 2 + h, v);
            if (ADD) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                v[2 * j] = fmaf(p.beta, half_bits_to_float<BF16>((uint16_t)(cw[ADD ? u : 0][h * 16 + j] & 0xFFFFu)), v[2 * j]);
                v[2 * j + 1] = fmaf(p.beta, half_bits_to_float<BF16>((uint16_t)(cw[ADD ? u : 0][h * 16 + j] >> 16)), v[2 * j + 1]);
              }
            }
#pragma unroll
            for (int ch = 0; ch < 4; ++ch)
              *reinterpret_cast<uint4*>(sb + staged<32>(lane, h * 4 + ch)) =
                  make_uint4(pack2<BF16>(v[8 * ch], v[8 * ch + 1]), pack2<BF16>(v[8 * ch + 2], v[8 * ch + 3]),
                             pack2<BF16>(v[8 * ch + 4], v[8 * ch + 5]), pack2<BF16>(v[8 * ch + 6], v[8 * ch + 7]));
          }
          __syncwarp();
          copy_out<T, 4>(p, sb, e0.d + u * kUnit, e0.rows, e0.cols - u * kUnit, lane);
          __syncwarp();
        }
      }
    }
  } else if (WGRAD && warp == 2) {
    // ---------------------------------------------------------------- wgrad: rows behind a group's end (both CTAs)
    int stage = 0;
    uint32_t fix_phase = 0;
    bool ok = true;
    for (int t = pair; ok && t < walk.items; t += num_pairs) {
      const PairLoop l = pair_loop<WGRAD>(p, pair_item<WGRAD>(p, tb, walk, t).x);
      const int stages = max(1, (l.k_blocks + kKPS - 1) / kKPS);
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
        // the k-block's rows of a 64-wide slab, 128 bytes each; two slabs an operand
        uint8_t* ops[2] = {sA + s * kShareBytes + j * (kHalfBytes / 2), sB + s * kShareBytes + j * (kHalfBytes / 2)};
#pragma unroll
        for (int o = 0; o < 2; ++o)
          for (int i = lane; i < 2 * n16; i += 32) {
            const int slab = i >= n16 ? 1 : 0;
            *reinterpret_cast<uint4*>(ops[o] + slab * kHalfBytes + l.fix_rows * 128 + (i - slab * n16) * 16) =
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

template <bool BF16, bool WGRAD, bool F32, bool ADD, bool I8 = false, typename P = GroupedParams>
cudaError_t prepare() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(grouped_pair_kernel<BF16, WGRAD, F32, ADD, I8, P>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  return cudaSuccess;
}

template <bool BF16, bool WGRAD, bool F32, bool ADD>
int clusters_of() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load();
  if (n > 0) return n;
  if (prepare<BF16, WGRAD, F32, ADD>() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaOccupancyMaxActiveClusters(&n, grouped_pair_kernel<BF16, WGRAD, F32, ADD>, &cfg) != cudaSuccess) return 0;
  known[dev].store(n);
  return n;
}

template <bool BF16, bool WGRAD, bool F32, bool ADD, bool I8 = false, typename P = GroupedParams>
cudaError_t launch(const P& p, int clusters, cudaStream_t stream) {
  cudaError_t e = prepare<BF16, WGRAD, F32, ADD, I8, P>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, grouped_pair_kernel<BF16, WGRAD, F32, ADD, I8, P>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Pairs that can be resident at once (0 on error): one CTA fits an SM whatever
// the variant.
int grouped_pair_clusters() { return clusters_of<true, false, false, false>(); }

cudaError_t launch_grouped_pair(bool bf16, bool wgrad, const GroupedParams& p, int clusters, cudaStream_t stream) {
  const bool add = p.C != nullptr;
#define TTC_PAIR(W, F, C) \
  (bf16 ? launch<true, W, F, C>(p, clusters, stream) : launch<false, W, F, C>(p, clusters, stream))
  if (!wgrad) return TTC_PAIR(false, false, false);
  if (p.out_f32) return add ? TTC_PAIR(true, true, true) : TTC_PAIR(true, true, false);
  return add ? TTC_PAIR(true, false, true) : TTC_PAIR(true, false, false);
#undef TTC_PAIR
}

cudaError_t launch_gated_pair(bool bf16, const GatedForward& p, int clusters, cudaStream_t stream) {
  return bf16 ? launch<true, false, false, false, false>(p, clusters, stream)
              : launch<false, false, false, false, false>(p, clusters, stream);
}

cudaError_t launch_gated_pair(bool bf16, const GatedGrad& p, int clusters, cudaStream_t stream) {
  return bf16 ? launch<true, false, false, false, false>(p, clusters, stream)
              : launch<false, false, false, false, false>(p, clusters, stream);
}

cudaError_t launch_pair_i8_scaled(bool bf16_out, const GroupedParams& p, int clusters, cudaStream_t stream) {
  if (p.out_f32) return launch<false, false, true, false, true>(p, clusters, stream);
  return bf16_out ? launch<true, false, false, false, true>(p, clusters, stream)
                  : launch<false, false, false, false, true>(p, clusters, stream);
}

}  // namespace ttc
