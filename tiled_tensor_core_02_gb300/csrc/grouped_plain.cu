// Grouped products for operands of any pitch and alignment: the kernel that is
// right for every case.  One CTA per 128 x 128 tile, persistent; eight warps
// bring the operands into 128-byte-swizzled shared memory, one thread issues
// tcgen05.mma, four warps drain the accumulator.  In the gradient of the weights
// the reduction runs over the group's rows, so both operands lie with the
// reduction outermost, as the MMA takes them too.
//
// Eight elements that start at any 2-byte boundary lie in one or two aligned
// 16-byte blocks; a thread loads those and shifts them into place, all of its
// eight pieces of a k-block before it stores the first, so that up to 64 KB are on
// the way.  Only blocks that hold a byte of the row are read; what is outside the
// group's rows and the operand's extents is zero and not loaded.
//
// fp32 gradients start a fresh accumulator every kSumKBlocks k-blocks, whose values
// the epilogue warps add up in tensor memory: 7e-7 of the result however many
// tokens there are, where one accumulator over 8192 is at 6.4e-6.
//
// Gated blocks run here too: forward a tile has 64 columns of either projection's weights,
// 8192 x 14336 x 4096 at 263 TFLOP/s.
//
// Bound by the producers, which a k-block of 2 x 16 KB takes 1.0 us (asking L2 for
// its lines four k-blocks ahead changed nothing): 8192 rows over 8 groups, 4099 x
// 4099, 1064 us or 259 TFLOP/s, the gradient 1110; 856 rows over 32 groups, 2712 x
// 3337, 320 us, where loads of single elements took 1633; 32 rows over 4 groups,
// 1001 x 4095, 69 us, 64 k-blocks one after the other.  Operands TMA can read take
// the other kernels.
#include "gated_common.cuh"

#include <atomic>
#include <type_traits>

namespace ttc {

namespace {

constexpr int kTile = kGroupedPlainTile;
constexpr int kStages = 4;
constexpr int kProducers = 8;  // warps; then four of the epilogue and the MMA issuer
constexpr int kIssuer = kProducers + 4;
constexpr int kThreads = 32 * (kIssuer + 1);
constexpr int kOperandBytes = kTile * kBK * 2;
constexpr int kTableBytes = 2 * (kMaxGroups + 4) * 4;
constexpr int kStagingBytes = 4 * 4096;
constexpr int kSmemBytes = 1024 + kStages * 2 * kOperandBytes + kStagingBytes + 256 + kTableBytes;

// A k-block's tile of an operand: ROWS rows of COLS contiguous elements from
// (outer0, inner0) on, in 64-column slabs of ROWS 128-byte rows with the 128-byte
// swizzle, the layout TMA writes.  One thread's pieces of eight elements.  (Leaving
// pieces outside D's rows and columns out put branches between the loads: 1683 us
// against 1164 for 8192 rows, 8 groups, 4099 x 4099.)
template <int ROWS, int COLS>
struct TilePieces {
  static constexpr int kPerRow = COLS / 8;
  static constexpr int kCount = ROWS * kPerRow / (32 * kProducers);
  uint4 lo[kCount], hi[kCount];
  uint32_t phase[kCount];
  int n[kCount];  // elements inside the operand

  __device__ __forceinline__ void load(const void* src, int64_t ld, int outer0, int inner0, int outer_ext,
                                       int inner_ext, int tid) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const int piece = tid + i * 32 * kProducers;
      const int go = outer0 + piece / kPerRow, gi = inner0 + piece % kPerRow * 8;
      n[i] = go < outer_ext ? max(0, min(8, inner_ext - gi)) : 0;
      const uintptr_t at = reinterpret_cast<uintptr_t>(src) + ((int64_t)go * ld + gi) * 2;
      phase[i] = (uint32_t)(at & 15);
      const uint4* blk = reinterpret_cast<const uint4*>(at - phase[i]);
      lo[i] = n[i] > 0 ? __ldg(blk) : make_uint4(0u, 0u, 0u, 0u);
      hi[i] = (int)phase[i] + 2 * n[i] > 16 ? __ldg(blk + 1) : make_uint4(0u, 0u, 0u, 0u);
    }
  }

  __device__ __forceinline__ void store(uint8_t* dst, int tid) const {
    constexpr layout::SwizzleBytes128 swz{};
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      uint32_t x[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
      // bytes down by the phase (even): stages of 8, 4 and 2
      const bool s8 = phase[i] & 8, s4 = phase[i] & 4;
#pragma unroll
      for (int k = 0; k < 6; ++k) x[k] = s8 ? x[k + 2] : x[k];
#pragma unroll
      for (int k = 0; k < 5; ++k) x[k] = s4 ? x[k + 1] : x[k];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = __funnelshift_r(x[k], x[k + 1], (phase[i] & 2) * 8);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = n[i] >= 2 * k + 2 ? x[k] : n[i] == 2 * k + 1 ? x[k] & 0xFFFFu : 0u;
      const int piece = tid + i * 32 * kProducers, r = piece / kPerRow, c = piece % kPerRow;
      *reinterpret_cast<uint4*>(dst + swz((uint32_t)((c / 8) * ROWS * 128 + r * 128 + (c % 8) * 16))) =
          make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
};

using Inner = TilePieces<kTile, kBK>;  // the reduction lies innermost
using Outer = TilePieces<kBK, kTile>;  // outermost
using HalfTile = TilePieces<kGatedPlainCols, kBK>;  // half of a gated block's columns, either way
static_assert(kGatedPlainCols == kBK && 2 * kGatedPlainCols == kTile, "a gated tile's halves are square");

// Tensor memory behind the two accumulators, for fp32 gradients: the sum of a tile's
// accumulators (there are no registers for 128 columns a thread).
constexpr int kSumsAt = 2 * kTile;

// Adds `more` accumulators of a tile, the it-th on, to the one behind them, in the
// warp's rows; false after an error.
__device__ __forceinline__ bool add_accumulators(uint32_t tmem_mine, int it, int more, uint64_t* tmem_full,
                                                 uint64_t* tmem_empty, const WaitCtx& wc) {
  for (int i = 0; i <= more; ++i, ++it) {
    if (!mbar_wait(&tmem_full[it & 1], (it >> 1) & 1, wc)) return false;
    tc_fence_after();
    const uint32_t acc = tmem_mine + (it & 1) * kTile, sums = tmem_mine + kSumsAt;
#pragma unroll 1
    for (int at = 0; at < kTile; at += 32) {
      uint32_t w[32], s[32];
      tmem_ld_32x32b_x32(acc + at, w);
      if (i > 0) tmem_ld_32x32b_x32(sums + at, s);
      tmem_ld_wait();
      if (i > 0) {
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(s[j]) + __uint_as_float(w[j]));
      }
      tmem_st_32x32b_x32((i < more ? sums : acc) + at, w);
    }
    tmem_st_wait();
    if (i < more) {
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&tmem_empty[it & 1]);
    }
  }
  return true;
}

// The epilogue's walk: each warp 32 rows of every tile, in blocks of 128 bytes a
// row through its staging block, so that C is read and D written a row an
// instruction whatever their alignment.
template <bool BF16, bool WGRAD, typename T>
__device__ __forceinline__ void drain_tiles(const GroupedParams& p, const GroupTable& tb, int tiles, uint32_t tmem_base,
                                            uint8_t* sb, uint64_t* tmem_full, uint64_t* tmem_empty, const WaitCtx& wc) {
  constexpr int kUnit = 128 / (int)sizeof(T);  // columns
  constexpr int kPer = 16 / (int)sizeof(T);    // of a 16-byte piece
  // rows of single columns read before the first is stored: short tiles of gradients are all
  // stores (1023 rows, 32 groups, 1001 x 1023 bf16: 56 us, by eight 80), forward by eight 1067 us
  // against 1088 (8192 rows, 8 groups, 4099 x 4099)
  constexpr int kAtOnce = WGRAD ? 32 : 8;
  const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  int it = 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
    const GroupedTile x = grouped_tile<kTile, WGRAD>(p, tb, t);
    const bool has_k = WGRAD ? x.hi > x.lo : p.k_blocks > 0;
    if constexpr (WGRAD && sizeof(T) == 4) {
      const int more = ((x.hi - x.lo + kBK - 1) / kBK - 1) / kSumKBlocks;
      if (more > 0) {
        if (!add_accumulators(tmem_base + ((uint32_t)(q * 32) << 16), it, more, tmem_full, tmem_empty, wc)) break;
        it += more;
      }
    }
    const int acc = it & 1;
    const int r0 = x.rb * kTile + q * 32;  // of the warp, in its group in forward
    const int64_t row0 = WGRAD ? r0 : (int64_t)x.lo + r0;
    const int rows = max(0, min(32, WGRAD ? p.K - r0 : x.hi - x.lo - r0));
    const int col0 = x.cb * kTile;
    T* d = static_cast<T*>(p.D) + (WGRAD ? (int64_t)x.g * p.strideD : 0) + row0 * p.ldd + col0;
    const T* c = WGRAD && p.C != nullptr ? static_cast<const T*>(p.C) + (int64_t)x.g * p.strideC + row0 * p.ldc + col0
                                         : nullptr;
    float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!WGRAD && p.bias != nullptr) bias = four_columns(p.bias + (int64_t)x.g * p.stride_bias + col0, lane, p.N - col0);
    if (!mbar_wait(&tmem_full[acc], (it >> 1) & 1, wc)) break;
    tc_fence_after();
#pragma unroll 1
    for (int at = 0; at < kTile; at += kUnit) {
      const int n = min(kUnit, p.N - col0 - at);
      if (c != nullptr) {
        for (int j = lane; j < n; j += 32) {
          const T* src = c + at + j;
          T y[32];  // all of them on their way before the first store
#pragma unroll
          for (int r = 0; r < 32; ++r) y[r] = r < rows ? src[(int64_t)r * p.ldc] : T{};
#pragma unroll
          for (int r = 0; r < 32; ++r)
            *reinterpret_cast<T*>(sb + staged<32>(r, j / kPer) + j % kPer * sizeof(T)) = y[r];
        }
        __syncwarp();
      }
#pragma unroll
      for (int h = 0; h < kUnit; h += 32) {
        uint32_t w[32];
        if (has_k) {
          tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(q * 32) << 16) + acc * kTile + at + h, w);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) w[j] = 0u;
        }
        float v[32];
        grouped_values(p, w, bias, (at + h) / 32, v);
#pragma unroll
        for (int i = 0; i < 32 / kPer; ++i) {
          uint4* piece = reinterpret_cast<uint4*>(sb + staged<32>(lane, h / kPer + i));
          uint32_t o[4];
          uint4 old = make_uint4(0u, 0u, 0u, 0u);
          if (c != nullptr) old = *piece;
          const uint32_t cw[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) {
              const float y = v[i * 4 + k];
              o[k] = __float_as_uint(c != nullptr ? fmaf(p.beta, __uint_as_float(cw[k]), y) : y);
            } else {
              float y0 = v[i * 8 + 2 * k], y1 = v[i * 8 + 2 * k + 1];
              if (c != nullptr) {
                y0 = fmaf(p.beta, half_bits_to_float<BF16>((uint16_t)(cw[k] & 0xFFFFu)), y0);
                y1 = fmaf(p.beta, half_bits_to_float<BF16>((uint16_t)(cw[k] >> 16)), y1);
              }
              o[k] = pack2<BF16>(y0, y1);
            }
          }
          *piece = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      if (at + kUnit >= kTile) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tmem_empty[acc]);
      }
      __syncwarp();
      if (n > 0) copy_out<T, kAtOnce>(p, sb, d + at, rows, n, lane);
      __syncwarp();
    }
  }
}

// The walk of a gated block's epilogue: forward both products of 64 columns lie side
// by side in an accumulator, its gradient has two units of 64 columns.
template <bool BF16, typename P>
__device__ __forceinline__ void drain_gated(const P& p, const GroupTable& tb, int tiles, uint32_t tmem_base, uint8_t* sb,
                                            uint64_t* tmem_full, uint64_t* tmem_empty, const WaitCtx& wc) {
  const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const bool has_k = p.k_blocks > 0;
  int it = 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
    const GroupedTile x = grouped_tile<kTile, false>(p, tb, t);
    const int acc = it & 1;
    const int r0 = x.rb * kTile + q * 32;
    const int64_t row = (int64_t)x.lo + r0;
    const int rows = max(0, min(32, x.hi - x.lo - r0));
    const uint32_t at = tmem_base + ((uint32_t)(q * 32) << 16) + acc * kTile;
    const auto wait = [&] {
      const bool ok = mbar_wait_warp(&tmem_full[acc], (it >> 1) & 1, wc);
      tc_fence_after();
      return ok;
    };
    const auto release = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tmem_empty[acc]);
    };
    if constexpr (kIsGatedForward<P>) {
      const int col = x.cb * kGatedPlainCols;
      if (!wait()) break;
      gated_forward_unit<BF16>(p, at, at + kGatedPlainCols, has_k, row, rows, col, p.N - col, sb, lane, release);
    } else {
      const int col = x.cb * kTile;
      if (!gated_grad_unit<BF16>(p, at, has_k, row, rows, col, p.N - col, sb, lane, wait, [] {})) break;
      if (!gated_grad_unit<BF16>(p, at + 64, has_k, row, rows, col + 64, p.N - col - 64, sb, lane, [] { return true; }, release))
        break;
    }
  }
}

// F32: gradients in fp32.  P: GroupedParams, or those of a gated block.
template <bool BF16, bool WGRAD, bool F32, typename P = GroupedParams>
__global__ void __launch_bounds__(kThreads, 1) grouped_plain_kernel(const __grid_constant__ P p) {
  static_assert(!kIsGated<P> || !(WGRAD || F32), "gated blocks are forward products");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + kStages * kOperandBytes;
  uint8_t* staging = sB + kStages * kOperandBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStagingBytes);
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
      mbar_init(&full[s], kProducers);
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
  if (warp == kIssuer) {
    tmem_alloc(tmem_slot, F32 ? 512 : 256);
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

  if (warp < kProducers) {
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
        const int tid = threadIdx.x;
        if constexpr (WGRAD) {
          const int r0 = x.lo + kb * kBK;
          Outer pa, pb;
          pa.load(p.A, p.lda, r0, x.rb * kTile, x.hi, p.K, tid);
          pb.load(p.B, p.ldb, r0, n0, x.hi, p.N, tid);
          pa.store(a, tid);
          pb.store(b, tid);
        } else {
          const uint16_t* bg = static_cast<const uint16_t*>(p.B) + (int64_t)x.g * p.strideB;
          const int k0 = kb * kBK;
          Inner pa;
          pa.load(p.A, p.lda, x.lo + x.rb * kTile, k0, x.hi, p.K, tid);
          if constexpr (kIsGatedForward<P>) {
            // 64 columns of the one's weights, then the same of the other's
            const uint16_t* ug = static_cast<const uint16_t*>(p.U) + (int64_t)x.g * p.strideB;
            HalfTile pg, pu;
            const int outer = p.b_mn ? k0 : x.cb * kGatedPlainCols, inner = p.b_mn ? x.cb * kGatedPlainCols : k0;
            const int outer_ext = p.b_mn ? p.K : p.N, inner_ext = p.b_mn ? p.N : p.K;
            pg.load(bg, p.ldb, outer, inner, outer_ext, inner_ext, tid);
            pu.load(ug, p.ldb, outer, inner, outer_ext, inner_ext, tid);
            pa.store(a, tid);
            pg.store(b, tid);
            pu.store(b + kOperandBytes / 2, tid);
          } else if (p.b_mn) {
            Outer pb;
            pb.load(bg, p.ldb, k0, n0, p.K, p.N, tid);
            pa.store(a, tid);
            pb.store(b, tid);
          } else {
            Inner pb;
            pb.load(bg, p.ldb, n0, k0, p.N, p.K, tid);
            pa.store(a, tid);
            pb.store(b, tid);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[stage]);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == kIssuer) {
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
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const GroupedTile x = grouped_tile<kTile, WGRAD>(p, tb, t);
        const int nkb = WGRAD ? (x.hi - x.lo + kBK - 1) / kBK : p.k_blocks;
        const int per_acc = F32 ? kSumKBlocks : nkb;
        int kb0 = 0;
        do {  // an accumulator: the tile's, or a part of its reduction
          const int acc = it & 1, n = min(per_acc, nkb - kb0);
          if (!mbar_wait(&tmem_empty[acc], ((it >> 1) & 1) ^ 1u, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int kb = 0; kb < n; ++kb) {
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
          ++it;
          kb0 += n;
        } while (kb0 < nkb);
      }
      if (any) {
        mma_commit(drain_bar);
        drain_wait(drain_bar, 0, 100000000ull);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    using T = typename std::conditional<F32, float, uint16_t>::type;
    uint8_t* sb = staging + (warp - kProducers) * 4096;
    if constexpr (kIsGated<P>)
      drain_gated<BF16>(p, tb, tiles, tmem_base, sb, tmem_full, tmem_empty, wc);
    else
      drain_tiles<BF16, WGRAD, T>(p, tb, tiles, tmem_base, sb, tmem_full, tmem_empty, wc);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem_base, F32 ? 512 : 256);
  }
}

template <bool BF16, bool WGRAD, bool F32, typename P>
cudaError_t launch(const P& p, int ctas, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(grouped_plain_kernel<BF16, WGRAD, F32, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
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
  e = cudaLaunchKernelEx(&cfg, grouped_plain_kernel<BF16, WGRAD, F32, P>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_plain(bool bf16, bool wgrad, const GroupedParams& p, int ctas, cudaStream_t stream) {
  if (!wgrad) return bf16 ? launch<true, false, false>(p, ctas, stream) : launch<false, false, false>(p, ctas, stream);
  if (p.out_f32) return bf16 ? launch<true, true, true>(p, ctas, stream) : launch<false, true, true>(p, ctas, stream);
  return bf16 ? launch<true, true, false>(p, ctas, stream) : launch<false, true, false>(p, ctas, stream);
}

cudaError_t launch_gated_plain(bool bf16, const GatedForward& p, int ctas, cudaStream_t stream) {
  return bf16 ? launch<true, false, false>(p, ctas, stream) : launch<false, false, false>(p, ctas, stream);
}

cudaError_t launch_gated_plain(bool bf16, const GatedGrad& p, int ctas, cudaStream_t stream) {
  return bf16 ? launch<true, false, false>(p, ctas, stream) : launch<false, false, false>(p, ctas, stream);
}

}  // namespace ttc
