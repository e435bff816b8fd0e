// Grouped products of few tokens with large weights:
//   D[i, f] = act(alpha sum_k A[i, k] W_g[f, k] + bias_g[f]).
//
// With few tokens the cost is the stream of the weights, so these take the MMA's
// 128-row side and the tokens its columns (16 to 64), the transpose of the
// other kernels' tiles: a stage of the pipeline is almost all weights, and the
// MMA's time, 39 to 48 clocks for 16 to 64 columns, stays below the stream's.
//
// A tile is `tile_cols` output columns (8 to 128, chosen by the host so that the
// tiles fill whole waves of SMs: 8192 columns are 147 tiles of 56, not 64 of 128)
// by one block of a group's tokens.  With fewer than 128 columns the MMA's last
// rows are whatever lies behind them in shared memory, and are not stored.  No
// split of K and no partial sums between CTAs.
//
// One thread loads with TMA: a stage is 128 of K, as deep a ring of stages as
// fits shared memory (what hides HBM's latency is the bytes on the way: 100 to
// 200 KB an SM); one warp issues tcgen05.mma into two accumulators; four warps
// drain them, a thread an output column, a register a token.  Of a block's tokens
// only those in the group are loaded, in boxes of at most 32: the others would
// come from L2 as often as there are tiles.
//
// Bound by HBM: 16 rows of 8 groups, 14336 x 4096 bf16 (6 groups with rows, 705
// MB): 105 us, 6.7 TB/s; the CTA-pair kernel takes 128.
#include <atomic>

#include "grouped_common.cuh"

namespace ttc {

namespace {

constexpr int kStageK = 128;
constexpr int kMaxStages = 16;
constexpr int kBarBytes = 512;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kThreads = 256;  // producer, MMA issuer, two spare warps, four of the epilogue

__host__ __device__ constexpr int stage_bytes_of(int rows) { return rows * kStageK * 2; }

// Shared memory around the ring: alignment, what a 128-row operand reads behind
// a narrower tile, barriers, group table.
int fixed_bytes(int groups) { return 1024 + 16384 + kBarBytes + 2 * (groups + 2) * 4; }

// All groups' blocks of tokens for one block of columns, then the next: blocks
// that share a tile of weights follow one another (it comes from HBM once), and
// large groups, whose other blocks find their weights in L2, are spread among the
// small ones that keep HBM busy.
template <int BT>
__device__ __forceinline__ GroupedTile few_tile(const GroupedParams& p, const GroupTable& tb, int blocks, int t) {
  GroupedTile x;
  x.cb = t / blocks;
  const int r = t - x.cb * blocks;
  int first;
  x.g = group_of_tile<BT>(p, tb, r, first);
  x.rb = r - first;
  group_rows(p, tb, x.g, x.lo, x.hi);
  return x;
}

template <int BT, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) few_tokens_kernel(const __grid_constant__ GroupedParams p) {
  constexpr int kTokenBytes = stage_bytes_of(BT);
  constexpr int kBox = few_tokens_box(BT);
  constexpr int kTmemCols = 2 * BT;  // two accumulators: 32 to 128 columns
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int w_bytes = stage_bytes_of(p.tile_cols);
  const int stage_bytes = w_bytes + kTokenBytes;
  const int S = p.stages;
  uint8_t* ring = smem;  // [stage][weights, tokens]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + S * stage_bytes + 16384);
  uint64_t* full = bars;
  uint64_t* empty = bars + kMaxStages;
  uint64_t* tmem_full = bars + 2 * kMaxStages;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* stall_bar = tmem_empty + 2;
  uint64_t* drain_bar = stall_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  static_assert((2 * kMaxStages + 6) * 8 + 4 <= kBarBytes, "barrier area");
  GroupTable tb;
  tb.offs = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);
  tb.start = tb.offs + p.groups + 2;
  tb.step = 1;
  tb.per = 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{p.err, p.timeout_ns};
  if (warp == 0) {
    if (lane < S) {
      mbar_init(&full[lane], 1);
      mbar_init(&empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&tmem_full[lane], 1);
      mbar_init(&tmem_empty[lane], 4);
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
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();
  build_group_table<BT>(p, tb);
  const int blocks = table_tiles(p, tb);  // of tokens, of all groups
  const int tiles = blocks * p.col_blocks;
  const int k_stages = (p.K + kStageK - 1) / kStageK;
  const int w_blk = p.tile_cols * kBK * 2;  // weights with K contiguous: from one k-block of a stage to the next

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t keep = policy_evict_last();
      const uint64_t pol_w = p.b_stream ? policy_evict_first() : keep;
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const GroupedTile x = few_tile<BT>(p, tb, blocks, t);
        const int f0 = x.cb * p.tile_cols, t0 = x.lo + x.rb * BT;
        const int z = p.strideB != 0 ? x.g : 0;
        const int boxes = (min(BT, x.hi - t0) + kBox - 1) / kBox;  // of tokens
        for (int ks = 0; ks < k_stages; ++ks) {
          const int k0 = ks * kStageK;
          const bool two = p.K - k0 > kBK;  // both k-blocks of the stage
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          uint8_t* w = ring + stage * stage_bytes;
          uint8_t* a = w + w_bytes;
          // weights with their rows contiguous come in boxes of 128 of K whatever K is
          mbar_arrive_expect_tx(&full[stage],
                                (two || p.b_mn ? w_bytes : w_bytes / 2) + (two ? 2 : 1) * boxes * (kBox * kBK * 2));
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (p.b_mn) {
            tma_load_3d(w, &p.tmB, f0, k0, z, &full[stage], pol_w);
            if (p.tile_cols > 64) tma_load_3d(w + 64 * kStageK * 2, &p.tmB, f0 + 64, k0, z, &full[stage], pol_w);
          } else {
            tma_load_3d(w, &p.tmB, k0, f0, z, &full[stage], pol_w);
            if (two) tma_load_3d(w + w_blk, &p.tmB, k0 + kBK, f0, z, &full[stage], pol_w);
          }
          for (int b = 0; b < boxes; ++b) {
            uint8_t* at = a + b * (kBox * kBK * 2);
            tma_load_3d(at, &p.tmA, k0, t0 + b * kBox, 0, &full[stage], keep);
            if (two) tma_load_3d(at + kTokenBytes / 2, &p.tmA, k0 + kBK, t0 + b * kBox, 0, &full[stage], keep);
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      drain_ring(full, S, armed, armed_parity);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t lead = elect_lead();
    const bool w_mn = p.b_mn;
    const uint32_t idesc = idesc_f16(BF16, w_mn, false, 128, BT);
    const uint64_t w0 = smem_desc_sw128(smem_u32(ring), w_mn ? 64 * kStageK * 2 : 16u, 1024);
    const uint64_t a0 = smem_desc_sw128(smem_u32(ring + w_bytes), 16u, 1024);
    const uint32_t w_step = (w_mn ? 2048u : 32u) >> 4;
    const uint32_t w_kb = (uint32_t)(w_mn ? kBK * 128 : w_blk) >> 4;
    constexpr uint32_t kTokenKb = BT * 128 >> 4;
    const int whole = p.K / kStageK;  // stages without a tail of K
    bool ok = true, any = false;
    if (p.inject_stall) ok = mbar_wait_warp(stall_bar, 0, wc);  // nothing arrives here
    int stage = 0, it = 0;
    uint32_t phase = 0;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++it) {
      const int acc = it & 1;
      if (!mbar_wait_warp(&tmem_empty[acc], ((it >> 1) & 1) ^ 1u, wc)) break;
      tc_fence_after();
      const uint32_t d = tmem_base + acc * BT;
      for (int ks = 0; ks < k_stages; ++ks) {
        if (!mbar_wait_warp(&full[stage], phase, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t wd = w0 + (uint32_t)(stage * stage_bytes >> 4);
        const uint64_t ad = a0 + (uint32_t)(stage * stage_bytes >> 4);
        const uint32_t add = ks != 0;
        if (ks < whole) {  // no condition between the MMAs: each would cost as much as one
          const uint32_t w_lo = (uint32_t)wd, w_hi = (uint32_t)(wd >> 32), a_lo = (uint32_t)ad, a_hi = (uint32_t)(ad >> 32);
          mma_f16_lead_lo(lead, d, w_lo, w_hi, a_lo, a_hi, idesc, add);
#pragma unroll
          for (int k = 1; k < kStageK / kUmmaK; ++k)
            mma_f16_lead_lo(lead, d, w_lo + (k >> 2) * w_kb + (k & 3) * w_step, w_hi, a_lo + (k >> 2) * kTokenKb + (k & 3) * 2u,
                            a_hi, idesc, 1u);
        } else {
          const int steps = (p.K - ks * kStageK + kUmmaK - 1) / kUmmaK;
#pragma unroll 1
          for (int k = 0; k < steps; ++k)
            mma_f16_lead(lead, d, wd + (k >> 2) * w_kb + (k & 3) * w_step, ad + (k >> 2) * kTokenKb + (k & 3) * 2u, idesc,
                         add | (k != 0 ? 1u : 0u));
        }
        any = true;
        mma_commit_lead(lead, &empty[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      mma_commit_lead(lead, &tmem_full[acc]);
    }
    if (any) {
      mma_commit_lead(lead, drain_bar);
      drain_wait(drain_bar, 0, 100000000ull);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const int col = q * 32 + lane;  // of the tile
    const uint32_t tmem_mine = tmem_base + ((uint32_t)(q * 32) << 16);
    int it = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++it) {
      const GroupedTile x = few_tile<BT>(p, tb, blocks, t);
      const int f = x.cb * p.tile_cols + col;
      const bool f_ok = col < p.tile_cols && f < p.N;
      const int row0 = x.lo + x.rb * BT, tokens = min(BT, x.hi - row0);
      const float bias = p.bias != nullptr && f_ok ? __ldg(p.bias + (int64_t)x.g * p.stride_bias + f) : 0.0f;
      uint16_t* d = static_cast<uint16_t*>(p.D) + (int64_t)row0 * p.ldd + f;
      const int acc = it & 1;
      if (!mbar_wait(&tmem_full[acc], (it >> 1) & 1, wc)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < BT; c += 16) {
        uint32_t w[16];
        tmem_ld_32x32b_x16<0>(tmem_mine + acc * BT + c, w);
        tmem_ld_wait();
        if (c + 16 == BT) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tmem_empty[acc]);
        }
        if (f_ok) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c + j < tokens) {
              float v = p.alpha * __uint_as_float(w[j]);
              if (p.bias != nullptr) v += bias;
              d[(int64_t)(c + j) * p.ldd] = (uint16_t)(pack2<BF16>(act_value(p.act, v), 0.0f) & 0xFFFFu);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <int BT, bool BF16>
cudaError_t launch(const GroupedParams& p, int ctas, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(few_tokens_kernel<BT, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = fixed_bytes(p.groups) + p.stages * stage_bytes_of(p.tile_cols + BT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, few_tokens_kernel<BT, BF16>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int few_tokens_stages(int tokens, int tile_cols, int groups) {
  const int n = (kSmemLimit - fixed_bytes(groups)) / stage_bytes_of(tile_cols + tokens);
  return n > kMaxStages ? kMaxStages : n;
}

cudaError_t launch_few_tokens(bool bf16, int tokens, const GroupedParams& p, int ctas, cudaStream_t stream) {
  switch (tokens) {
    case 16: return bf16 ? launch<16, true>(p, ctas, stream) : launch<16, false>(p, ctas, stream);
    case 32: return bf16 ? launch<32, true>(p, ctas, stream) : launch<32, false>(p, ctas, stream);
    case 64: return bf16 ? launch<64, true>(p, ctas, stream) : launch<64, false>(p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ttc
