// Block-scaled fp8 products of few tokens with large weights, the transpose of the other
// kernels' tiles as in few_tokens.cu: the weights on the MMA's 128-row side, the tokens on
// its columns (16 to 64), `tile_cols` output columns (8 to 128) by one block of a group's
// tokens a tile.
//
// A block of 128 k has sums of its own: a stage's two go side by side into one of four
// accumulators in tensor memory, and the epilogue warps, a thread an output column of 16
// tokens, add it to their sums in registers times its weights' scale and the token's.  The
// tokens' scales come into shared memory once a tile and 32 blocks of K, the weights' a stage
// ahead.  (An accumulator for each block: 4099 rows of 64 groups, 1536 x 2048 65.6 us against
// 58.4; a second set of epilogue warps for every other one changed nothing.)
//
// Up to 32 tokens bound by HBM on wide layers, behind a few microseconds of start: 1 x 14336 x 4096
// 12.3 us, 16 x 8192 x 8192 16.0; on narrower ones by a tile's stages, which follow one another, 0.31 us
// each: 1 x 4096 x K 4.4, 6.0, 8.7 and 13.8 us for K = 1024, 2048, 4096 and 8192, the weights' bytes
// 0.6 to 4.9 (with one thread that loads 10.1 for K = 4096).  With 64 tokens a tile by shared memory, which gives the MMAs 24 KB a block of K, takes as much from TMA and hands 64
// tokens' scales to every warp: 0.31 us a block, 64 x 8192 x 8192 21.1 us.
#include <atomic>

#include "f8_blocks.cuh"
#include "grouped_common.cuh"

namespace ttc {

namespace {

constexpr int kKPS = 2;  // blocks of K of a stage
constexpr int kStageK = kKPS * kF8Block;
constexpr int kMaxStages = 16;
constexpr int kAccs = 4;  // accumulators, each with a place for either block of a stage
constexpr int kBarBytes = 512;
constexpr int kSmemLimit = 227 * 1024;
// Producer, MMA issuer, two spare warps; of the epilogue four for each kPart tokens: with all
// of a block's 64 in four warps an accumulator took these longer than HBM its weights.
constexpr int kPart = 16;
template <int BT>
constexpr int kEpiThreads = 128 * (BT / kPart);
template <int BT>
constexpr int kThreads = 128 + kEpiThreads<BT>;
constexpr int kScaleK = 32;    // blocks of K whose token scales are in shared memory at a time

__host__ __device__ constexpr int stage_bytes_of(int rows) { return rows * kStageK; }

// Shared memory around the ring: alignment, what a 128-row operand reads behind a narrower
// tile, the tokens' scales, barriers, group table.
int fixed_bytes(int tokens, int groups) { return 1024 + 16384 + 2 * kScaleK * tokens * 4 + kBarBytes + 2 * (groups + 2) * 4; }

// All groups' blocks of tokens for one block of columns, then the next (see few_tokens.cu).
template <int BT>
__device__ __forceinline__ GroupedTile few_tile(const F8Params& p, const GroupTable& tb, int blocks, int t) {
  GroupedTile x;
  x.cb = t / blocks;
  const int r = t - x.cb * blocks;
  int first;
  x.g = group_of_tile<BT>(p, tb, r, first);
  x.rb = r - first;
  group_rows(p, tb, x.g, x.lo, x.hi);
  return x;
}

template <int THREADS>
__device__ __forceinline__ void barrier_of_epilogue() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
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

// Two tokens at a time: half the instructions, 2 % of 64 x 8192 x 8192.
__device__ __forceinline__ void add_pair(float* sum, const uint32_t* w, float2 token_scale, float scale) {
  const float2 v = __ffma2_rn(__fmul2_rn(token_scale, make_float2(scale, scale)),
                              make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), make_float2(sum[0], sum[1]));
  sum[0] = v.x;
  sum[1] = v.y;
}

// Blocks of K whose weights' scales a thread reads at a time.  A column's own scales are
// 4 bytes of a line for each thread and block: four at a time took 500 rows of 16 groups,
// 4096 x 4096, from 82 us to 58, where one for 128 columns, the same for all threads, lost 2 %
// by the registers.
template <bool BY_COLUMN>
constexpr int kFetch = BY_COLUMN ? 4 : kKPS;

template <int BT, int OUT, bool BY_COLUMN>
__global__ void __launch_bounds__(kThreads<BT>, 1) f8_tokens_kernel(const __grid_constant__ F8Params p) {
  constexpr int kTokenBytes = stage_bytes_of(BT);
  constexpr int kBox = few_tokens_box(BT);
  constexpr int kTmemCols = kAccs * kKPS * BT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int w_bytes = stage_bytes_of(p.tile_cols);
  const int stage_bytes = w_bytes + kTokenBytes;
  const int S = p.stages;
  uint8_t* ring = smem;  // [stage][weights, tokens]
  float* token_scales = reinterpret_cast<float*>(ring + S * stage_bytes + 16384);  // [chunk of K, alternately][block][token]
  uint64_t* bars = reinterpret_cast<uint64_t*>(token_scales + 2 * kScaleK * BT);
  uint64_t* full = bars;
  uint64_t* empty = bars + kMaxStages;
  uint64_t* tmem_full = bars + 2 * kMaxStages;
  uint64_t* tmem_empty = tmem_full + kAccs;
  uint64_t* stall_bar = tmem_empty + kAccs;
  uint64_t* drain_bar = stall_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  static_assert(kScaleK % kKPS == 0 && kTmemCols <= 512, "chunks of scales hold whole stages");
  static_assert((2 * kMaxStages + 2 * kAccs + 2) * 8 + 4 <= kBarBytes, "barrier area");
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
    if (lane < kAccs) {
      mbar_init(&tmem_full[lane], 1);
      mbar_init(&tmem_empty[lane], kEpiThreads<BT> / 32);
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
  const int k_stages = (p.k_blocks + kKPS - 1) / kKPS;
  const int w_blk = p.tile_cols * kF8Block;  // from one block of K of a stage to the next

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    const uint32_t lead = elect_lead();  // a converged warp, one lane of which loads
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
        const bool two = p.k_blocks - ks * kKPS > 1;  // both blocks of the stage
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, wc)) {
          ok = false;
          break;
        }
        uint8_t* w = ring + stage * stage_bytes;
        uint8_t* a = w + w_bytes;
        if (lead) mbar_arrive_expect_tx(full + stage, (two ? 2 : 1) * (w_blk + boxes * (kBox * kF8Block)));
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        tma_load_3d_lead(lead, w, &p.tmB, k0, f0, z, &full[stage], pol_w);
        if (two) tma_load_3d_lead(lead, w + w_blk, &p.tmB, k0 + kF8Block, f0, z, &full[stage], pol_w);
        for (int b = 0; b < boxes; ++b) {
          uint8_t* at = a + b * (kBox * kF8Block);
          tma_load_3d_lead(lead, at, &p.tmA, k0, t0 + b * kBox, 0, &full[stage], keep);
          if (two) tma_load_3d_lead(lead, at + kTokenBytes / 2, &p.tmA, k0 + kF8Block, t0 + b * kBox, 0, &full[stage], keep);
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    drain_ring_lanes(full, armed, armed_parity);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t lead = elect_lead();
    const uint32_t idesc = idesc_f8(p.b_e5m2 != 0, p.a_e5m2 != 0, 128, BT);  // the weights are the MMA's A
    const uint64_t w0 = smem_desc_sw128(smem_u32(ring), 16u, 1024);
    const uint64_t a0 = smem_desc_sw128(smem_u32(ring + w_bytes), 16u, 1024);
    const uint32_t w_hi = (uint32_t)(w0 >> 32), a_hi = (uint32_t)(a0 >> 32);
    const uint32_t w_kb = (uint32_t)w_blk >> 4;
    constexpr uint32_t kTokenKb = BT * kF8Block >> 4;
    bool ok = true, any = false;
    if (p.inject_stall) ok = mbar_wait_warp(stall_bar, 0, wc);  // nothing arrives here
    int stage = 0;
    uint32_t it = 0, phase = 0;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      for (int ks = 0; ok && ks < k_stages; ++ks) {
        if (!mbar_wait_warp(&full[stage], phase, wc)) {
          ok = false;
          break;
        }
        const uint32_t w_lo = (uint32_t)w0 + (uint32_t)(stage * stage_bytes >> 4);
        const uint32_t a_lo = (uint32_t)a0 + (uint32_t)(stage * stage_bytes >> 4);
        const uint32_t acc = it & (kAccs - 1);
        if (!mbar_wait_warp(&tmem_empty[acc], ((it / kAccs) & 1) ^ 1u, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * (kKPS * BT);
#pragma unroll
        for (int k = 0; k < kF8Block / 32; ++k) mma_f8_lead(lead, d, w_lo + k * 2, w_hi, a_lo + k * 2, a_hi, idesc, k != 0);
        if (p.k_blocks - ks * kKPS > 1) {
#pragma unroll
          for (int k = 0; k < kF8Block / 32; ++k)
            mma_f8_lead(lead, d + BT, w_lo + w_kb + k * 2, w_hi, a_lo + kTokenKb + k * 2, a_hi, idesc, k != 0);
        }
        any = true;
        ++it;
        mma_commit_lead(lead, &tmem_full[acc]);
        mma_commit_lead(lead, &empty[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (any) {
      mma_commit_lead(lead, drain_bar);
      drain_wait(drain_bar, 0, 100000000ull);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, tid = threadIdx.x - 128;
    const int col = q * 32 + lane;  // of the tile
    const int j0 = tid / 128 * kPart;  // this thread's first token
    const uint32_t tmem_mine = tmem_base + ((uint32_t)(q * 32) << 16) + j0;
    uint32_t it = 0;
    int buffer = 0;
    bool ok = true;  // after an error the walk goes on without waits: its barriers take all warps
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const GroupedTile x = few_tile<BT>(p, tb, blocks, t);
      const int f = x.cb * p.tile_cols + col;
      const bool f_ok = col < p.tile_cols && f < p.N;
      const int row0 = x.lo + x.rb * BT, tokens = min(BT, x.hi - row0);
      const float* sb = p.scale_b + (int64_t)x.g * p.stride_sb + (int64_t)((f_ok ? f : 0) >> p.b_shift) * p.lds_b;
      float sums[kPart];
#pragma unroll
      for (int j = 0; j < kPart; ++j) sums[j] = 0.0f;
      for (int kb0 = 0; kb0 < p.k_blocks; kb0 += kScaleK) {
        const int n = min(kScaleK, p.k_blocks - kb0);
        // eight threads a token: rows of scales are read in whole pieces
        float* ts = token_scales + buffer * kScaleK * BT;
        {
          const int token = tid >> 3;
          const float* sa = p.scale_a + (int64_t)(row0 + token) * p.lds_a + kb0;
#pragma unroll
          for (int k = 0; k < kScaleK / 8; ++k) {
            const int kb = (tid & 7) + k * 8;
            ts[kb * BT + token] = token < tokens && kb < n ? __ldg(sa + kb) : 0.0f;
          }
        }
        barrier_of_epilogue<kEpiThreads<BT>>();
        buffer ^= 1;
        ts += j0;
        // the weights' scales, a stage's or, of a column's own, two stages' ahead
        float next[kFetch<BY_COLUMN>], now[kFetch<BY_COLUMN>];
        const auto fetch = [&](int i) {
          const float* at = sb + kb0 + i;
          if constexpr (BY_COLUMN) {
            if (p.sb_vec && f_ok && i + 4 <= n) {
              const float4 v = __ldg(reinterpret_cast<const float4*>(at));
              next[0] = v.x;
              next[1] = v.y;
              next[2] = v.z;
              next[3] = v.w;
              return;
            }
          }
#pragma unroll
          for (int k = 0; k < kFetch<BY_COLUMN>; ++k) next[k] = f_ok && i + k < n ? __ldg(at + k) : 0.0f;
        };
        fetch(0);
        for (int i = 0; i < n; i += kKPS, ++it, ts += kKPS * BT) {
          const int in_fetch = i % kFetch<BY_COLUMN>;
          if (in_fetch == 0) {
#pragma unroll
            for (int k = 0; k < kFetch<BY_COLUMN>; ++k) now[k] = next[k];
            fetch(i + kFetch<BY_COLUMN>);
          }
          const float scale[kKPS] = {in_fetch == 0 ? now[0] : now[kFetch<BY_COLUMN> - 2],
                                     in_fetch == 0 ? now[1] : now[kFetch<BY_COLUMN> - 1]};
          const uint32_t acc = it & (kAccs - 1);
          if (ok) ok = mbar_wait_warp(&tmem_full[acc], (it / kAccs) & 1, wc);
          if (!ok) continue;
          tc_fence_after();
          uint32_t w[kKPS][16];
#pragma unroll
          for (int k = 0; k < kKPS; ++k) tmem_ld_32x32b_x16<0>(tmem_mine + acc * (kKPS * BT) + k * BT, w[k]);
          tmem_ld_wait_for(w[0]);
          tmem_ld_wait_for(w[1]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tmem_empty[acc]);
#pragma unroll
          for (int k = 0; k < kKPS; ++k) {
            if (i + k >= n) break;  // what lies there is of an earlier block
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 s = *reinterpret_cast<const float4*>(ts + k * BT + j);
              add_pair(sums + j, w[k] + j, make_float2(s.x, s.y), scale[k]);
              add_pair(sums + j + 2, w[k] + j + 2, make_float2(s.z, s.w), scale[k]);
            }
          }
        }
      }
      if (!ok || !f_ok) continue;
      const float bias = p.bias != nullptr ? __ldg(p.bias + (int64_t)x.g * p.stride_bias + f) : 0.0f;
#pragma unroll
      for (int j = 0; j < kPart; ++j) {
        if (j0 + j >= tokens) break;
        const int64_t row = row0 + j0 + j;
        float v = sums[j];
        if (p.C != nullptr) v += load_result<OUT>(p.C, row * p.ldc + f);
        if (p.bias != nullptr) v += bias;
        store_result<OUT>(p.D, row * p.ldd + f, act_value(p.act, v));
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

template <int BT, int OUT, bool BY_COLUMN>
cudaError_t launch(const F8Params& p, int ctas, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(f8_tokens_kernel<BT, OUT, BY_COLUMN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads<BT>, 1, 1);
  cfg.dynamicSmemBytes = fixed_bytes(BT, p.groups) + p.stages * stage_bytes_of(p.tile_cols + BT);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, f8_tokens_kernel<BT, OUT, BY_COLUMN>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int BT>
cudaError_t launch_out(const F8Params& p, F8Result out, int ctas, cudaStream_t stream) {
  const bool by_column = p.b_shift == 0;
  switch (out) {
    case kF8ResultF16: return by_column ? launch<BT, kF8ResultF16, true>(p, ctas, stream) : launch<BT, kF8ResultF16, false>(p, ctas, stream);
    case kF8ResultBF16: return by_column ? launch<BT, kF8ResultBF16, true>(p, ctas, stream) : launch<BT, kF8ResultBF16, false>(p, ctas, stream);
    case kF8ResultF32: return by_column ? launch<BT, kF8ResultF32, true>(p, ctas, stream) : launch<BT, kF8ResultF32, false>(p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int f8_tokens_stages(int tokens, int tile_cols, int groups) {
  const int n = (kSmemLimit - fixed_bytes(tokens, groups)) / stage_bytes_of(tile_cols + tokens);
  return n > kMaxStages ? kMaxStages : n;
}

cudaError_t launch_f8_tokens(const F8Params& p, F8Result out, int tokens, int ctas, cudaStream_t stream) {
  switch (tokens) {
    case 16: return launch_out<16>(p, out, ctas, stream);
    case 32: return launch_out<32>(p, out, ctas, stream);
    case 64: return launch_out<64>(p, out, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ttc
