// int8 products for some hundred tokens on the tensor cores:
//   D[i, f] = act(scaleA[i] scaleB[f] sum_k A[i, k] B[f, k] + bias[f]).
//
// There is no int8 tcgen05.mma on this device (and the warp-level one does 262
// multiply-adds a clock and SM: 113 us for 64 x 8192 x 8192), so the operands are
// widened to fp16 on their way through the SM, exactly.  The weights B take the
// MMA's 128-row side and are widened straight into tensor memory, from where the
// MMA reads that operand: through shared memory their fp16 copy would be written
// once and read once more at twice the size, and with the raw bytes' two passes
// shared memory would set the pace (0.57 us for a stage of 56 rows).  The tokens,
// the MMA's columns, are widened into shared memory.
//
// A CTA takes `tile_cols` channels by one block of tokens by its share of K, and
// ends; the CTAs of a cluster share a tile's K.  The host picks both so that the
// CTAs fill one wave of SMs.  One thread brings stages of 128 of K with TMA, as
// many as fit; sixteen warps in four groups widen stages in turn, warp q of a
// group the 32 rows of tensor memory it may write, a row a thread; one warp issues
// the MMAs.
//
// Exactness: products of int8 values and sums of 1024 of them are exact in fp32.
// Each 1024 of a CTA's K has an accumulator of its own (256 columns of tensor
// memory hold them all), so nothing is drained on the way; at the end the same
// sixteen warps add them up as int32, the cluster's CTAs exchange their sums
// through shared memory, and one conversion, two scales, the bias and the
// activation follow.
//
// Bound by HBM's share of an SM or the widening of a stage (0.3 to 0.4 us), whichever
// is more, and at these sizes by what surrounds the stream: 24 x 8192 x 8192 17.0 us,
// 10 of them at 6.7 TB/s, 1.7 before the first stage is there, 4 for the sums and
// their exchange; 256 x 4096 x 4096 17.6 us.
#include <atomic>

#include "gemm_kernel.cuh"
#include "i8_rows.cuh"

namespace ttc {

namespace {

constexpr int kWarp0 = 4;       // the first widening warp; 0 producer, 1 MMA issuer
constexpr int kWidenWarps = 16;
constexpr int kThreads = 32 * (kWarp0 + kWidenWarps);
// Groups of widening warps, which take stages in turn.  A group waits for its slot
// before it waits for its stage's bytes: the slot is free once the MMAs of
// kGroups stages before are done, and with them, in order, of all earlier ones.
// In a ring of at least kGroups stages the place's previous use is then over, and
// cannot be taken for the one the group waits for.
constexpr int kGroups = 4, kGroupWarps = kWidenWarps / kGroups;
constexpr int kMaxStages = 16;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kAccStages = 1024 / kI8TokenStage;  // stages of an accumulator

constexpr int kAlign = 1024;
int ring_stage_bytes(int block, int tile_cols) { return (block + tile_cols) * kI8TokenStage; }
int fixed_bytes(int block) { return kAlign + 1024 + kGroups * block * kI8TokenStage * 2; }
int total_bytes(int block, int tile_cols, int stages) {
  const int n = fixed_bytes(block) + stages * ring_stage_bytes(block, tile_cols);
  const int sums = kAlign + 1024 + block * 128 * 4;  // the exchange reuses the slots and the ring
  return n > sums ? n : sums;
}

template <int BT, int OUT>
__global__ void __launch_bounds__(kThreads, 1) i8_tokens_kernel(const __grid_constant__ I8TokensParams q) {
  constexpr int kSlotBytes = BT * kI8TokenStage * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);  // in front: the exchange at the end leaves them alone
  uint8_t* slots = smem + 1024;                        // [group][k-block][token][64 fp16]
  uint8_t* ring = slots + kGroups * kSlotBytes;        // [stage][weights, tokens]
  const I8ScaledParams& p = q.p;
  const int w_bytes = q.tile_cols * kI8TokenStage, stage_bytes = w_bytes + BT * kI8TokenStage, S = q.stages;
  uint64_t* full = bars;
  uint64_t* empty = bars + kMaxStages;
  uint64_t* wide_full = bars + 2 * kMaxStages;
  uint64_t* wide_empty = wide_full + kGroups;
  uint64_t* done_bar = wide_empty + kGroups;
  uint64_t* stall_bar = done_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stall_bar + 1);
  static_assert((2 * kMaxStages + 2 * kGroups + 2) * 8 + 4 <= 1024, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{q.err, q.timeout_ns};
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const int f0 = tile * q.tile_cols, token0 = blockIdx.y * BT;
  const int s_lo = min(p.chunks, rank * p.chunks_per_cta), n_stages = min(p.chunks, s_lo + p.chunks_per_cta) - s_lo;

  if (warp == 0) {
    if (lane < S) {
      mbar_init(&full[lane], 1);
      mbar_init(&empty[lane], kGroupWarps);  // the widening group's warps
    }
    if (lane < kGroups) {
      mbar_init(&wide_full[lane], kGroupWarps);
      mbar_init(&wide_empty[lane], 1);
    }
    if (lane == 0) {
      mbar_init(done_bar, 1);
      mbar_init(stall_bar, 1);
      prefetch_tmap(&q.tmA);
      prefetch_tmap(&q.tmB);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);  // accumulators in columns 0 .. 255, widened weights from 256 on
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  uint32_t armed = 0, armed_parity = 0;  // stages that the producer has armed
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t keep = policy_evict_last();
      const uint64_t pol_w = gridDim.y == 1 ? policy_evict_first() : keep;
      int stage = 0;
      uint32_t phase = 0;
      for (int n = 0; n < n_stages; ++n) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) break;
        uint8_t* w = ring + stage * stage_bytes;
        mbar_arrive_expect_tx(&full[stage], stage_bytes);
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        tma_load_3d(w, &q.tmB, (s_lo + n) * kI8TokenStage, f0, 0, &full[stage], pol_w);
        tma_load_3d(w + w_bytes, &q.tmA, (s_lo + n) * kI8TokenStage, token0, 0, &full[stage], keep);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t lead = elect_lead();
    const uint32_t idesc = idesc_f16(false, false, false, 128, BT);
    const uint64_t x0 = smem_desc_sw128(smem_u32(slots), 16u, 1024);
    constexpr uint32_t kTokenKb = BT * 128 >> 4;
    const int whole = p.K / kI8TokenStage - s_lo;  // stages without a tail of K
    bool ok = true;
    if (q.inject_stall) ok = mbar_wait_warp(stall_bar, 0, wc);  // nothing arrives here
    int g = 0;
    uint32_t phase = 0;
    for (int n = 0; ok && n < n_stages; ++n) {
      if (!mbar_wait_warp(&wide_full[g], phase, wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem_base + (n / kAccStages) * BT;
      const uint32_t w = tmem_base + kI8TokenCols + g * (kI8TokenStage / 2);
      const uint64_t x = x0 + (uint32_t)(g * kSlotBytes >> 4);
      const uint32_t add = n % kAccStages != 0;
      if (n < whole) {
        // without a condition between them an MMA takes about 25 clocks to issue, with one 57
        const uint32_t x_lo = (uint32_t)x, x_hi = (uint32_t)(x >> 32);
        mma_f16_ta_lead_lo(lead, d, w, x_lo, x_hi, idesc, add);
#pragma unroll
        for (int k = 1; k < kI8TokenStage / kUmmaK; ++k)
          mma_f16_ta_lead_lo(lead, d, w + 8 * k, x_lo + (k >> 2) * kTokenKb + (k & 3) * 2u, x_hi, idesc, 1u);
      } else {
        const int steps = (p.K - (s_lo + n) * kI8TokenStage + kUmmaK - 1) / kUmmaK;
#pragma unroll 1
        for (int k = 0; k < steps; ++k)
          mma_f16_ta_lead(lead, d, w + 8 * k, x + (k >> 2) * kTokenKb + (k & 3) * 2u, idesc, add | (k != 0 ? 1u : 0u));
      }
      mma_commit_lead(lead, &wide_empty[g]);
      if (++g == kGroups) {
        g = 0;
        phase ^= 1u;
      }
    }
    // every MMA issued is done when this completes, whether or not all were
    mma_commit_lead(lead, done_bar);
    drain_wait(done_bar, 0, 100000000ull);
  } else if (warp >= kWarp0) {
    // ---------------------------------------------------------------- widening
    const int group = (warp - kWarp0) / kGroupWarps, quarter = warp & 3;
    const int tid = (int)threadIdx.x % (kGroupWarps * 32);
    const int row = quarter * 32 + lane;  // of the weights' tile, and of tensor memory
    uint8_t* slot = slots + group * kSlotBytes;
    const uint32_t tmem_w =
        tmem_base + ((uint32_t)(quarter * 32) << 16) + kI8TokenCols + group * (kI8TokenStage / 2);
    // where this thread's bytes lie: of its row (the piece's place turned by the
    // row), and of its pieces of the tokens, sixteen bytes each
    constexpr int kPieces = BT * 8 / (kGroupWarps * 32);
    const bool in = row < q.tile_cols, any = quarter * 32 < q.tile_cols;
    const int x_row = tid >> 3, x_c = tid & 7;  // its first piece; the others are kRows rows further each
    constexpr int kRows = kGroupWarps * 4;
    const uint32_t x_src = x_row * 128 + ((x_c ^ (x_row & 7)) << 4);
    const uint32_t x_dst = (x_c >> 2) * (BT * 128) + x_row * 128;
    const uint32_t x_lo = (((x_c & 3) * 2) ^ (x_row & 7)) << 4, x_hi = (((x_c & 3) * 2 + 1) ^ (x_row & 7)) << 4;
    static_assert(kRows % 8 == 0, "the turn is the same for all of a thread's pieces");
    uint32_t wide_phase = 0, phase = 0;
    int stage = group;
    for (int n = group; n < n_stages; n += kGroups) {
      if (!mbar_wait(&wide_empty[group], wide_phase ^ 1u, wc)) break;  // first: see kGroups
      if (!mbar_wait(&full[stage], phase, wc)) break;
      tc_fence_after();
      const uint8_t* w8 = ring + stage * stage_bytes;
      const uint8_t* x8 = w8 + w_bytes + x_src;
      // all loads before the first store: they do not move above one
      uint4 xv[kPieces], wv[8];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) xv[i] = *reinterpret_cast<const uint4*>(x8 + i * (kRows * 128));
      if (any) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          wv[c] = in ? *reinterpret_cast<const uint4*>(w8 + row * 128 + ((c ^ (row & 7)) << 4)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            widen4(wv[h * 4 + c].x, w[8 * c], w[8 * c + 1]);
            widen4(wv[h * 4 + c].y, w[8 * c + 2], w[8 * c + 3]);
            widen4(wv[h * 4 + c].z, w[8 * c + 4], w[8 * c + 5]);
            widen4(wv[h * 4 + c].w, w[8 * c + 6], w[8 * c + 7]);
          }
          tmem_st_32x32b_x32(tmem_w + h * 32, w);
        }
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        uint32_t h[8];
        widen4(xv[i].x, h[0], h[1]);
        widen4(xv[i].y, h[2], h[3]);
        widen4(xv[i].z, h[4], h[5]);
        widen4(xv[i].w, h[6], h[7]);
        uint8_t* dst = slot + x_dst + i * (kRows * 128);
        *reinterpret_cast<uint4*>(dst + x_lo) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(dst + x_hi) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&wide_full[group]);
        mbar_arrive(&empty[stage]);
      }
      wide_phase ^= 1u;
      stage += kGroups;
      if (stage >= S) {
        stage -= S;
        phase ^= 1u;
      }
    }
  }
  // a thread's channel from here on, and what its results take: asked for before the wait
  const int col = threadIdx.x & 127, f = f0 + col;
  const bool f_ok = col < q.tile_cols && f < p.N;
  const float scale_b = f_ok ? __ldg(p.scaleB + f) : 0.0f, bias = f_ok && p.bias != nullptr ? __ldg(p.bias + f) : 0.0f;
  if (warp == 0) {  // after the loads above, which would come late behind it
    drain_ring_lanes(full, armed, armed_parity);
  }
  // every MMA is done (the issuer waited) and every byte is there and read
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // ------------------------------------------------------------------ sums and result
  // four sets of four warps; set g takes the tokens from g * kCols on, a thread a channel
  constexpr int kCols = BT / 4;
  static_assert(kCols == 8 || kCols == 16, "blocks of 32 or 64 tokens");
  int32_t* red = reinterpret_cast<int32_t*>(slots);  // [token][128 channels]
  const int tokens = min(BT, p.M - token0);
  auto result = [&](int32_t s, int token, float scale_a) {
    float v = __int2float_rn(s) * scale_a * scale_b;
    if (p.bias != nullptr) v += bias;
    v = act_value(p.act, v);
    const int64_t o = (int64_t)token * p.ldd + f;
    if constexpr (OUT == kI8ResultF32)
      static_cast<float*>(p.D)[o] = v;
    else
      static_cast<uint16_t*>(p.D)[o] = (uint16_t)(pack2<OUT == kI8ResultBF16>(v, 0.0f) & 0xFFFFu);
  };
  if (warp >= kWarp0) {
    const int group = (warp - kWarp0) >> 2, quarter = warp & 3;
    const int c0 = group * kCols;
    if (quarter * 32 < q.tile_cols) {
      const int parts = (n_stages + kAccStages - 1) / kAccStages;
      int32_t sum[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) sum[j] = 0;
      for (int a = 0; a < parts; ++a) {
        uint32_t w[kCols];
        const uint32_t from = tmem_base + ((uint32_t)(quarter * 32) << 16) + a * BT + c0;
        if constexpr (kCols == 16)
          tmem_ld_32x32b_x16<0>(from, w);
        else
          tmem_ld_32x32b_x8(from, w);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kCols; ++j) sum[j] += __float2int_rn(__uint_as_float(w[j]));
      }
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int i = c0 + j;
        if (p.split > 1)
          red[i * 128 + col] = sum[j];
        else if (i < tokens && f_ok)
          result(sum[j], token0 + i, __ldg(p.scaleA + token0 + i));
      }
    }
  }
  if (p.split > 1) {
    cluster_sync();
    // each CTA of the cluster adds up and stores its share
    static_assert(kThreads % 128 == 0, "a thread keeps its channel");
    for (int e = rank * kThreads + threadIdx.x; f_ok && e < tokens * 128; e += p.split * kThreads) {
      const float scale_a = __ldg(p.scaleA + token0 + (e >> 7));
      const uint32_t at = smem_u32(red + e);
      int32_t s = 0;
      for (int r0 = 0; r0 < p.split; r0 += 4) {  // four loads on the way
        uint32_t v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = 0;
          if (r0 + r < p.split)
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v[r]) : "r"(mapa_shared(at, (uint32_t)(r0 + r))) : "memory");
        }
        s += (int32_t)(v[0] + v[1] + v[2] + v[3]);
      }
      result(s, token0 + (e >> 7), scale_a);
    }
    cluster_sync();  // no CTA leaves while another may read its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int BT, int OUT>
cudaError_t launch(const I8TokensParams& q, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(i8_tokens_kernel<BT, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(q.p.split * ((q.p.N + q.tile_cols - 1) / q.tile_cols)), (unsigned)((q.p.M + BT - 1) / BT), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = total_bytes(BT, q.tile_cols, q.stages);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)q.p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  add_pdl_attribute(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, i8_tokens_kernel<BT, OUT>, q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int BT>
cudaError_t launch_block(const I8TokensParams& q, I8ResultType out, cudaStream_t stream) {
  switch (out) {
    case kI8ResultF16: return launch<BT, kI8ResultF16>(q, stream);
    case kI8ResultBF16: return launch<BT, kI8ResultBF16>(q, stream);
    case kI8ResultF32: return launch<BT, kI8ResultF32>(q, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int i8_tokens_stages(int block, int tile_cols) {
  const int n = (kSmemLimit - fixed_bytes(block)) / ring_stage_bytes(block, tile_cols);
  return n > kMaxStages ? kMaxStages : n < kGroups ? 0 : n;
}

// One CTA an SM, whatever its block: all of tensor memory.
int i8_tokens_clusters(int split) {
  static std::atomic<int> known[64][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || split < 1 || split > 8) return 0;
  int n = known[dev][split].load();
  if (n > 0) return n;
  if (cudaFuncSetAttribute(i8_tokens_kernel<64, kI8ResultBF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) !=
      cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)split, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemLimit;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, i8_tokens_kernel<64, kI8ResultBF16>, &cfg) != cudaSuccess) return 0;
  known[dev][split].store(n);
  return n;
}

cudaError_t launch_i8_tokens(const I8TokensParams& q, int block, I8ResultType out, cudaStream_t stream) {
  switch (block) {
    case 32: return launch_block<32>(q, out, stream);
    case 64: return launch_block<64>(q, out, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ttc
