// int8 products for few tokens:
//   D[i, j] = act(scaleA[i] scaleB[j] sum_k A[i, k] B[j, k] + bias[j]).
//
// With few tokens the work is the stream of the weights B, one byte per 2 M
// operations, so the weights go straight from HBM into registers, sixteen
// bytes a lane, and are widened there to fp16 (exactly: an int8 fits in the
// eleven bits of its significand).  The tensor cores then take sixteen output
// channels by sixteen k of them against eight tokens at a time
// (mma.m16n8k16).  A sum may take its terms in any order, so the sixteen
// bytes of a lane serve four such products as they lie: lane (g, t) of a warp
// holds bytes 16 t .. 16 t + 15 of a 64-wide stretch of rows g and g + 8, the
// product s takes bytes 4 s .. 4 s + 3 of each, and the tokens' fragment is
// read at the same k.  The tokens of a chunk of K are widened once into shared
// memory, rows 16 bytes off a multiple of 128 so that eight lanes of one load
// meet no bank twice.
//
// Exactness: products of int8 values and their sums below 2^24 are exact in
// fp32; after 1024 of K at most 2^24 can have been reached, so the sums move
// to int32 there.  The CTAs of a cluster share the K of their output channels
// and add their int32 sums through distributed shared memory: the order of an
// integer sum does not matter.  Then one conversion, two scales, the bias.
//
// Bound by the stream of the weights and, at these sizes, by the launch and its
// first bytes: 1 x 14336 x 4096 13.9 us, 4.2 TB/s (a plain read of as many bytes
// takes 12.5).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_kernel.cuh"
#include "i8_rows.cuh"

namespace ttc {

namespace {

constexpr int kThreads = 256;
constexpr int kPitch = kI8RowsChunk * 2 + 16;  // bytes of a widened token row in shared memory
constexpr int kDrainChunks = 1024 / kI8RowsChunk;
constexpr int kAhead = 2;  // chunks of weights that L2 is asked for ahead of the next one

// m16n8k16: A sixteen rows by sixteen k, B eight columns, fp32 sums
__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bytes k .. k + 15 of a row of K (k < K); those past its end are whatever
// lies in their 16-byte block, or 0.  Only aligned blocks that hold a byte of
// the row are read.
__device__ __forceinline__ uint4 row16(const int8_t* row, int k, int K, bool aligned) {
  if (aligned) return __ldcs(reinterpret_cast<const uint4*>(row + k));
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
  const uint32_t ph = (uint32_t)(at & 15);
  const uint4* blk = reinterpret_cast<const uint4*>(at - ph);
  const uint4 a = __ldg(blk);
  uint4 b = make_uint4(0u, 0u, 0u, 0u);
  if (ph != 0 && k + 16 - (int)ph < K) b = __ldg(blk + 1);
  uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const bool s8 = ph & 8, s4 = ph & 4;
#pragma unroll
  for (int i = 0; i < 6; ++i) x[i] = s8 ? x[i + 2] : x[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) x[i] = s4 ? x[i + 1] : x[i];
  const uint32_t bits = 8 * (ph & 3);
  return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                    __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
}

__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int n) {  // the first n bytes of a word
  return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u);
}

template <int NT, int OUT>
__global__ void __launch_bounds__(kThreads, 2) i8_rows_kernel(const I8ScaledParams p) {
  constexpr int kTokens = 8 * NT;
  constexpr int kXVecs = kTokens * (kI8RowsChunk / 16);  // 16-byte vectors of a chunk's tokens
  constexpr int kXIters = (kXVecs + kThreads - 1) / kThreads;
  constexpr int kXBytes = kTokens * kPitch;
  constexpr int kRedBytes = kTokens * kI8RowsFeatures * 4;
  __shared__ __align__(16) uint8_t smem[2 * kXBytes > kRedBytes ? 2 * kXBytes : kRedBytes];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = p.split;
  const int rank = blockIdx.x % split;  // of the cluster
  const int block = blockIdx.x / split;  // of output channels
  const int token0 = (blockIdx.y + blockIdx.z * gridDim.y) * kTokens;
  if (token0 >= p.M) return;  // the whole cluster
  const int c_lo = rank * p.chunks_per_cta, c_hi = min(p.chunks, c_lo + p.chunks_per_cta);
  const int feature0 = block * kI8RowsFeatures + warp * 16;
  // rows past the last channel repeat it; their sums are not stored
  const int8_t* w0 = p.B + (int64_t)min(feature0 + g, p.N - 1) * p.ldb;
  const int8_t* w1 = p.B + (int64_t)min(feature0 + g + 8, p.N - 1) * p.ldb;

  float acc[NT][4];
  int32_t sum[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[n][i] = 0.0f;
      sum[n][i] = 0;
    }

  uint4 w[4][2];  // four 64-wide stretches of the chunk, rows g and g + 8
  uint4 x[kXIters];
  auto load_w = [&](int c, int j) {
    const int k = c * kI8RowsChunk + j * 64 + t * 16;
    const bool in = c < c_hi && k < p.K;
    w[j][0] = in ? row16(w0, k, p.K, p.b_vec != 0) : make_uint4(0u, 0u, 0u, 0u);
    w[j][1] = in ? row16(w1, k, p.K, p.b_vec != 0) : make_uint4(0u, 0u, 0u, 0u);
  };
  // two lines of each of the warp's sixteen rows, one a lane
  const int8_t* ahead = p.B + (int64_t)min(feature0 + (lane >> 1), p.N - 1) * p.ldb + (lane & 1) * 128;
  auto prefetch_w = [&](int c) {
    if (c < c_hi && c * kI8RowsChunk + (lane & 1) * 128 < p.K) prefetch_l2_line(ahead + c * kI8RowsChunk);
  };
  auto load_x = [&](int c) {
#pragma unroll
    for (int i = 0; i < kXIters; ++i) {
      const int v = threadIdx.x + i * kThreads;
      const int token = token0 + v / (kI8RowsChunk / 16);
      const int k = c * kI8RowsChunk + (v % (kI8RowsChunk / 16)) * 16;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (v < kXVecs && token < p.M && c < c_hi && k < p.K) {
        x[i] = row16(p.A + (int64_t)token * p.lda, k, p.K, p.a_vec != 0);
        // zeros past K: what lies there of the weights then does not count
        const int n = p.K - k;
        x[i] = make_uint4(keep_bytes(x[i].x, n), keep_bytes(x[i].y, n - 4), keep_bytes(x[i].z, n - 8),
                          keep_bytes(x[i].w, n - 12));
      }
    }
  };
  auto store_x = [&](uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < kXIters; ++i) {
      const int v = threadIdx.x + i * kThreads;
      if (v < kXVecs) {
        uint32_t h[8];
        widen4(x[i].x, h[0], h[1]);
        widen4(x[i].y, h[2], h[3]);
        widen4(x[i].z, h[4], h[5]);
        widen4(x[i].w, h[6], h[7]);
        uint4* d = reinterpret_cast<uint4*>(buf + (v / (kI8RowsChunk / 16)) * kPitch + (v % (kI8RowsChunk / 16)) * 32);
        d[0] = make_uint4(h[0], h[1], h[2], h[3]);
        d[1] = make_uint4(h[4], h[5], h[6], h[7]);
      }
    }
  };
  auto drain = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[n][i] += __float2int_rn(acc[n][i]);
        acc[n][i] = 0.0f;
      }
  };

  grid_dependency_wait();
  grid_dependents_launch();
#pragma unroll
  for (int j = 0; j < 4; ++j) load_w(c_lo, j);
#pragma unroll
  for (int c = 1; c <= kAhead; ++c) prefetch_w(c_lo + c);
  load_x(c_lo);
  store_x(smem);
  __syncthreads();
  int buf = 0, until_drain = kDrainChunks;
  for (int c = c_lo; c < c_hi; ++c) {
    load_x(c + 1);
    prefetch_w(c + 1 + kAhead);
    const uint8_t* xb = smem + buf * kXBytes + g * kPitch + t * 32;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t r0[4] = {w[j][0].x, w[j][0].y, w[j][0].z, w[j][0].w};
      const uint32_t r1[4] = {w[j][1].x, w[j][1].y, w[j][1].z, w[j][1].w};
      uint32_t a[4][4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        widen4(r0[s], a[s][0], a[s][2]);
        widen4(r1[s], a[s][1], a[s][3]);
      }
      load_w(c + 1, j);  // the next chunk's, in flight while this one is worked on
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b0 = *reinterpret_cast<const uint4*>(xb + n * 8 * kPitch + j * 128);
        const uint4 b1 = *reinterpret_cast<const uint4*>(xb + n * 8 * kPitch + j * 128 + 16);
        mma_m16n8k16(acc[n], a[0][0], a[0][1], a[0][2], a[0][3], b0.x, b0.y);
        mma_m16n8k16(acc[n], a[1][0], a[1][1], a[1][2], a[1][3], b0.z, b0.w);
        mma_m16n8k16(acc[n], a[2][0], a[2][1], a[2][2], a[2][3], b1.x, b1.y);
        mma_m16n8k16(acc[n], a[3][0], a[3][1], a[3][2], a[3][3], b1.z, b1.w);
      }
    }
    if (--until_drain == 0) {
      drain();
      until_drain = kDrainChunks;
    }
    buf ^= 1;
    store_x(smem + buf * kXBytes);
    __syncthreads();
  }
  drain();

  // sums of this CTA's K into shared memory, tokens by channels
  int32_t* red = reinterpret_cast<int32_t*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      red[(n * 8 + 2 * t + (i & 1)) * kI8RowsFeatures + warp * 16 + g + (i >> 1) * 8] = sum[n][i];
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  // each CTA of the cluster adds up and stores its share of the tokens' channels
  const int tokens = min(kTokens, p.M - token0);
  for (int e = rank * kThreads + threadIdx.x; e < tokens * kI8RowsFeatures; e += split * kThreads) {
    const int i = e / kI8RowsFeatures, j = e % kI8RowsFeatures;
    const int col = block * kI8RowsFeatures + j;
    if (col >= p.N) continue;
    int32_t s = red[e];
    if (split > 1) {
      const uint32_t at = smem_u32(red + e);
      s = 0;
      for (int r = 0; r < split; ++r) {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(at, (uint32_t)r)) : "memory");
        s += (int32_t)v;
      }
    }
    const int row = token0 + i;
    float v = __int2float_rn(s) * __ldg(p.scaleA + row) * __ldg(p.scaleB + col);
    if (p.bias != nullptr) v += __ldg(p.bias + col);
    v = act_value(p.act, v);
    const int64_t o = (int64_t)row * p.ldd + col;
    if constexpr (OUT == kI8ResultF32)
      static_cast<float*>(p.D)[o] = v;
    else
      static_cast<uint16_t*>(p.D)[o] = (uint16_t)(pack2<OUT == kI8ResultBF16>(v, 0.0f) & 0xFFFFu);
  }
  if (split > 1) cluster_sync();  // no CTA leaves while another may read its sums
}

template <int NT, int OUT>
cudaError_t launch(const I8ScaledParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const unsigned blocks = (unsigned)((p.N + kI8RowsFeatures - 1) / kI8RowsFeatures);
  const unsigned tokens = (unsigned)((p.M + 8 * NT - 1) / (8 * NT));
  const unsigned planes = (tokens + 32767u) / 32768u;
  cfg.gridDim = dim3((unsigned)p.split * blocks, (tokens + planes - 1) / planes, planes);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  add_pdl_attribute(cfg, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, i8_rows_kernel<NT, OUT>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int OUT>
cudaError_t launch_out(const I8ScaledParams& p, cudaStream_t stream) {
  if (p.M <= 8) return launch<1, OUT>(p, stream);
  if (p.M <= 16) return launch<2, OUT>(p, stream);
  return launch<4, OUT>(p, stream);
}

}  // namespace

cudaError_t launch_i8_rows(const I8ScaledParams& p, I8ResultType out, cudaStream_t stream) {
  switch (out) {
    case kI8ResultF16: return launch_out<kI8ResultF16>(p, stream);
    case kI8ResultBF16: return launch_out<kI8ResultBF16>(p, stream);
    case kI8ResultF32: return launch_out<kI8ResultF32>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ttc
