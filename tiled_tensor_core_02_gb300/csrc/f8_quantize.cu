// 8-bit floats with a fp32 scale for each block:
//   scale = max |x| / top,   q = round(x * (1 / scale)),
// top = 448 (e4m3) or 57344 (e5m2), the formats' largest finite values; the quotients
// and the product rounded to nearest in fp32, the last rounding to the nearest 8-bit
// float, ties to even, so the result is one defined set of bits.  |x| / scale is top at
// most up to a rounding, which the conversion takes back.  A block whose scale would be
// below the least normal number, 2^-126, counts as zeros (scale 0); one with a NaN or an
// infinity gets that as its scale and zeros, so that every product with it is NaN.
//
// Blocks are 128 elements of a row, or 128 x 128, of the matrix or of its transpose.
// A row's blocks need nothing of one another: half a warp takes a block of 16-bit
// values (16 bytes a lane), a warp one of 32-bit values, several on their way at once.
// Square blocks and transposed rows take a tile of 128 x 128 to a CTA, held in registers
// between the maxima and the rounding; transposed bytes pass through shared memory so
// that rows of 128 bytes leave.  A block's quotients are one lane's work, handed round: done
// by every lane they were a third of the instructions.
//
// Bound by HBM for rows: 8192 x 14336 bf16 56 us, 6.3 TB/s, fp32 90, 6.6; 16 x 4096 bf16 2.5.  Tiles wait
// for their maxima between loads and stores, with four of them on an SM (fp32: two): square
// blocks 56 us, fp32 139; transposed rows 66, fp32 114; transposed square blocks 59, fp32 125.  fp32 square
// blocks keep HBM 42 % busy where transposed rows have 55: twice the stores (4 bytes a lane) and a fifth
// more instructions at two tiles an SM.
// Rows off 16-byte boundaries, an element a load: 8192 x 14335 111 us, transposed 132.
#include <cuda_fp8.h>

#include "f8_blocks.cuh"
#include "gemm_kernel.cuh"

namespace ttc {

namespace {

template <int IN>
struct In;
template <>
struct In<kF8QuantF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float to_float(T v) { return __half2float(__ushort_as_half(v)); }
};
template <>
struct In<kF8QuantBF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float to_float(T v) { return __uint_as_float((uint32_t)v << 16); }
};
template <>
struct In<kF8QuantF32> {
  using T = float;
  static __device__ __forceinline__ float to_float(T v) { return v; }
};
template <int IN>
constexpr int kVec = 16 / (int)sizeof(typename In<IN>::T);  // elements of 16 bytes

// 16 bytes of the input as they are: kVec elements.
template <int IN>
struct Piece {
  uint32_t w[4];

  // `n` elements from src on (0 to kVec), zeros behind them; `vec`: src lies on a 16-byte
  // boundary wherever n is kVec.
  __device__ __forceinline__ void load(const typename In<IN>::T* src, int n, bool vec) {
    if (vec && n == kVec<IN>) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src));
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (IN == kF8QuantF32) {
          w[i] = i < n ? __float_as_uint(src[i]) : 0u;
        } else {
          w[i] = 2 * i < n ? src[2 * i] : 0u;
          if (2 * i + 1 < n) w[i] |= (uint32_t)src[2 * i + 1] << 16;
        }
      }
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (IN == kF8QuantF32)
      return __uint_as_float(w[e]);
    else
      return In<IN>::to_float((uint16_t)(e % 2 == 0 ? w[e / 2] & 0xFFFFu : w[e / 2] >> 16));
  }
};

// Magnitudes as unsigned integers: in order, infinity after every number and NaN behind.
// 16-bit ones two a word.
template <int IN>
__device__ __forceinline__ uint32_t mags(uint32_t w) {
  return w & (IN == kF8QuantF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
}
template <int IN>
__device__ __forceinline__ uint32_t max_mags(uint32_t a, uint32_t b) {
  if constexpr (IN == kF8QuantF32) return max(a, b);
  uint32_t v;
  asm("max.u16x2 %0, %1, %2;" : "=r"(v) : "r"(a), "r"(b));
  return v;
}
// The bits of the largest magnitude of a word as fp32, and of either of its columns (one of fp32).
template <int IN>
__device__ __forceinline__ uint32_t mag_of(uint32_t w, int column) {
  if constexpr (IN == kF8QuantF32) return w;
  return __float_as_uint(In<IN>::to_float((uint16_t)(column == 0 ? w & 0xFFFFu : w >> 16)));
}
template <int IN>
__device__ __forceinline__ uint32_t top_mag(uint32_t w) {
  if constexpr (IN == kF8QuantF32) return w;
  return mag_of<IN>(max(w & 0xFFFFu, w >> 16), 0);
}

struct BlockScale {
  float scale, inv;
};
template <bool E5M2>
__device__ __forceinline__ BlockScale block_scale(uint32_t m) {
  BlockScale r;
  r.scale = __fdiv_rn(__uint_as_float(m), E5M2 ? 57344.0f : 448.0f);
  if (m >= 0x7F800000u) {
    r.scale = __uint_as_float(m);
    r.inv = 0.0f;
  } else if (r.scale < 1.17549435e-38f) {
    r.scale = 0.0f;
    r.inv = 0.0f;
  } else {
    r.inv = __frcp_rn(r.scale);
  }
  return r;
}

// Two values to two bytes, the first in the low one.  What comes without an inverse (of a block
// of zeros, or with a NaN or an infinity) is no result: such a block's is 0.
template <bool E5M2>
__device__ __forceinline__ uint32_t to_f8x2(float a, float b, float inv) {
  const float2 v = __fmul2_rn(make_float2(a, b), make_float2(inv, inv));
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
}

// ------------------------------------------------------------------ rows
constexpr int kAtOnce = 4;  // vectors of a lane on their way

// A warp takes kAtOnce * 32 vectors of a row, whole blocks of 128; VEC: rows of x on
// 16-byte and of q on kVec-byte boundaries.
template <int IN, bool E5M2, bool VEC>
__global__ void __launch_bounds__(256) f8_rows_kernel(const F8QuantParams p, int parts, int64_t items) {
  constexpr int V = kVec<IN>, kLanes = kF8Block / V;  // lanes of a block
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * 8) {
    const int64_t row = parts == 1 ? it : it / parts;
    const int part = parts == 1 ? 0 : (int)(it - row * parts);
    const typename In<IN>::T* src = static_cast<const typename In<IN>::T*>(p.x) + row * p.ldx;
    const int c0 = part * (kAtOnce * 32 * V) + lane * V;
    Piece<IN> f[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int c = c0 + i * 32 * V;
      f[i].load(src + c, max(0, min(V, p.cols - c)), VEC);
    }
    uint32_t m[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      m[i] = mags<IN>(f[i].w[0]);
#pragma unroll
      for (int k = 1; k < 4; ++k) m[i] = max_mags<IN>(m[i], mags<IN>(f[i].w[k]));
      m[i] = top_mag<IN>(m[i]);
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) m[i] = max(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
    }
    // a lane a block: the quotients are the costly part
    const int mine = lane % kLanes % kAtOnce;
    uint32_t top = m[0];
#pragma unroll
    for (int i = 1; i < kAtOnce; ++i) top = mine == i ? m[i] : top;
    const BlockScale s = block_scale<E5M2>(top);
    const int block = (c0 + mine * 32 * V) / kF8Block;
    if (lane % kLanes < kAtOnce && block * kF8Block < p.cols) p.scale[row * p.lds + block] = s.scale;
    const bool empty = __any_sync(0xFFFFFFFFu, s.inv == 0.0f);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float inv = __shfl_sync(0xFFFFFFFFu, s.inv, lane / kLanes * kLanes + i);
      const int c = c0 + i * 32 * V, n = p.cols - c;
      uint32_t o[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) o[e] = to_f8x2<E5M2>(f[i][2 * e], f[i][2 * e + 1], inv);
      if (empty && inv == 0.0f) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) o[e] = 0u;
      }
      uint8_t* dst = p.q + row * p.ldq + c;
      if (VEC && n >= V) {
        if constexpr (V == 8)
          *reinterpret_cast<uint2*>(dst) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
        else
          *reinterpret_cast<uint32_t*>(dst) = o[0] | o[1] << 16;
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e < n) dst[e] = (uint8_t)(o[e / 2] >> (e % 2 * 8));
      }
    }
  }
}

// ------------------------------------------------------------------ tiles of 128 x 128
// A thread holds V columns of kRows consecutive rows: a warp reads whole rows of the
// tile, and a column's bytes of a thread are eight (or sixteen) in a row of the transpose.
template <int IN>
struct TileOf {
  static constexpr int V = kVec<IN>, kGroups = kF8Block / V;  // column groups
  static constexpr int kRows = kF8Block * kGroups / 256;
};

// Place of the 8-byte piece `piece` of the transpose's row `col` in shared memory: turned
// so that neither a warp's writes (V columns apart) nor its reads meet a bank twice.
__device__ __forceinline__ int turned(int col, int piece) { return col * 128 + ((piece ^ (col >> 3)) & 15) * 8; }

// SQUARE: one scale for the tile; else (TURN) one for each of its columns.
template <int IN, bool E5M2, bool SQUARE, bool TURN, bool VEC>
__global__ void __launch_bounds__(256, IN == kF8QuantF32 ? 2 : 4) f8_tiles_kernel(const F8QuantParams p, int tiles_x, int64_t tiles) {
  using TO = TileOf<IN>;
  constexpr int V = TO::V, R = TO::kRows;
  __shared__ __align__(16) uint8_t bytes[TURN ? kF8Block * 128 : 16];
  __shared__ uint32_t part[8][SQUARE ? 1 : 4 * TO::kGroups];
  __shared__ float inverse[SQUARE ? 1 : kF8Block];
  const int cg = threadIdx.x % TO::kGroups, rg = threadIdx.x / TO::kGroups, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t ty = t / tiles_x;
    const int tx = (int)(t - ty * tiles_x);
    const int row0 = (int)ty * kF8Block, col0 = tx * kF8Block;
    const int c = col0 + cg * V, nc = max(0, min(V, p.cols - c));
    const int r0 = row0 + rg * R;
    const typename In<IN>::T* src = static_cast<const typename In<IN>::T*>(p.x) + (int64_t)r0 * p.ldx + c;
    Piece<IN> f[R];
#pragma unroll
    for (int i = 0; i < R; ++i) f[i].load(src + (int64_t)i * p.ldx, r0 + i < p.rows ? nc : 0, VEC);
    float inv[SQUARE ? 1 : V];
    if constexpr (SQUARE) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) m = max_mags<IN>(m, mags<IN>(f[i].w[k]));
      m = __reduce_max_sync(0xFFFFFFFFu, top_mag<IN>(m));
      if (lane == 0) part[warp][0] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, part[i][0]);
      const BlockScale s = block_scale<E5M2>(m);
      inv[0] = s.inv;
      if (threadIdx.x == 0) p.scale[(TURN ? tx : ty) * p.lds + (TURN ? ty : (int64_t)tx)] = s.scale;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < R; ++i) m = max_mags<IN>(m, mags<IN>(f[i].w[k]));
        if constexpr (TO::kGroups == 16) m = max_mags<IN>(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
        if (lane < TO::kGroups) part[warp][cg * 4 + k] = m;
      }
      __syncthreads();
      // a thread a column: the quotients are the costly part
      if (threadIdx.x < kF8Block) {
        constexpr int kPer = V / 4;  // columns of a word
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_mags<IN>(m, part[i][threadIdx.x / kPer]);
        const BlockScale s = block_scale<E5M2>(mag_of<IN>(m, threadIdx.x % kPer));
        inverse[threadIdx.x] = s.inv;
        if (col0 + (int)threadIdx.x < p.cols) p.scale[(int64_t)(col0 + (int)threadIdx.x) * p.lds + ty] = s.scale;
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; ++e) inv[e] = inverse[cg * V + e];
    }
    if constexpr (!TURN) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (r0 + i >= p.rows) continue;
        uint32_t o[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) o[e] = inv[0] == 0.0f ? 0u : to_f8x2<E5M2>(f[i][2 * e], f[i][2 * e + 1], inv[0]);
        uint8_t* dst = p.q + (int64_t)(r0 + i) * p.ldq + c;
        if (VEC && nc == V) {
          if constexpr (V == 8)
            *reinterpret_cast<uint2*>(dst) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
          else
            *reinterpret_cast<uint32_t*>(dst) = o[0] | o[1] << 16;
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (e < nc) dst[e] = (uint8_t)(o[e / 2] >> (e % 2 * 8));
        }
      }
      __syncthreads();  // part is written again for the next tile
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float s = inv[SQUARE ? 0 : e];
#pragma unroll
        for (int i = 0; i < R; i += 8) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = s == 0.0f ? 0u : to_f8x2<E5M2>(f[i + 2 * k][e], f[i + 2 * k + 1][e], s);
          *reinterpret_cast<uint2*>(bytes + turned(cg * V + e, (rg * R + i) / 8)) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
        }
      }
      __syncthreads();
      // rows of the transpose: 16 lanes take one, 8 bytes each
      const int piece = threadIdx.x & 15, at = row0 + piece * 8, n = min(8, p.rows - at);
#pragma unroll
      for (int i = 0; i < kF8Block / 16; ++i) {
        const int col = i * 16 + (threadIdx.x >> 4);
        if (col0 + col >= p.cols || n <= 0) continue;
        const uint2 w = *reinterpret_cast<const uint2*>(bytes + turned(col, piece));
        uint8_t* dst = p.q + (int64_t)(col0 + col) * p.ldq + at;
        if (VEC && n == 8) {
          *reinterpret_cast<uint2*>(dst) = w;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < n) dst[e] = (uint8_t)((e < 4 ? w.x : w.y) >> (e % 4 * 8));
        }
      }
      __syncthreads();
    }
  }
}

template <typename K, typename... Args>
cudaError_t launch_one(K kernel, int64_t blocks, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int IN, bool E5M2>
cudaError_t launch_in(const F8QuantParams& p, bool square, bool turn, int sm_count, cudaStream_t stream) {
  constexpr int V = kVec<IN>;
  const int q_vec = turn ? 8 : V;  // bytes that are written at once
  const bool vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx % V == 0 && reinterpret_cast<uintptr_t>(p.q) % q_vec == 0 &&
                   p.ldq % q_vec == 0;
  if (!square && !turn) {
    const int parts = (p.cols + kAtOnce * 32 * V - 1) / (kAtOnce * 32 * V);
    const int64_t items = (int64_t)p.rows * parts, cap = (int64_t)sm_count * 64;
    int64_t blocks = (items + 7) / 8;
    if (blocks > cap) blocks = cap;
    return vec ? launch_one(f8_rows_kernel<IN, E5M2, true>, blocks, stream, p, parts, items)
               : launch_one(f8_rows_kernel<IN, E5M2, false>, blocks, stream, p, parts, items);
  }
  const int tiles_x = (p.cols + kF8Block - 1) / kF8Block;
  const int64_t tiles = (int64_t)((p.rows + kF8Block - 1) / kF8Block) * tiles_x, cap = (int64_t)sm_count * 16;
  const int64_t blocks = tiles < cap ? tiles : cap;
#define TTC_TILES(S, T)                                                                              \
  (vec ? launch_one(f8_tiles_kernel<IN, E5M2, S, T, true>, blocks, stream, p, tiles_x, tiles)        \
       : launch_one(f8_tiles_kernel<IN, E5M2, S, T, false>, blocks, stream, p, tiles_x, tiles))
  if (!square) return TTC_TILES(false, true);
  return turn ? TTC_TILES(true, true) : TTC_TILES(true, false);
#undef TTC_TILES
}

}  // namespace

cudaError_t launch_f8_quantize(const F8QuantParams& p, F8QuantIn in, bool e5m2, bool square, bool turn, int sm_count,
                               cudaStream_t stream) {
  switch (in) {
    case kF8QuantF16: return e5m2 ? launch_in<kF8QuantF16, true>(p, square, turn, sm_count, stream)
                                  : launch_in<kF8QuantF16, false>(p, square, turn, sm_count, stream);
    case kF8QuantBF16: return e5m2 ? launch_in<kF8QuantBF16, true>(p, square, turn, sm_count, stream)
                                   : launch_in<kF8QuantBF16, false>(p, square, turn, sm_count, stream);
    case kF8QuantF32: return e5m2 ? launch_in<kF8QuantF32, true>(p, square, turn, sm_count, stream)
                                  : launch_in<kF8QuantF32, false>(p, square, turn, sm_count, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ttc
