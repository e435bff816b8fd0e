// Symmetric int8 rows with a scale each:
//   scale_i = max_j |x_ij| / 127,   q_ij = round(x_ij * (1 / scale_i)),
// both quotients and the product rounded to nearest in fp32, the last
// rounding to the nearest integer with ties to even, so the result is one
// defined set of bits.  |x| <= 127 scale up to a rounding of 2^-23, so no
// integer beyond +-127 arises.  A row whose scale would be below the least
// normal number, 2^-126, counts as zeros (scale 0): its reciprocal would not
// be finite.  A row with a NaN or an infinity gets that as its scale and
// zeros as its integers, so every product with it is NaN rather than wrong.
//
// The row's maximum has to be known before its first integer, so a row is
// read whole into registers: by one warp up to 32 vectors of 16 bytes per
// lane's worth, else by a block of 256 threads; longer or unaligned rows are
// read twice, the second time from L2.  Bound by HBM: every input byte is read
// once, every int8 written once: 8192 x 14336 bf16 55 us, 6.4 TB/s; 8192 x 8192 fp32
// 49 us, 6.9 TB/s; 16 x 4096 1.7 us.  Rows read twice, an element a load: 8192 x 14335
// bf16 130 us, 2.7 TB/s; 8192 x 14336 fp32 158 us, 3.7 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gemm_kernel.cuh"
#include "quantize.cuh"

namespace ttc {

namespace {

template <int IN>
struct QuantElem;
template <>
struct QuantElem<kQuantF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float to_float(T v) { return __half2float(__ushort_as_half(v)); }
};
template <>
struct QuantElem<kQuantBF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float to_float(T v) { return __uint_as_float((uint32_t)v << 16); }
};
template <>
struct QuantElem<kQuantF32> {
  using T = float;
  static __device__ __forceinline__ float to_float(T v) { return v; }
};

// max of magnitudes that keeps a NaN: as unsigned integers, the bit patterns
// of non-negative floats are ordered, infinity after every number and NaN
// after infinity.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct RowScale {
  float scale, inv;
};
__device__ __forceinline__ RowScale row_scale(uint32_t m) {
  RowScale r;
  r.scale = __fdiv_rn(__uint_as_float(m), 127.0f);
  if (m >= 0x7F800000u) {
    r.scale = __uint_as_float(m);
    r.inv = 0.0f;
  } else if (r.scale < 1.17549435e-38f) {
    r.scale = 0.0f;
    r.inv = 0.0f;
  } else {
    r.inv = __fdiv_rn(1.0f, r.scale);
  }
  return r;
}

// inv == 0 (a zero or non-finite row) gives 0 for every x, NaN and infinity
// included: the conversion of a NaN to an integer is 0.
__device__ __forceinline__ int to_i8(float x, float inv) { return __float2int_rn(__fmul_rn(x, inv)); }

// one 16-byte vector of the row, as floats
template <int IN>
struct QuantVec {
  static constexpr int kElems = 16 / (int)sizeof(typename QuantElem<IN>::T);
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[kElems]) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (IN == kQuantF32) {
        f[i] = __uint_as_float(ws[i]);
      } else {
        f[2 * i] = QuantElem<IN>::to_float((uint16_t)(ws[i] & 0xFFFFu));
        f[2 * i + 1] = QuantElem<IN>::to_float((uint16_t)(ws[i] >> 16));
      }
    }
  }
};

template <int THREADS>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if constexpr (THREADS > 32) {
    __shared__ uint32_t part[THREADS / 32];
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) m = max(m, part[i]);
    __syncthreads();  // part is written again for the block's next row
  }
  return m;
}

// Rows of whole, aligned 16-byte vectors, held in registers between the two
// passes: THREADS threads take a row, VECS vectors each at most.
template <int IN, int THREADS, int VECS>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
  constexpr int kElems = QuantVec<IN>::kElems;
  constexpr int kRowsPerBlock = 256 / THREADS;
  const int lane = threadIdx.x % THREADS;
  const int nvec = p.cols / kElems;
  grid_dependency_wait();
  grid_dependents_launch();
  for (int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + threadIdx.x / THREADS; row < p.rows;
       row += (int64_t)gridDim.x * kRowsPerBlock) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const typename QuantElem<IN>::T*>(p.x) + row * p.ldx);
    uint4 w[VECS];
#pragma unroll
    for (int v = 0; v < VECS; ++v)
      w[v] = lane + v * THREADS < nvec ? __ldcs(src + lane + v * THREADS) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t m = 0u;
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      float f[kElems];
      QuantVec<IN>::unpack(w[v], f);
#pragma unroll
      for (int e = 0; e < kElems; ++e) m = max(m, mag(f[e]));
    }
    const RowScale rs = row_scale(group_max<THREADS>(m));
    if (lane == 0) p.scale[row] = rs.scale;
    int8_t* dst = p.q + row * p.ldq;
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      const int i = lane + v * THREADS;
      if (i < nvec) {
        float f[kElems];
        QuantVec<IN>::unpack(w[v], f);
        uint32_t o[kElems / 4];
#pragma unroll
        for (int e = 0; e < kElems; e += 4) {
          const uint32_t lo = __byte_perm((uint32_t)to_i8(f[e], rs.inv), (uint32_t)to_i8(f[e + 1], rs.inv), 0x0040);
          const uint32_t hi = __byte_perm((uint32_t)to_i8(f[e + 2], rs.inv), (uint32_t)to_i8(f[e + 3], rs.inv), 0x0040);
          o[e / 4] = __byte_perm(lo, hi, 0x5410);
        }
        if constexpr (kElems == 8)
          *reinterpret_cast<uint2*>(dst + (int64_t)i * 8) = make_uint2(o[0], o[1]);
        else
          *reinterpret_cast<uint32_t*>(dst + (int64_t)i * 4) = o[0];
      }
    }
  }
}

// Rows of any length and alignment: element loads, two passes.
template <int IN>
__global__ void __launch_bounds__(256) quantize_any_kernel(const QuantParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const typename QuantElem<IN>::T* src = static_cast<const typename QuantElem<IN>::T*>(p.x) + row * p.ldx;
    uint32_t m = 0u;
#pragma unroll 8
    for (int c = threadIdx.x; c < p.cols; c += 256) m = max(m, mag(QuantElem<IN>::to_float(src[c])));
    const RowScale rs = row_scale(group_max<256>(m));
    if (threadIdx.x == 0) p.scale[row] = rs.scale;
    int8_t* dst = p.q + row * p.ldq;
#pragma unroll 8
    for (int c = threadIdx.x; c < p.cols; c += 256) dst[c] = (int8_t)to_i8(QuantElem<IN>::to_float(src[c]), rs.inv);
  }
}

template <typename K>
cudaError_t launch_one(K kernel, const QuantParams& p, int64_t blocks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int IN>
cudaError_t launch_in(const QuantParams& p, int sm_count, cudaStream_t stream) {
  constexpr int kElems = QuantVec<IN>::kElems;
  constexpr int esize = 16 / kElems;
  const bool vec = p.cols % kElems == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && (p.ldx * esize) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(p.q) % kElems == 0 && p.ldq % kElems == 0;
  const int nvec = p.cols / kElems;
  const int64_t cap = (int64_t)sm_count * 32;
  if (vec && nvec <= 32 * 4) {  // a warp per row
    int64_t blocks = ((int64_t)p.rows + 7) / 8;
    if (blocks > cap) blocks = cap;
    return nvec <= 32 ? launch_one(quantize_rows_kernel<IN, 32, 1>, p, blocks, stream)
                      : launch_one(quantize_rows_kernel<IN, 32, 4>, p, blocks, stream);
  }
  const int64_t blocks = p.rows < cap ? p.rows : cap;
  if (vec && nvec <= 256 * 2) return launch_one(quantize_rows_kernel<IN, 256, 2>, p, blocks, stream);
  if (vec && nvec <= 256 * 4) return launch_one(quantize_rows_kernel<IN, 256, 4>, p, blocks, stream);
  if (vec && nvec <= 256 * 8) return launch_one(quantize_rows_kernel<IN, 256, 8>, p, blocks, stream);
  return launch_one(quantize_any_kernel<IN>, p, blocks, stream);
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantParams& p, QuantIn in, int sm_count, cudaStream_t stream) {
  switch (in) {
    case kQuantF16: return launch_in<kQuantF16>(p, sm_count, stream);
    case kQuantBF16: return launch_in<kQuantBF16>(p, sm_count, stream);
    case kQuantF32: return launch_in<kQuantF32>(p, sm_count, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ttc
