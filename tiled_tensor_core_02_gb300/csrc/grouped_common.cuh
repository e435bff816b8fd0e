// Device side of the grouped products: the table of groups and tiles that
// every CTA builds from the device's offsets, and the values of the epilogue.
#pragma once
#include "gemm_kernel.cuh"
#include "grouped.cuh"

namespace ttc {

// The group table of a CTA in shared memory.  offs[g] is the first row of group
// g, held to [0, M] (offs[groups] ends the last one); null where shared memory
// has no room for it and the device's offsets are read instead.  start[i] is
// the first tile of group i * step, its last entry the number of tiles; null in
// the weights' gradient, where every group has as many tiles as another.  A
// block of a group's rows counts as `per` tiles.
struct GroupTable {
  int* offs;
  int* start;
  int step;
  int per;
};

__device__ __forceinline__ int offset_of(const GroupedParams& p, const GroupTable& tb, int g) {
  return tb.offs != nullptr ? tb.offs[g] : min(max(__ldg(p.offsets + g), 0), p.M);
}

__device__ __forceinline__ void group_rows(const GroupedParams& p, const GroupTable& tb, int g, int& lo, int& hi) {
  lo = offset_of(p, tb, g);
  hi = max(lo, offset_of(p, tb, g + 1));
}

template <int ROWS>
__device__ __forceinline__ int group_tiles(const GroupedParams& p, const GroupTable& tb, int g) {
  int lo, hi;
  group_rows(p, tb, g, lo, hi);
  return (hi - lo + ROWS - 1) / ROWS * tb.per;
}

// Fills the table; all threads of the CTA.  ROWS: rows of a tile.
template <int ROWS>
__device__ __forceinline__ void build_group_table(const GroupedParams& p, const GroupTable& tb) {
  if (tb.offs != nullptr) {
    for (int i = threadIdx.x; i <= p.groups; i += blockDim.x)
      tb.offs[i] = p.offsets != nullptr ? min(max(__ldg(p.offsets + i), 0), p.M) : i * p.M;
    __syncthreads();
  }
  if (tb.start == nullptr) return;
  if (threadIdx.x < 32) {
    const int entries = (p.groups + tb.step - 1) / tb.step;
    int carry = 0;
    for (int i0 = 0; i0 < entries; i0 += 32) {
      const int i = i0 + (int)threadIdx.x;
      int n = 0;
      for (int g = i * tb.step; g < min((i + 1) * tb.step, p.groups); ++g) n += group_tiles<ROWS>(p, tb, g);
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if ((int)threadIdx.x >= o) sum += v;
      }
      if (i < entries) tb.start[i] = carry + sum - n;
      carry += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (threadIdx.x == 0) tb.start[entries] = carry;
  }
  __syncthreads();
}

__device__ __forceinline__ int table_tiles(const GroupedParams& p, const GroupTable& tb) {
  return tb.start[(p.groups + tb.step - 1) / tb.step];
}

// The group of tile t, which has tiles, and its first tile.
template <int ROWS>
__device__ __forceinline__ int group_of_tile(const GroupedParams& p, const GroupTable& tb, int t, int& first) {
  int lo = 0, hi = (p.groups + tb.step - 1) / tb.step - 1;  // the first i with start[i + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tb.start[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  first = tb.start[lo];
  if (tb.step == 1) return lo;
  int g = lo * tb.step;
  const int last = min(g + tb.step, p.groups) - 1;
  for (; g < last; ++g) {
    const int n = group_tiles<ROWS>(p, tb, g);
    if (first + n > t) break;
    first += n;
  }
  return g;
}

struct GroupedTile {
  int g;         // group
  int lo, hi;    // its rows
  int rb, cb;    // block of D's rows (forward: counted from the group's first row) and of its columns
};

// Tiles of a group walk `group_rows` row blocks of one column block before the
// next column block, so that CTAs at work together share panels of A and B.
template <int ROWS, bool WGRAD>
__device__ __forceinline__ GroupedTile grouped_tile(const GroupedParams& p, const GroupTable& tb, int t) {
  GroupedTile x;
  int first, rows;
  if constexpr (WGRAD) {
    const int per = p.row_blocks * p.col_blocks;
    x.g = t / per;
    first = x.g * per;
    group_rows(p, tb, x.g, x.lo, x.hi);
    rows = p.row_blocks;
  } else {
    x.g = group_of_tile<ROWS>(p, tb, t, first);
    group_rows(p, tb, x.g, x.lo, x.hi);
    rows = (x.hi - x.lo + ROWS - 1) / ROWS;
  }
  int r = t - first;
  const int band = p.group_rows * p.col_blocks;
  const int b = r / band;
  const int above = b * p.group_rows;
  const int size = min(rows - above, p.group_rows);
  r -= b * band;
  x.rb = above + r % size;
  x.cb = r / size;
  return x;
}

// 32 values of a row (columns col0 .. col0 + 31, `n` of them inside D) from
// their accumulator: alpha, C, bias, activation.
template <bool BF16>
__device__ __forceinline__ void grouped_values(const GroupedParams& p, const uint32_t (&r)[32], const void* c_row,
                                               const float* bias, int n, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = p.alpha * __uint_as_float(r[j]);
  if (c_row != nullptr) {
    if (p.out_f32) {
      const float* c = static_cast<const float*>(c_row);
      if (p.c_vec && n == 32) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(c) + u);
          v[4 * u] = fmaf(p.beta, w.x, v[4 * u]);
          v[4 * u + 1] = fmaf(p.beta, w.y, v[4 * u + 1]);
          v[4 * u + 2] = fmaf(p.beta, w.z, v[4 * u + 2]);
          v[4 * u + 3] = fmaf(p.beta, w.w, v[4 * u + 3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < n) v[j] = fmaf(p.beta, __ldg(c + j), v[j]);
      }
    } else {
      const uint16_t* c = static_cast<const uint16_t*>(c_row);
      if (p.c_vec && n == 32) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(c) + u);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            v[8 * u + 2 * h] = fmaf(p.beta, half_bits_to_float<BF16>((uint16_t)(ws[h] & 0xFFFFu)), v[8 * u + 2 * h]);
            v[8 * u + 2 * h + 1] = fmaf(p.beta, half_bits_to_float<BF16>((uint16_t)(ws[h] >> 16)), v[8 * u + 2 * h + 1]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < n) v[j] = fmaf(p.beta, half_bits_to_float<BF16>(__ldg(c + j)), v[j]);
      }
    }
  }
  if (bias != nullptr) {
    if (n == 32 && (reinterpret_cast<uintptr_t>(bias) & 15) == 0) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(bias) + u);
        v[4 * u] += w.x;
        v[4 * u + 1] += w.y;
        v[4 * u + 2] += w.z;
        v[4 * u + 3] += w.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) v[j] += __ldg(bias + j);
    }
  }
  if (p.act != kActNone) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = act_value(p.act, v[j]);
  }
}

// Writes `n` of a row's 32 values to d_row, rounded to nearest even for 16-bit outputs.
template <bool BF16>
__device__ __forceinline__ void store_row(const GroupedParams& p, const float (&v)[32], void* d_row, int n) {
  if (p.out_f32) {
    float* d = static_cast<float*>(d_row);
    if (p.d_vec && n == 32) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        reinterpret_cast<float4*>(d)[u] = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) d[j] = v[j];
    }
  } else {
    uint16_t* d = static_cast<uint16_t*>(d_row);
    if (p.d_vec && n == 32) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        reinterpret_cast<uint4*>(d)[u] =
            make_uint4(pack2<BF16>(v[8 * u], v[8 * u + 1]), pack2<BF16>(v[8 * u + 2], v[8 * u + 3]),
                       pack2<BF16>(v[8 * u + 4], v[8 * u + 5]), pack2<BF16>(v[8 * u + 6], v[8 * u + 7]));
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < n) d[j] = (uint16_t)(pack2<BF16>(v[j], 0.0f) & 0xFFFFu);
    }
  }
}

}  // namespace ttc
