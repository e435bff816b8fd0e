// Device side of the grouped products: the table of groups and tiles that
// every CTA builds from the device's offsets, and the values of the epilogue.
#pragma once
#include "gemm_kernel.cuh"
#include "grouped.cuh"

namespace ttc {

// The tensor cores cut, not round, each addition to an accumulator, an error that
// grows with the number of them: fp32 results start a fresh accumulator every so
// many k-blocks, 768 tokens, and the partial sums are added up rounded to nearest.
constexpr int kSumKBlocks = 12;

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

__device__ __forceinline__ int divide(int n, FastDiv f) { return (int)((__umulhi((uint32_t)n, f.mul) + (uint32_t)n) >> f.shift); }

// Tiles of a group walk 2^group_shift row blocks of one column block before the
// next column block, so that CTAs at work together share panels of A and B.
template <int ROWS, bool WGRAD>
__device__ __forceinline__ GroupedTile grouped_tile(const GroupedParams& p, const GroupTable& tb, int t) {
  GroupedTile x;
  int first, rows;
  if constexpr (WGRAD) {
    x.g = divide(t, p.by_group);
    first = x.g * p.row_blocks * p.col_blocks;
    group_rows(p, tb, x.g, x.lo, x.hi);
    rows = p.row_blocks;
  } else {
    x.g = group_of_tile<ROWS>(p, tb, t, first);
    group_rows(p, tb, x.g, x.lo, x.hi);
    rows = (x.hi - x.lo + ROWS - 1) / ROWS;
  }
  int r = t - first;
  const int b = divide(r, p.by_band), above = b << p.group_shift;
  const int size = rows - above;  // row blocks of the band, where it is the last one
  r -= (b * p.col_blocks) << p.group_shift;
  if (size >= 1 << p.group_shift) {
    x.cb = r >> p.group_shift;
    x.rb = above + (r & ((1 << p.group_shift) - 1));
  } else {
    x.cb = WGRAD ? divide(r, p.by_rest) : r / size;
    x.rb = above + r - x.cb * size;
  }
  return x;
}

// CTA pairs: what they take in turn, `whole` tiles, then halves of tiles.
struct PairWalk {
  int whole, items;
};
__device__ __forceinline__ PairWalk pair_walk(int tiles, int pairs) {
  const int rest = tiles % pairs;
  PairWalk w{tiles, tiles};
  if (2 * rest <= pairs) {
    w.whole = tiles - rest;
    w.items = tiles + rest;
  }
  return w;
}

struct PairItem {
  GroupedTile x;
  int half;  // of the tile's columns; -1: all of them
};
template <bool WGRAD>
__device__ __forceinline__ PairItem pair_item(const GroupedParams& p, const GroupTable& tb, const PairWalk& w, int t) {
  const int over = t - w.whole;
  PairItem it;
  it.half = over < 0 ? -1 : over & 1;
  it.x = grouped_tile<kGroupedPairTile, WGRAD>(p, tb, over < 0 ? t : w.whole + (over >> 1));
  return it;
}

// A lane's four of the warp's 128 columns, zeros outside `n` columns.
__device__ __forceinline__ float4 four_columns(const float* c0, int lane, int n) {
  const float* c = c0 + lane * 4;
  n -= lane * 4;
  if (n >= 4 && (reinterpret_cast<uintptr_t>(c) & 15) == 0) return __ldg(reinterpret_cast<const float4*>(c));
  return make_float4(n > 0 ? __ldg(c) : 0.0f, n > 1 ? __ldg(c + 1) : 0.0f, n > 2 ? __ldg(c + 2) : 0.0f,
                     n > 3 ? __ldg(c + 3) : 0.0f);
}

// 32 values of a row (columns s32 * 32 on of the warp's 128) from their
// accumulator: alpha, bias, activation.  Each lane has four columns' biases and
// hands them round: loaded here they would cost a wait for L2 each time.
__device__ __forceinline__ void grouped_values(const GroupedParams& p, const uint32_t (&r)[32], float4 bias, int s32,
                                               float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = p.alpha * __uint_as_float(r[j]);
  if (p.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int src = s32 * 8 + i;
      v[4 * i] += __shfl_sync(0xFFFFFFFFu, bias.x, src);
      v[4 * i + 1] += __shfl_sync(0xFFFFFFFFu, bias.y, src);
      v[4 * i + 2] += __shfl_sync(0xFFFFFFFFu, bias.z, src);
      v[4 * i + 3] += __shfl_sync(0xFFFFFFFFu, bias.w, src);
    }
  }
  if (p.act != kActNone) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = act_value(p.act, v[j]);
  }
}

// The warp's staging block: 32 rows of 4 W bytes in 16-byte pieces, turned so
// that neither a row per lane nor whole rows meet a bank twice (eight lanes take
// a row of 128 bytes, four lanes one of 64).
template <int W>
__device__ __forceinline__ int staged(int r, int piece) {
  return W == 32 ? r * 128 + ((piece ^ (r & 7)) << 4) : r * 64 + ((piece ^ ((r >> 1) & 3)) << 4);
}

// Writes 32 staged rows to D: `rows` of them, from d0 on with pitch ldd, and `n`
// columns are inside D.  Whole 128-byte lines where D allows it: stores of half
// lines took 1.6 times as long (gradient to fp32 of 8 x 4096 x 4096, 128 tokens
// a group: 172 us against 109).  Columns that no 16-byte store reaches go one
// by one, kAtOnce rows of them read before the first is stored.
template <typename T, int kAtOnce>
__device__ __forceinline__ void copy_out(const GroupedParams& p, const uint8_t* sb, T* d0, int rows, int n, int lane) {
  constexpr int kElems = 16 / (int)sizeof(T), kCols = 128 / (int)sizeof(T);
  n = max(0, min(n, kCols));  // a warp's columns may all lie behind D's last
  const int whole = p.d_vec ? n & ~(kElems - 1) : 0;  // columns stored as 16-byte pieces
  const int piece = lane & 7, r0 = lane >> 3;
  if (piece * kElems < whole) {
    T* d = d0 + (int64_t)r0 * p.ldd + piece * kElems;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(sb + staged<32>(i * 4 + r0, piece));
      if (i * 4 + r0 < rows) *reinterpret_cast<uint4*>(d + (int64_t)(i * 4) * p.ldd) = v;
    }
  }
  if (whole < n) {
    for (int c = whole + lane; c < n; c += 32) {
      T* d = d0 + c;
#pragma unroll 1
      for (int r = 0; r < rows; r += kAtOnce) {
        T y[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          y[i] = *reinterpret_cast<const T*>(sb + staged<32>(r + i, c / kElems) + (c % kElems) * sizeof(T));
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (r + i < rows) d[(int64_t)(r + i) * p.ldd] = y[i];
      }
    }
  }
}

}  // namespace ttc
