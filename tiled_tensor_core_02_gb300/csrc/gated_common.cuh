// Device side of the gated feed-forward blocks: activations with their derivatives,
// and what an epilogue warp does with 32 rows of 64 columns.
//
// All values are fp32 from the accumulator to the one rounding of each result; the
// kept projections are rounded when they are written, D is computed from what they
// were before.  The gradient reads the kept, rounded ones.
#pragma once
#include "grouped_common.cuh"

namespace ttc {

constexpr int kActSilu = 3;  // gated blocks only

// The logistic function.  exp overflows to infinity for v below -88.7: 0, as it should be.
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// ACT: the activation, which a warp tells apart once for all of its values: a branch for each
// of them cost more than the arithmetic.
template <int ACT>
__device__ __forceinline__ float gated_act(float v) {
  // v / (1 + exp(-v)) with the division's own limit in mind: __fdividef gives 0 for
  // denominators from 2^126 on, where the quotient is below 2^-119
  if constexpr (ACT == kActSilu) return __fdividef(v, 1.0f + __expf(-v));
  return act_value(ACT, v);
}

// act(v) and its derivative.  SiLU: s + v s (1 - s), s the logistic function; GELU
// (tanh form) is v q with q the logistic function of 2 u(v), its derivative q + v q (1 - q)
// 2 u'(v); that last term is 0 in fp32 for |v| > 16, where u' could overflow.
// ReLU's derivative is 0 at 0.
struct ActSlope {
  float value, slope;
};
template <int ACT>
__device__ __forceinline__ ActSlope act_slope(float v) {
  ActSlope r{v, 1.0f};
  if constexpr (ACT == kActSilu) {
    const float s = logistic(v);
    r.value = v * s;
    r.slope = fmaf(r.value, 1.0f - s, s);
  } else if constexpr (ACT == kActGelu) {
    const float c = fminf(fmaxf(v, -16.0f), 16.0f);
    const float q = logistic(1.5957691216057308f * fmaf(0.044715f * c, c * c, c));
    r.value = v * q;
    r.slope = fmaf(c * q * (1.0f - q), 1.5957691216057308f * fmaf(0.134145f * c, c, 1.0f), q);
    if (v != v) r.value = r.slope = v;
  } else if constexpr (ACT == kActRelu) {
    r.value = v < 0.0f ? 0.0f : v;
    r.slope = v > 0.0f ? 1.0f : 0.0f;
  }
  return r;
}

// Calls f with the activation as a constant.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == kActSilu)
    f(std::integral_constant<int, kActSilu>{});
  else if (act == kActGelu)
    f(std::integral_constant<int, kActGelu>{});
  else if (act == kActRelu)
    f(std::integral_constant<int, kActRelu>{});
  else
    f(std::integral_constant<int, kActNone>{});
}

// 32 staged rows of 64 16-bit columns to global memory (pitch ld), `rows` and `n` of
// them inside the matrix; `vec`: rows start on 16-byte boundaries.
__device__ __forceinline__ void store_unit(const uint8_t* sb, uint16_t* d0, int64_t ld, bool vec, int rows, int n, int lane) {
  n = min(n, 64);
  const int whole = vec ? n & ~7 : 0;
  const int piece = lane & 7, r0 = lane >> 3;
  if (piece * 8 < whole) {
    uint16_t* d = d0 + (int64_t)r0 * ld + piece * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(sb + staged<32>(i * 4 + r0, piece));
      if (i * 4 + r0 < rows) *reinterpret_cast<uint4*>(d + (int64_t)(i * 4) * ld) = v;
    }
  }
  for (int c = whole + lane; c < n; c += 32) {
    uint16_t* d = d0 + c;
#pragma unroll 1
    for (int r = 0; r < rows; r += 4) {
      uint16_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const uint16_t*>(sb + staged<32>(r + i, c / 8) + (c % 8) * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < rows) d[(int64_t)(r + i) * ld] = y[i];
    }
  }
}

// 64 columns of the lane's row, two a word, into the staging block.
__device__ __forceinline__ void stage_words(uint8_t* sb, int lane, const uint32_t (&w)[32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(sb + staged<32>(lane, i)) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// The reverse of store_unit, in two steps so that both matrices' loads are on their way
// together: into registers in the order of store_unit, 16 bytes a lane where rows start on
// 16-byte boundaries and the piece lies inside (`n` columns do), else element by element, all of
// them asked for before the first is used; then through the staging block to a row per lane.
// Zeros outside `rows` and `n` columns.
__device__ __forceinline__ void fetch_unit(const uint16_t* c0, int64_t ld, bool vec, int rows, int n, int lane,
                                           uint32_t (&w)[32]) {
  const int piece = lane & 7, r0 = lane >> 3;
  const uint16_t* src = c0 + (int64_t)r0 * ld + piece * 8;
  n -= piece * 8;
  if (vec && n >= 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (i * 4 + r0 < rows) v = *reinterpret_cast<const uint4*>(src + (int64_t)(i * 4) * ld);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = i * 4 + r0 < rows;
        const uint16_t* at = src + (int64_t)(i * 4) * ld + 2 * e;
        const uint32_t lo = in && 2 * e < n ? at[0] : 0u, hi = in && 2 * e + 1 < n ? at[1] : 0u;
        w[4 * i + e] = lo | hi << 16;
      }
  }
}
__device__ __forceinline__ void turn_unit(int lane, uint8_t* sb, uint32_t (&w)[32]) {
  const int piece = lane & 7, r0 = lane >> 3;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(sb + staged<32>(i * 4 + r0, piece)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  __syncwarp();
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

// 32 columns of an accumulator, zeros where the product has no terms.
__device__ __forceinline__ void sums_32(uint32_t taddr, bool has_k, uint32_t (&w)[32]) {
  if (has_k) {
    tmem_ld_32x32b_x32(taddr, w);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) w[j] = 0u;
  }
}

// Forward: rows `row` .. of `rows`, columns `col` .. of `n`, from the accumulators of
// both projections.  `release` is called when the last of them has been read.  The
// kept projections are written first, a third of the reads of tensor memory for as
// many registers less.
template <bool BF16, typename R>
__device__ __forceinline__ void gated_forward_unit(const GatedParams& p, uint32_t gate_at, uint32_t up_at, bool has_k,
                                                   int64_t row, int rows, int col, int n, uint8_t* sb, int lane, R release) {
  if (n <= 0 || rows <= 0) {
    release();
    return;
  }
  if (p.gate != nullptr) {
#pragma unroll 1
    for (int o = 0; o < 2; ++o) {
      const uint32_t at = o == 0 ? gate_at : up_at;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[32];
        sums_32(at + h * 32, has_k, w);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(sb + staged<32>(lane, h * 4 + i)) =
              make_uint4(pack2<BF16>(__uint_as_float(w[8 * i]), __uint_as_float(w[8 * i + 1])),
                         pack2<BF16>(__uint_as_float(w[8 * i + 2]), __uint_as_float(w[8 * i + 3])),
                         pack2<BF16>(__uint_as_float(w[8 * i + 4]), __uint_as_float(w[8 * i + 5])),
                         pack2<BF16>(__uint_as_float(w[8 * i + 6]), __uint_as_float(w[8 * i + 7])));
      }
      __syncwarp();
      store_unit(sb, static_cast<uint16_t*>(o == 0 ? p.gate : p.up) + row * p.ldp + col, p.ldp, p.p_vec != 0, rows, n, lane);
      __syncwarp();
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t g[32], u[32];
    sums_32(gate_at + h * 32, has_k, g);
    sums_32(up_at + h * 32, has_k, u);
    tmem_ld_wait();
    if (h == 1) release();
    float v[32];
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = gated_act<decltype(act)::value>(__uint_as_float(g[j])) * __uint_as_float(u[j]);
    });
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(sb + staged<32>(lane, h * 4 + i)) =
          make_uint4(pack2<BF16>(v[8 * i], v[8 * i + 1]), pack2<BF16>(v[8 * i + 2], v[8 * i + 3]),
                     pack2<BF16>(v[8 * i + 4], v[8 * i + 5]), pack2<BF16>(v[8 * i + 6], v[8 * i + 7]));
  }
  __syncwarp();
  store_unit(sb, static_cast<uint16_t*>(p.D) + row * p.ldd + col, p.ldd, p.d_vec != 0, rows, n, lane);
  __syncwarp();
}

__device__ __forceinline__ void unpack2(bool bf16, uint32_t w, float& a, float& b) {
  if (bf16) {
    a = half_bits_to_float<true>((uint16_t)(w & 0xFFFFu));
    b = half_bits_to_float<true>((uint16_t)(w >> 16));
  } else {
    a = half_bits_to_float<false>((uint16_t)(w & 0xFFFFu));
    b = half_bits_to_float<false>((uint16_t)(w >> 16));
  }
}

// Gradient of 32 rows by 64 columns.  Both projections are read while the products are on
// their way; `wait` returns whether those are done, `release` is called behind the last
// read of them.  Exponential and quotient serve the gradients and D alike (8192 x 14336 x
// 4096: 634 us; with D computed and written on its own while the products came 728; with
// the next 64 columns' projections loaded while these results are written 643, asked
// of L2 in time 652).
template <bool BF16, typename W, typename R>
__device__ __forceinline__ bool gated_grad_unit(const GatedParams& p, uint32_t at, bool has_k, int64_t row, int rows, int col,
                                                int n, uint8_t* sb, int lane, W wait, R release) {
  if (n <= 0 || rows <= 0) {
    if (!wait()) return false;
    release();
    return true;
  }
  uint32_t g[32], u[32], d[32];
  fetch_unit(static_cast<const uint16_t*>(p.gate) + row * p.ldp + col, p.ldp, p.p_vec != 0, rows, n, lane, g);
  fetch_unit(static_cast<const uint16_t*>(p.up) + row * p.ldp + col, p.ldp, p.p_vec != 0, rows, n, lane, u);
  turn_unit(lane, sb, g);
  turn_unit(lane, sb, u);
  if (!wait()) return false;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t w[16];
    if (has_k) {
      tmem_ld_32x32b_x16<0>(at + h * 16, w);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = 0u;
    }
    tmem_ld_wait_for(w);
    if (h == 3) release();
    with_act(p.act, [&](auto act) {
      constexpr int kAct = decltype(act)::value;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float g0, g1, u0, u1;
        unpack2(BF16, g[h * 8 + j], g0, g1);
        unpack2(BF16, u[h * 8 + j], u0, u1);
        const ActSlope a0 = act_slope<kAct>(g0), a1 = act_slope<kAct>(g1);
        const float d0 = __uint_as_float(w[2 * j]), d1 = __uint_as_float(w[2 * j + 1]);
        g[h * 8 + j] = pack2<BF16>(d0 * u0 * a0.slope, d1 * u1 * a1.slope);
        u[h * 8 + j] = pack2<BF16>(d0 * a0.value, d1 * a1.value);
        d[h * 8 + j] = pack2<BF16>(a0.value * u0, a1.value * u1);
      }
    });
  }
  stage_words(sb, lane, g);
  __syncwarp();
  store_unit(sb, static_cast<uint16_t*>(p.dgate) + row * p.lddp + col, p.lddp, p.dp_vec != 0, rows, n, lane);
  __syncwarp();
  stage_words(sb, lane, u);
  __syncwarp();
  store_unit(sb, static_cast<uint16_t*>(p.dup) + row * p.lddp + col, p.lddp, p.dp_vec != 0, rows, n, lane);
  __syncwarp();
  if (p.D != nullptr) {
    stage_words(sb, lane, d);
    __syncwarp();
    store_unit(sb, static_cast<uint16_t*>(p.D) + row * p.ldd + col, p.ldd, p.d_vec != 0, rows, n, lane);
    __syncwarp();
  }
  return true;
}

}  // namespace ttc
