// Host side of the gated feed-forward blocks: argument checks, the choice of a
// kernel, tensor maps, launch.  See include/ttc.h for the contract.
#include "operators_host.cuh"

using namespace ttc;

namespace {

bool is_gated_act(ttc_act a) { return is_act(a) || a == TTC_ACT_SILU; }

// A matrix of 16-bit elements.
struct Mat {
  const void* p;
  int64_t ld, rows, cols;
};
int64_t bytes_of(const Mat& a) { return span_bytes(1, 0, a.rows, a.ld, a.cols, 2); }
// Two matrices of the same pitch may lie side by side in one buffer: then their
// spans overlap, their elements do not.
bool side_by_side(const Mat& a, const Mat& b) {
  if (a.ld != b.ld) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t pitch = (uint64_t)(2 * a.ld);
  const uint64_t apart = y >= x ? (y - x) % pitch : (pitch - (x - y) % pitch) % pitch;  // from a's columns on to b's
  return apart >= (uint64_t)(2 * a.cols) && pitch - apart >= (uint64_t)(2 * b.cols);
}
bool clash(const Mat& a, const Mat& b) {
  return a.p != nullptr && b.p != nullptr && byte_ranges_overlap(a.p, bytes_of(a), b.p, bytes_of(b)) && !side_by_side(a, b);
}

// What both calls refuse of their products' operands; TTC_OK with `nothing` set for
// an empty result.  A and one group's B as they are read, and how many of B; none with K == 0.
// The offsets are one row of 16-bit elements.
struct Products {
  bool nothing;
  Mat offsets, a, b;
  int64_t mats, stride;
};
ttc_status check_products(int64_t groups, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const int32_t* offsets,
                          const void* B, int64_t ldb, int64_t strideB, ttc_layout layoutB, ttc_act act, ttc_dtype dtype,
                          Products& out) {
  out = Products{};
  if (groups < 0 || M < 0 || N < 0 || K < 0 || strideB < 0) return TTC_ERR_INVALID_ARG;
  if (layoutB != TTC_ROW_MAJOR && layoutB != TTC_COL_MAJOR) return TTC_ERR_INVALID_ARG;
  if (!is_gated_act(act) || !is_dtype(dtype)) return TTC_ERR_INVALID_ARG;
  if (!is_16bit(dtype)) return TTC_ERR_UNSUPPORTED;
  if (groups == 0 || M == 0 || N == 0) {
    out.nothing = true;
    return TTC_OK;
  }
  if (offsets == nullptr && groups != 1) return TTC_ERR_INVALID_ARG;
  if (lda < at_least_1(K) || ldb < at_least_1(layoutB == TTC_ROW_MAJOR ? N : K)) return TTC_ERR_INVALID_ARG;
  if (K > 0 && (A == nullptr || B == nullptr || !aligned(A, 2) || !aligned(B, 2))) return TTC_ERR_INVALID_ARG;
  if (!aligned(offsets, 4)) return TTC_ERR_INVALID_ARG;
  if (groups > kMaxGroups || M > kSizeLimit || N > kSizeLimit || K > kSizeLimit || lda > kSizeLimit || ldb > kSizeLimit ||
      strideB > kStrideLimit)
    return TTC_ERR_UNSUPPORTED;
  if ((blocks_of(M, kGroupedPlainTile) + groups) * blocks_of(N, kGatedPlainCols) > kSizeLimit) return TTC_ERR_UNSUPPORTED;
  out.offsets = Mat{offsets, 0, 1, 2 * (groups + 1)};
  if (K > 0) {
    out.a = Mat{A, lda, M, K};
    out.b = layoutB == TTC_ROW_MAJOR ? Mat{B, ldb, K, N} : Mat{B, ldb, N, K};
    out.mats = strideB != 0 ? groups : 1;
    out.stride = strideB;
  }
  return TTC_OK;
}

// Whether an output touches what is read while it is written: the offsets (which CTAs that work on
// one tile each read for themselves), A, a group's B, or of the forward pass its U, laid out as B.
bool hits_operands(const Mat& d, const Products& o, const void* U) {
  if (d.p == nullptr) return false;
  if (clash(d, Mat{o.offsets.p, d.ld, o.offsets.rows, o.offsets.cols})) return true;  // a single row has any pitch
  if (o.mats == 0) return false;
  if (clash(d, o.a)) return true;
  const int64_t all = span_bytes(o.mats, o.stride, o.b.rows, o.b.ld, o.b.cols, 2);
  for (const void* w : {o.b.p, U}) {
    if (w == nullptr || !byte_ranges_overlap(d.p, bytes_of(d), w, all)) continue;
    for (int64_t g = 0; g < o.mats; ++g)
      if (clash(d, Mat{static_cast<const uint16_t*>(w) + g * o.stride, o.b.ld, o.b.rows, o.b.cols})) return true;
  }
  return false;
}

bool rows_on_16(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

template <typename P>
void gated_params(P& p, const HostEnv& env, int64_t groups, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                  const int32_t* offsets, const void* B, int64_t ldb, int64_t strideB, ttc_layout layoutB, ttc_act act) {
  std::memset(&p, 0, sizeof p);
  common_params(p, env, groups, M, N, K, A, lda, B, ldb, offsets);
  p.strideB = strideB;
  p.b_mn = layoutB == TTC_ROW_MAJOR;
  p.k_blocks = (int)blocks_of(K, kBK);
  p.alpha = 1.0f;
  p.act = (int)act;
}

// The other projection's map, where TMA reads its weights as it reads the gate's.
bool map_up(GatedForward& p, ttc_dtype dtype, int box_rows) {
  if (!tma_rows_ok(p.U, p.ldb, 2)) return false;
  const CUtensorMapDataType dt = dtype == TTC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const int64_t mats = p.strideB != 0 ? p.groups : 1;
  return p.b_mn ? encode_matrices(&p.tmU, dt, 2, p.U, p.N, p.K, p.ldb, mats, p.strideB, 64, 128, sw)
                : encode_matrices(&p.tmU, dt, 2, p.U, p.K, p.N, p.ldb, mats, p.strideB, kBK, box_rows, sw);
}
bool map_up(GatedGrad&, ttc_dtype, int) { return true; }

// Block of tokens of the few-token kernel, 0 for CTA pairs: as ttc_gemm_grouped chooses it, and
// with more rows too wherever blocks of 64 make one wave of tiles of `width` columns (100 x 4096 x
// 4096 18.9 us against 23.7, the gradient 20.2 against 24.2, with the block's values 21.9; 100 x
// 1000 x 1000 9.3 against 11.4, 13.0 against 13.8; 512 x 1024 x 1024, where it loses most, 8.8
// against 9.9, 12.1 against 11.9 and 13.5 against 12.4).
int gated_few_block(int64_t rows, int64_t n, int64_t groups, int width, int sm_count) {
  const int block = few_block(rows, groups);
  if (block != 0) return block;
  return few_blocks(rows, 64, groups) * blocks_of(n, width) <= sm_count ? 64 : 0;
}

// Launches the kernel for these operands.
template <typename P>
ttc_status launch_gated(P& p, ttc_dtype dtype, const HostEnv& env, cudaStream_t stream) {
  constexpr bool kForward = kIsGatedForward<P>;
  const bool bf16 = dtype == TTC_BF16;
  const int64_t groups = p.groups < p.M ? p.groups : p.M;  // that have rows, as far as the host knows
  const int block = gated_few_block(p.M, p.N, groups, kForward ? 64 : 128, env.sm_count);
  if (block != 0 && few_maps(p, dtype, block, groups, env, kForward) && map_up(p, dtype, p.tile_cols)) {
    const int64_t tiles = (blocks_of(p.M, block) + groups) * p.col_blocks;
    if (launch_few_tokens(bf16, block, p, (int)(tiles < env.sm_count ? tiles : env.sm_count), stream) != cudaSuccess)
      return TTC_ERR_CUDA;
    count_launches(1);
    return TTC_OK;
  }
  if (pair_maps(p, false, dtype, env) && map_up(p, dtype, 128)) {
    const int clusters = grouped_pair_clusters();
    if (clusters <= 0) return TTC_ERR_CUDA;
    set_walk(p, 0, blocks_of(p.N, kForward ? kGatedPairCols : kGroupedPairTile), 3);
    p.b_stream = p.M <= p.groups * kGroupedPairTile;
    const int64_t tiles = (blocks_of(p.M, kGroupedPairTile) + groups) * p.col_blocks;
    if (launch_gated_pair(bf16, p, (int)(2 * tiles < clusters ? 2 * tiles : clusters), stream) != cudaSuccess)
      return TTC_ERR_CUDA;
    count_launches(1);
    return TTC_OK;
  }
  const int64_t col_blocks = blocks_of(p.N, kForward ? kGatedPlainCols : kGroupedPlainTile);
  set_walk(p, 0, col_blocks, 4);
  const int64_t tiles = (blocks_of(p.M, kGroupedPlainTile) + groups) * col_blocks;
  if (launch_gated_plain(bf16, p, (int)(tiles < env.sm_count ? tiles : env.sm_count), stream) != cudaSuccess)
    return TTC_ERR_CUDA;
  count_launches(1);
  return TTC_OK;
}

}  // namespace

extern "C" {

ttc_status ttc_gemm_gated(int64_t groups, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const int32_t* offsets,
                          const void* Bgate, const void* Bup, int64_t ldb, int64_t strideB, ttc_layout layoutB, void* D,
                          int64_t ldd, void* gate, void* up, int64_t ldp, ttc_act act, ttc_dtype dtype, void* stream) {
  Products o;
  ttc_status st = check_products(groups, M, N, K, A, lda, offsets, Bgate, ldb, strideB, layoutB, act, dtype, o);
  if (st != TTC_OK || o.nothing) return st;
  const bool save = gate != nullptr || up != nullptr;
  if (D == nullptr || ldd < N || !aligned(D, 2) || (K > 0 && (Bup == nullptr || !aligned(Bup, 2)))) return TTC_ERR_INVALID_ARG;
  if (save && (gate == nullptr || up == nullptr || ldp < N || !aligned(gate, 2) || !aligned(up, 2))) return TTC_ERR_INVALID_ARG;
  if (ldd > kSizeLimit || (save && ldp > kSizeLimit)) return TTC_ERR_UNSUPPORTED;
  const Mat d{D, ldd, M, N}, g{gate, ldp, M, N}, u{up, ldp, M, N};
  if (hits_operands(d, o, Bup) || hits_operands(g, o, Bup) || hits_operands(u, o, Bup) || clash(d, g) || clash(d, u) ||
      clash(g, u))
    return TTC_ERR_INVALID_ARG;

  HostEnv env;
  st = host_env(env);
  if (st != TTC_OK) return st;
  GatedForward p;
  gated_params(p, env, groups, M, N, K, A, lda, offsets, Bgate, ldb, strideB, layoutB, act);
  p.U = Bup;
  p.D = D;
  p.ldd = ldd;
  p.d_vec = rows_on_16(D, ldd);
  p.gate = gate;
  p.up = up;
  p.ldp = ldp;
  p.p_vec = rows_on_16(gate, ldp) && rows_on_16(up, ldp);
  return launch_gated(p, dtype, env, static_cast<cudaStream_t>(stream));
}

ttc_status ttc_gemm_gated_grad(int64_t groups, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                               const int32_t* offsets, const void* B, int64_t ldb, int64_t strideB, ttc_layout layoutB,
                               const void* gate, const void* up, int64_t ldp, void* dgate, void* dup, int64_t lddp, void* D,
                               int64_t ldd, ttc_act act, ttc_dtype dtype, void* stream) {
  Products o;
  ttc_status st = check_products(groups, M, N, K, A, lda, offsets, B, ldb, strideB, layoutB, act, dtype, o);
  if (st != TTC_OK || o.nothing) return st;
  if (gate == nullptr || up == nullptr || dgate == nullptr || dup == nullptr || ldp < N || lddp < N || (D != nullptr && ldd < N))
    return TTC_ERR_INVALID_ARG;
  if (!aligned(gate, 2) || !aligned(up, 2) || !aligned(dgate, 2) || !aligned(dup, 2) || !aligned(D, 2)) return TTC_ERR_INVALID_ARG;
  if (ldp > kSizeLimit || lddp > kSizeLimit || (D != nullptr && ldd > kSizeLimit)) return TTC_ERR_UNSUPPORTED;
  const Mat g{gate, ldp, M, N}, u{up, ldp, M, N}, dg{dgate, lddp, M, N}, du{dup, lddp, M, N}, d{D, ldd, M, N};
  const bool in_place = gate == dgate && up == dup && ldp == lddp;
  if (hits_operands(dg, o, nullptr) || hits_operands(du, o, nullptr) || hits_operands(d, o, nullptr) || clash(dg, du) ||
      clash(d, g) || clash(d, u) || clash(d, dg) || clash(d, du))
    return TTC_ERR_INVALID_ARG;
  if (!in_place && (clash(dg, g) || clash(dg, u) || clash(du, g) || clash(du, u)))
    return TTC_ERR_INVALID_ARG;

  HostEnv env;
  st = host_env(env);
  if (st != TTC_OK) return st;
  GatedGrad p;
  gated_params(p, env, groups, M, N, K, A, lda, offsets, B, ldb, strideB, layoutB, act);
  p.D = D;
  p.ldd = ldd;
  p.d_vec = rows_on_16(D, ldd);
  p.gate = const_cast<void*>(gate);
  p.up = const_cast<void*>(up);
  p.ldp = ldp;
  p.p_vec = rows_on_16(gate, ldp) && rows_on_16(up, ldp);
  p.dgate = dgate;
  p.dup = dup;
  p.lddp = lddp;
  p.dp_vec = rows_on_16(dgate, lddp) && rows_on_16(dup, lddp);
  return launch_gated(p, dtype, env, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
