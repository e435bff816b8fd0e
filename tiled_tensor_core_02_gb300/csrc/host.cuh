// What the entry points that live outside gemm.cu share with it on the host:
// the device's properties, the debug knobs that apply to every kernel, the
// tensor-map encoder and the launch counter.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ttc.h"

namespace ttc {

// Largest size or leading dimension accepted (elements): the kernels index
// rows, columns and k in 32-bit integers and step past the end by up to a
// grid's stride (well under 2^24) before a loop test, which must not wrap.
constexpr int64_t kSizeLimit = (1ll << 31) - (1ll << 24);

struct HostEnv {
  int sm_count;
  uint32_t* err;        // the device error word
  uint64_t timeout_ns;  // budget of a kernel's barrier waits
  int inject_stall;
  bool plain_loads;  // TTC_KNOB_FORCE_GENERIC_LOAD
};

// The current device, set up on first use.
ttc_status host_env(HostEnv& env);

// 3-D tensor map of `dt` elements of `esize` bytes: `inner` contiguous ones,
// `outer` rows `pitch` elements apart, `count` matrices `stride` elements
// apart; boxes of box_inner x box_outer x 1.
bool encode_matrices(CUtensorMap* m, CUtensorMapDataType dt, int esize, const void* base, int64_t inner, int64_t outer,
                     int64_t pitch, int64_t count, int64_t stride, int box_inner, int box_outer, CUtensorMapSwizzle sw);

// What TMA can address: a base on a 16-byte boundary and a pitch (and, with
// more than one matrix, a stride) of whole 16-byte granules.
bool tma_rows_ok(const void* p, int64_t ld, int esize);
bool tma_stride_ok(int64_t count, int64_t stride, int esize);

bool byte_ranges_overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes);

void count_launches(int n);

}  // namespace ttc
