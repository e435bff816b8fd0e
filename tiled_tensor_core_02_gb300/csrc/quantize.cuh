// Rows of int8 with a scale each (quantize.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace ttc {

enum QuantIn : int { kQuantF16 = 0, kQuantBF16 = 1, kQuantF32 = 2 };

struct QuantParams {
  const void* x;
  int64_t ldx;
  int8_t* q;
  int64_t ldq;
  float* scale;
  int rows, cols;
};

cudaError_t launch_quantize_rows(const QuantParams& p, QuantIn in, int sm_count, cudaStream_t stream);

}  // namespace ttc
