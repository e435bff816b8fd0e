// Instantiations and launch of the CTA-pair int8 kernel with a scaled result.
#include <cuda_runtime.h>

#include <atomic>

#include "gemm2sm_kernel.cuh"
#include "gemm_launch.cuh"

namespace ttc {

namespace {

using Cfg = PairCfg<256, true, 8>;
constexpr int kThreads = 64 + 32 * 8;

template <int kScaled>
cudaError_t launch(const GemmParams& p, int clusters, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(gemm_pair_kernel<256, false, true, 8, kScaled>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters, 1, 1);  // clusters of 2 from the kernel's __cluster_dims__
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  add_pdl_attribute(cfg, attr);
  e = cudaLaunchKernelEx(&cfg, gemm_pair_kernel<256, false, true, 8, kScaled>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_pair_i8_scaled(I8Result out, const GemmParams& p, int clusters, cudaStream_t stream) {
  switch (out) {
    case kI8ToF16: return launch<kI8ToF16>(p, clusters, stream);
    case kI8ToBF16: return launch<kI8ToBF16>(p, clusters, stream);
    case kI8ToF32: return launch<kI8ToF32>(p, clusters, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ttc
