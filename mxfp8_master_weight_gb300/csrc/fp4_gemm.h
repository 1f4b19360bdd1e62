// The kernels of a product of NVFP4 operands (host code).
#pragma once

#include <cuda_runtime.h>

#include "linear.h"

namespace mxfp8 {

constexpr int kFp4StageK = 256;  // values of k per pipeline stage: one 128-byte row

cudaError_t launch_fp4_gemm_pair(const Fp4GemmParams& p, unsigned* given_up, const DeviceInfo& dev, cudaStream_t stream,
                                 const char** what);
cudaError_t launch_fp4_gemm_split(const Fp4GemmParams& p, unsigned* given_up, const DeviceInfo& dev,
                                  cudaStream_t stream, const char** what);

}  // namespace mxfp8
