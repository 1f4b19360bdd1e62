// What a kernel with much shared memory needs before a launch (host code).
#pragma once

#include "status.h"

namespace mxfp8 {

// Lets a kernel take `bytes` of dynamic shared memory, once per device: `done` has a bit for each that was told.
inline cudaError_t allow_smem(const void* kernel, int bytes, int device, std::atomic<unsigned long long>* done) {
  const unsigned long long bit = device < kMaxDevices ? 1ull << device : 0;
  if (done->load() & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit);
  return e;
}

}  // namespace mxfp8
