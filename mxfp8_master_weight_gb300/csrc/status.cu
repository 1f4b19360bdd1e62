// The health of the operators' kernels (see mxfp8_device_status).
#include "status.h"

namespace mxfp8 {

// Kernels that gave up a wait on this device.  Never set back: a write of zero would lose what another stream's
// kernels add between the reading and the write.
static __device__ unsigned g_given_up = 0;

// Looked up once per device.
cudaError_t given_up_address(int device, unsigned** out) {
  static std::atomic<unsigned*> known[kMaxDevices];
  unsigned* p = device < kMaxDevices ? known[device].load() : nullptr;
  if (p == nullptr) {
    const cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void**>(&p), g_given_up);
    if (e != cudaSuccess) return e;
    if (device < kMaxDevices) known[device].store(p);
  }
  *out = p;
  return cudaSuccess;
}

cudaError_t waits_given_up(cudaStream_t stream, unsigned* count) {
  static Told told[kMaxDevices];
  *count = 0;
  int device = 0;
  unsigned seen = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess && device >= kMaxDevices) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(&seen, g_given_up, sizeof seen, 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) *count = told[device].news(seen);
  return e;
}

}  // namespace mxfp8
