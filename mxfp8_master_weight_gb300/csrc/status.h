// The count of kernels that gave up a wait, per device.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace mxfp8 {

constexpr int kMaxDevices = 64;

// Of a count that only grows (and may wrap): what has been added since it was last asked about.  However
// readings of several threads overlap, every addition is told once.
struct Told {
  std::atomic<unsigned> known{0};
  unsigned news(unsigned seen) {
    unsigned before = known.load();
    while (int(seen - before) > 0)
      if (known.compare_exchange_weak(before, seen)) return seen - before;
    return 0;
  }
};

// Where the current device's kernels count the waits that they gave up.
cudaError_t given_up_address(int device, unsigned** out);
// Waits for the stream; *count: those of the current device that no call has told before.
cudaError_t waits_given_up(cudaStream_t stream, unsigned* count);

}  // namespace mxfp8
