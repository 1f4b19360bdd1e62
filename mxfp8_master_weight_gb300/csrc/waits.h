// When a kernel's wait is given up, apart from the waiting itself (host and device code).
#pragma once

#ifdef __CUDACC__
#define MXFP8_HD __host__ __device__ __forceinline__
#else
#define MXFP8_HD inline
#endif

namespace mxfp8 {
namespace tc {

constexpr unsigned kWaitCycles = 4000000000u;  // about two seconds of waiting
constexpr unsigned kPollCycles = 1u << 24;     // what one interval between two looks counts at most (8 ms)

// The clock of one wait.  It counts the time that passed while the thread looked, not what went by meanwhile: a
// grid that is taken off the GPU in favour of another process, or stopped in a debugger, looks once
// after it is back, and that interval counts as kPollCycles however long it was.  The 32-bit clock
// serves: an interval that wraps it still counts as kPollCycles at most.
struct Patience {
  unsigned last, spent;
  MXFP8_HD explicit Patience(unsigned now) : last(now), spent(0) {}
  MXFP8_HD bool out(unsigned now) {
    const unsigned d = now - last;
    last = now;
    spent += d < kPollCycles ? d : kPollCycles;
    return spent > kWaitCycles;
  }
};
static_assert(kWaitCycles + kPollCycles > kWaitCycles, "spent fits 32 bits");

}  // namespace tc
}  // namespace mxfp8
