// Product of two NVFP4 operands, out = A B^T (+ addend), on the tensor cores.
//
//   out[i][j] = (1 / Sa) (1 / Sb) sum_p s_a(i, p / 16) s_b(j, p / 16) A(i, p) B(j, p)
//
// with E2M1 codes and one E4M3 scale per 16 values of p.  The block-scaled matrix instruction of 4-bit operands
// (tcgen05.mma kind::mxf4nvf4, four scales per 64 values) takes codes and scales as they lie and adds into F32 sums in
// tensor memory; the two tensor scales join in the epilogue.  Rows and bytes past the matrix are zeros,
// which add nothing.
//
// This file chooses the kernel: tiles of 256 x 256 by pairs of CTAs (fp4_gemm_pair.cu), or tiles of 128 rows with the
// contraction split over a cluster (fp4_gemm_split.cu).
#include "fp4_gemm.h"

#include "status.h"

namespace mxfp8 {

cudaError_t launch_fp4_gemm(const Fp4GemmParams& p, const DeviceInfo& dev, cudaStream_t stream, const char** what) {
  unsigned* given_up = nullptr;
  const cudaError_t e = given_up_address(dev.device, &given_up);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((p.g.m + 127) / 128) * ((p.g.n + 127) / 128), stages = (p.g.k + kFp4StageK - 1) / kFp4StageK;
  const bool few = 4 * tiles <= dev.sms && stages >= 15 + tiles / 2;
  const bool split = p.g.k > 0 && (p.g.m <= 64 || p.g.n <= 64 || few);
  return split ? launch_fp4_gemm_split(p, given_up, dev, stream, what)
               : launch_fp4_gemm_pair(p, given_up, dev, stream, what);
}

}  // namespace mxfp8
