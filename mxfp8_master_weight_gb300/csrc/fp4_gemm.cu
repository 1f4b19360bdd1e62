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
  // Split over k: outputs of at most 64 rows or columns (a tile of the pair kernel would stay mostly empty: split / pairs
  // 1 x 4096 x 4096 4.2 / 8.8 us, 64 x 1024 x 4096 5.7 / 7.0, 64 x 8192 x 8192 11.9 / 12.5; 64 x 16384 x 4096 11.7 / 11.3 is the
  // exception), and tiles so few that four CTAs can share each, with a k that pays for joining the sums, the longer the more
  // tiles there are (128 x 1024 x 8192 7.7 / 10.7, 256 x 256 x 8192 7.0 / 10.6, 512 x 1024 x 8192 8.8 / 10.8, 512 x 512 x 4096
  // 7.6 / 7.4, 512 x 512 x 2048 7.1 / 5.6, 300 x 300 x 300 13.1 / 5.3).  From 65 to 256 tokens against a large weight pairs take about
  // the same time, however full their tiles are (of 8192 x 8192: 65 rows 12.6, 128 13.0, 256 13.2, 512 16.1; of 16384 x 4096: 11.5,
  // 12.1, 12.5, 17.7; floors 5.8 to 9).
  const int64_t tiles = ((p.g.m + 127) / 128) * ((p.g.n + 127) / 128), stages = (p.g.k + kFp4StageK - 1) / kFp4StageK;
  const bool few = 4 * tiles <= dev.sms && stages >= 15 + tiles / 2;
  const bool split = p.g.k > 0 && (p.g.m <= 64 || p.g.n <= 64 || few);
  return split ? launch_fp4_gemm_split(p, given_up, dev, stream, what)
               : launch_fp4_gemm_pair(p, given_up, dev, stream, what);
}

}  // namespace mxfp8
