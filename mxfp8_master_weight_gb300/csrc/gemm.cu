// Block-scaled product out = A B^T (+ addend) on the tensor cores.
//
//   out[i][j] = sum_p 2^(ea - 127) 2^(eb - 127) A(i, p) B(j, p)
//
// with E4M3 codes and one E8M0 scale per 32 or 128 values of p in each operand.  The scales are
// powers of two, so the block-scaled matrix instruction (tcgen05.mma kind::mxf8f6f4) takes them
// as they are: it multiplies each 32-value partial product by both scales and adds into F32 sums
// in tensor memory, with no pass over the sums in between.  A scale column in tensor memory
// holds four bytes per row; with 32 values per scale the four instructions of a 128-value stage
// take bytes 0..3, with 128 values they all take byte (stage % 4), so both block sizes read the
// same 128x4-tile layout and may meet in one product.
//
// An operand is read as it lies: a box of 128 stored rows by 128 bytes goes to shared memory under
// the 128-byte swizzle whether its rows run along k or across it, and the instruction descriptor
// says which.  Rows and bytes past the matrix are zeros, which add nothing (a scale is never
// infinite; padding scales are finite).
//
// This file chooses the kernel: tiles of 256 x 256 by pairs of CTAs (gemm_pair.cu), or tiles of 128
// rows with the contraction split over a cluster (gemm_split.cu).
#include "gemm_impl.cuh"
#include "gemm_maps.h"
#include "status.h"

namespace mxfp8 {

cudaError_t launch_gemm(const GemmParams& p, const DeviceInfo& dev, cudaStream_t stream, const char** what) {
  unsigned* given_up = nullptr;
  const cudaError_t e = given_up_address(dev.device, &given_up);
  if (e != cudaSuccess) return e;
  // Split over k: outputs of at most 64 rows or columns (a tile of the pair kernel would stay mostly
  // empty: 64 x 4096 x 4096 6.8 us split, 9.9 us by pairs), and tiles so few that four CTAs can share
  // each with an SM to themselves, with a k that pays for joining the sums, the longer the more tiles
  // there are (split / pairs: 160 x 96 x 2048 6.2 / 7.2 us, 512 x 512 x 2048 7.4 / 7.0, 512 x 512 x 4096 8.2 /
  // 9.7, 512 x 1024 x 8192 10.7 / 15.4, 128 x 4096 x 4096 8.8 / 9.9, 256 x 4096 x 8192 17.7 / 16.3).  Operands
  // that are realigned take longer per stage, so the split pays from fewer stages and to more tiles (both
  // operands off 16 bytes: 301 x 303 x 1005 10.8 / 16.8, 1000 x 1111 x 999 15.0 / 18.2, 301 x 303 x 305 15.9 / 10.4;
  // beyond the rule's tiles too with three weights in turn: 2001 x 1111 x 1999 27.7 / 33.9).
  const int64_t tiles = ((p.m + 127) / 128) * ((p.n + 127) / 128), stages = (p.k + kBlockK - 1) / kBlockK;
  const bool few = 4 * tiles <= dev.sms && stages >= 15 + tiles / 2;
  const bool realigned = !(p.a.aligned && p.b.aligned) && 2 * tiles <= dev.sms && stages >= 8;
  const bool split = p.k > 0 && (p.m <= 64 || p.n <= 64 || few || realigned);
  return split ? launch_gemm_split(p, given_up, dev, stream, what) : launch_gemm_pair(p, given_up, dev, stream, what);
}

}  // namespace mxfp8
