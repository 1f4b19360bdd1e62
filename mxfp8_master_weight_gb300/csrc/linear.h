// Internal interface between the C entry points of the training operators
// (linear_capi.cu) and their kernels.  Parameters are validated before any launch.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace mxfp8 {

constexpr int kCkptBlock = 128;  // values per scale of an activation checkpoint

// Bytes of 128x4 scale tiles per 128 logical rows: 512 per 4 blocks.
inline __host__ __device__ int64_t scale_tile_cols(int64_t nblocks) { return (nblocks + 3) / 4; }

struct CheckpointSaveParams {
  const void* in;
  int64_t rows, cols, ld;
  uint8_t* q_r;        // rowwise codes or nullptr
  int64_t ld_r;
  uint8_t* s_r;
  uint8_t* q_c;        // columnwise codes or nullptr
  int64_t ld_c;
  uint8_t* s_c;
  int32_t vec_in;      // base and row stride are multiples of 8 elements' bytes (16 or 32)
  int32_t vec_r, vec_c;  // codes take 8-byte stores
};

struct CheckpointRestoreParams {
  const uint8_t* q;
  const uint8_t* s;
  int64_t rows, cols, ld_q;
  void* out;
  int64_t ld_o;
  int32_t colwise;
  int32_t vec_q;       // codes take 8-byte loads
  int32_t vec_out;     // likewise of the output
};

// One operand of a product: `codes` is the matrix [mn][k] (rowwise) or [k][mn] (columnwise).
struct GemmOperand {
  const uint8_t* codes;
  int64_t ld;
  const uint8_t* scale;
  int64_t mn;
  int32_t colwise;
  int32_t block;       // 128 or 32
  int32_t aligned;     // base and row stride are multiples of 16 bytes
};

struct GemmParams {
  GemmOperand a, b;
  int64_t m, n, k;
  const float* addend;  // [m][ld_c] or nullptr
  int64_t ld_c;
  void* out;            // [m][ld_o]
  int64_t ld_o;
  int32_t out_f32;      // else BF16
  int32_t vec_out;      // out (and addend) rows start on 16-byte boundaries
};

struct NormForwardParams {
  const void* x;
  int64_t rows, cols, ld_x;
  const void* weight;
  const void* bias;     // or nullptr
  void* y;
  int64_t ld_y;
  float* mean;
  float* rstd;
  float eps;
  int32_t vec;          // rows of x and y, weight and bias start on 16-byte boundaries
};

struct NormBackwardParams {
  const void* dy;
  int64_t rows, cols, ld_dy;
  const void* x;
  int64_t ld_x;
  const uint8_t* x_scale;  // GEMM layout; x holds E4M3 codes when not nullptr
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  int64_t ld_dx;
  float* dweight;
  float* dbias;            // or nullptr
  float* workspace;
  int32_t vec;             // every row starts on a vector boundary
};

cudaError_t launch_checkpoint_save(const CheckpointSaveParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_checkpoint_restore(const CheckpointRestoreParams& p, int dtype, cudaStream_t stream);
// *what names the step that failed when it is not the launch itself.
cudaError_t launch_gemm(const GemmParams& p, const DeviceInfo& dev, cudaStream_t stream,
                        const char** what);
// dtype: of x / dy; wdtype: of weight and bias (0 = F32, 1 = BF16).
cudaError_t launch_norm_forward(const NormForwardParams& p, int dtype, int wdtype,
                                const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormBackwardParams& p, int dtype, int wdtype,
                                 const DeviceInfo& dev, cudaStream_t stream);
// Rows of partial sums (2 * cols floats each) that the backward pass leaves, at most.
int64_t norm_partials(int64_t rows, int64_t cols);

}  // namespace mxfp8
