// TMA descriptors of a product's operands and scales (host code).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "linear.h"

namespace mxfp8 {

// Boxes of `rows` stored rows by 128 bytes under the 128-byte swizzle; zeros past the matrix.
cudaError_t operand_map(const GemmOperand& o, int64_t k, int rows, CUtensorMap* map, const char** what);
// Boxes of half as many m or n: 64 rows by 128 bytes, or (columnwise) 128 rows by 64 bytes under the
// 64-byte swizzle.
cudaError_t half_operand_map(const GemmOperand& o, int64_t k, CUtensorMap* map, const char** what);
// 16 maps of an operand that is not aligned: map s has the rows 16 q + s, in boxes of 8 rows by 160
// bytes from the 16-byte unit that holds a row's first byte.
cudaError_t residue_maps(const GemmOperand& o, int64_t k, CUtensorMap* maps, const char** what);
// Boxes of `row_tiles` 512-byte scale tiles, one above the other, by `k_tiles` along k: coordinates (0, tile along k,
// 128-row block); zeros past them.
cudaError_t scale_map(const GemmOperand& o, int64_t k, int row_tiles, CUtensorMap* map, const char** what, int k_tiles = 1);

// Boxes of 32 rows by 128 bytes of the output under the 128-byte swizzle, for stores; its rows start and end on 16 bytes.
cudaError_t output_map(const GemmParams& g, CUtensorMap* map, const char** what);

// The kernels, for operands of any alignment.
cudaError_t launch_gemm_pair(const GemmParams& g, unsigned* given_up, const DeviceInfo& dev, cudaStream_t stream,
                             const char** what);
cudaError_t launch_gemm_split(const GemmParams& g, unsigned* given_up, const DeviceInfo& dev, cudaStream_t stream,
                              const char** what);

}  // namespace mxfp8
