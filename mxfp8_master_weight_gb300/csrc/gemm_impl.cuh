// Pieces shared by the block-scaled product kernels: tile order, scale tiles, epilogue.
#pragma once

#include "common.cuh"
#include "linear.h"
#include "tensor_core.cuh"

namespace mxfp8 {

constexpr int kBlockK = 128;           // values of k per pipeline stage: one 128-byte row
constexpr int kScaleTile = 512;        // bytes of a 128x4 scale tile
constexpr int kBoxBytes = 128 * 128;   // 128 rows of 128 bytes

// Tile (row, column) of the index-th tile: bands of kBand tile rows, walked column by column, so
// that tiles in flight at one time share operand rows and columns in L2.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_at(int64_t index, int64_t tiles_m, int64_t tiles_n, int64_t& tm, int64_t& tn) {
  const int64_t per_band = kBand * tiles_n;
  const int64_t band = index / per_band, in = index - band * per_band;
  const int64_t h = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
  tn = in / h;
  tm = band * kBand + (in - tn * h);
}

// Stage kb of k: the scale tile (along k) that holds its scales, and the byte of the tile's four
// that the j-th 32 values take.  With 32 values per scale a tile is one stage; with 128 it is four.
__device__ __forceinline__ int64_t scale_tile_of(int64_t kb, int block) { return block == 32 ? kb : kb >> 2; }
__device__ __forceinline__ uint32_t scale_id_of(int64_t kb, int j, int block) {
  return block == 32 ? uint32_t(j) : uint32_t(kb & 3);
}
__host__ __device__ inline int64_t scale_tiles_along_k(int64_t k, int block) {
  return scale_tile_cols((k + block - 1) / block);
}

// Writes 32 sums of one output row at columns col .. col + 31 (those below n).
__device__ __forceinline__ void store_row32(const GemmParams& p, int64_t row, int64_t col, float (&v)[32]) {
  if (row >= p.m || col >= p.n) return;
  const bool vec = p.vec_out && col + 32 <= p.n;
  if (p.addend != nullptr) {
    const float* c = p.addend + row * p.ld_c + col;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(c + i);
        v[i] += a.x; v[i + 1] += a.y; v[i + 2] += a.z; v[i + 3] += a.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i < p.n) v[i] += c[i];
    }
  }
  if (p.out_f32) {
    float* o = static_cast<float*>(p.out) + row * p.ld_o + col;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i < p.n) o[i] = v[i];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + row * p.ld_o + col;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = bf16x2_rn(v[2 * i], v[2 * i + 1]);
    if (vec) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) *reinterpret_cast<uint4*>(o + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i < p.n) o[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  }
}

}  // namespace mxfp8
