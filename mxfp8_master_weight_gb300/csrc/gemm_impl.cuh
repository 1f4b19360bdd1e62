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

// Writes 128 bytes of each of 32 output rows (32 F32 or 64 BF16 columns) that a warp holds a row per
// lane.  A store straight from there would touch 32 lines for 512 bytes; through 4 KB of
// shared memory of the warp's own (16-byte unit c of row r at c ^ (r % 8)) every store fills
// four whole lines (3 us less for 4096^3 with BF16 output, 34 us for 8192^3 with F32 output).
// `sums` is called with the first of 32 columns and gives this lane's row.
template <class Sums>
__device__ __forceinline__ void write_rows(const GemmParams& p, char* stage, int64_t row0, int64_t col, Sums sums) {
  const int lane = threadIdx.x & 31, unit = lane & 7;
  const int width = p.out_f32 ? 32 : 64;
  const bool vec = p.vec_out && col + width <= p.n;
  const bool add = p.out_f32 && p.addend != nullptr;
  const int rows = p.m - row0 < 32 ? int(p.m - row0) : 32;
  float c[32];  // the addend's values, on their way before the sums are: as they will be stored
  if (add && vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r < rows) a = *reinterpret_cast<const float4*>(p.addend + (row0 + r) * p.ld_c + col + 4 * unit);
      c[4 * i] = a.x; c[4 * i + 1] = a.y; c[4 * i + 2] = a.z; c[4 * i + 3] = a.w;
    }
  } else if (add) {
    const float* a = p.addend + row0 * p.ld_c + col + lane;
#pragma unroll
    for (int r = 0; r < 32; ++r, a += p.ld_c) c[r] = r < rows && col + lane < p.n ? *a : 0.0f;
  }
  if (p.out_f32) {
    float v[32];
    sums(0, v);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      *reinterpret_cast<float4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
      sums(32 * h, v);
      if (p.addend != nullptr && row0 + lane < p.m) {  // before the rounding
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + 32 * h + i < p.n) v[i] += p.addend[(row0 + lane) * p.ld_c + col + 32 * h + i];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * h + u) ^ (lane & 7)) << 4)) =
            make_uint4(bf16x2_rn(v[8 * u], v[8 * u + 1]), bf16x2_rn(v[8 * u + 2], v[8 * u + 3]),
                       bf16x2_rn(v[8 * u + 4], v[8 * u + 5]), bf16x2_rn(v[8 * u + 6], v[8 * u + 7]));
    }
  }
  __syncwarp();
  if (vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      if (r >= rows) continue;
      uint4 w = *reinterpret_cast<const uint4*>(stage + r * 128 + ((unit ^ (r & 7)) << 4));
      if (p.out_f32) {
        if (add)
          w = make_uint4(__float_as_uint(__uint_as_float(w.x) + c[4 * i]), __float_as_uint(__uint_as_float(w.y) + c[4 * i + 1]),
                         __float_as_uint(__uint_as_float(w.z) + c[4 * i + 2]), __float_as_uint(__uint_as_float(w.w) + c[4 * i + 3]));
        *reinterpret_cast<uint4*>(static_cast<float*>(p.out) + (row0 + r) * p.ld_o + col + 4 * unit) = w;
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (row0 + r) * p.ld_o + col + 8 * unit) = w;
      }
    }
  } else {  // rows that start anywhere, or end inside: an element per lane
    const bool in0 = col + lane < p.n, in1 = !p.out_f32 && col + 32 + lane < p.n;
    if (p.out_f32) {
      float* o = static_cast<float*>(p.out) + row0 * p.ld_o + col + lane;
#pragma unroll
      for (int r = 0; r < 32; ++r, o += p.ld_o) {
        const float v = *reinterpret_cast<const float*>(stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3));
        if (r < rows && in0) *o = add ? v + c[r] : v;
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(p.out) + row0 * p.ld_o + col + lane;
#pragma unroll 8
      for (int r = 0; r < 32; ++r, o += p.ld_o) {
        const char* line = stage + r * 128 + 2 * (lane & 7);
        const uint16_t v0 = *reinterpret_cast<const uint16_t*>(line + (((lane >> 3) ^ (r & 7)) << 4));
        const uint16_t v1 = *reinterpret_cast<const uint16_t*>(line + (((4 + (lane >> 3)) ^ (r & 7)) << 4));
        if (r < rows && in0) o[0] = v0;
        if (r < rows && in1) o[32] = v1;
      }
    }
  }
  __syncwarp();
}

}  // namespace mxfp8
