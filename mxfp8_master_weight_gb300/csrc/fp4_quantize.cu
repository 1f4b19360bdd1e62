// NVFP4 activations: the largest magnitude of a matrix, its codes and scales along rows and columns from one read,
// the values that a copy stands for; and 4-bit weights laid out for the products.
//
//   S = 2688 / G,  s = E4M3((A / 6) S),  code = E2M1(x (S / s)),  value = code s (1 / S)
//
// with G the tensor's largest magnitude and A that of 16 values; every step is one F32 rounding.  The matrix instruction
// of 4-bit operands reads them with the contraction along their rows only, so the columnwise copy is written
// transposed: row j holds column j's codes.
//
// All of them are streaming passes.  A block of the quantisation owns a tile of 128 x 128: thread (warp w, lane l)
// has rows 16 w + 8 (l / 16) .. + 7 of columns 8 (l % 16) .. + 7, so a row's block of 16 is two lanes, a column's block
// two halves of a warp, and both maxima are one shuffle away.  Column codes pass through shared memory to
// leave as whole 64-byte pieces of the transposed rows.
#include "fp4.cuh"
#include "linear.h"

namespace mxfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;

// Eight elements at p as F32 values; zeros past n.
template <class T>
__device__ __forceinline__ void load8(const char* p, int n, bool vec, float (&v)[8]) {
  if (vec && n >= 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    if constexpr (T::kBytes == 4) {
      const uint4 b = *reinterpret_cast<const uint4*>(p + 16);
      const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = __uint_as_float(w[k]);
        v[4 + k] = __uint_as_float(u[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = k < n ? load_bits<T>(p, k) : 0u;
      v[k] = T::kBytes == 4 ? __uint_as_float(b) : __uint_as_float(b << 16);
    }
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// ------------------------------------------------------------------------------ largest magnitude
// Items of a row's 2048 values (a dense matrix is one row); a block folds its items into one atomic maximum of
// non-negative bit patterns, which order as their values, NaN above infinity.
template <class T>
__global__ void __launch_bounds__(kThreads) k_tensor_amax(const __grid_constant__ Fp4AmaxParams p) {
  __shared__ uint32_t s_max[kThreads / 32];
  grid_dependency_sync();
  const int64_t per_row = (p.cols + 8 * kThreads - 1) / (8 * kThreads), items = per_row * p.rows;
  uint32_t m = 0;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t row = item / per_row, col = (item - row * per_row) * (8 * kThreads) + 8 * threadIdx.x;
    if (col >= p.cols) continue;
    float v[8];
    load8<T>(static_cast<const char*>(p.in) + (row * p.ld + col) * T::kBytes, p.cols - col < 8 ? int(p.cols - col) : 8, p.vec, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, abs_bits(v[k]));
  }
  m = __reduce_max_sync(kFullMask, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, s_max[w]);
    atomicMax(reinterpret_cast<uint32_t*>(p.amax), canonical_nan<F32T>(m));
  }
}

// ------------------------------------------------------------------------------ quantisation
template <class T, bool kRow, bool kCol>
__global__ void __launch_bounds__(kThreads) k_fp4_quantize(const __grid_constant__ Fp4QuantizeParams p) {
  __shared__ float s_mult[128];
  __shared__ __align__(16) uint8_t s_scale[2][1024];
  __shared__ __align__(16) uint32_t s_col[kTile][17];
  grid_dependency_sync();
  const float S = fp4_tensor_scale(*p.amax);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t < 128) s_mult[t] = fp4_multiplier(uint32_t(t), S);
  const int64_t tiles_c = (p.cols + kTile - 1) / kTile;
  const int64_t rb = blockIdx.x / tiles_c, cb = blockIdx.x - rb * tiles_c;
  const int r8 = warp * 16 + (lane >> 4) * 8, c8 = (lane & 15) * 8;
  const int64_t row = rb * kTile + r8, col = cb * kTile + c8;
  const int n = p.cols - col >= 8 ? 8 : (p.cols > col ? int(p.cols - col) : 0);
  const int left = p.rows - row >= 8 ? 8 : (p.rows > row ? int(p.rows - row) : 0);
  float v[8][8];
  const char* src = static_cast<const char*>(p.in) + (row * p.ld + col) * T::kBytes;
#pragma unroll
  for (int i = 0; i < 8; ++i) load8<T>(src + i * p.ld * T::kBytes, i < left ? n : 0, p.vec_in, v[i]);
  __syncthreads();
  if constexpr (kRow) {
    uint8_t* q = p.q_r + row * p.ld_r + (col >> 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, abs_bits(v[i][k]));
      m = max(m, __shfl_xor_sync(kFullMask, m, 1));
      const bool inside = i < left && (col & ~int64_t(15)) < p.cols;
      const uint32_t s = inside ? fp4_block_scale(m, S) : 0u;
      const float f = s_mult[s];
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; k += 2) mul2_rn(v[i][k], v[i][k + 1], f, f, y[k], y[k + 1]);
      const uint32_t codes = fp4_codes(y);
      if ((lane & 1) == 0) {  // block c8 / 16 of row r8 + i
        const int r = r8 + i, b = c8 >> 4;
        s_scale[0][(b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3)] = uint8_t(s);
      }
      if (i < left) {
        if (p.vec_r && n == 8) {
          *reinterpret_cast<uint32_t*>(q + i * p.ld_r) = codes;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (2 * k < n) q[i * p.ld_r + k] = uint8_t(codes >> (8 * k));
        }
      }
    }
  }
  if constexpr (kCol) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i][k]));
      m = max(m, __shfl_xor_sync(kFullMask, m, 16));
      const bool inside = k < n && (row & ~int64_t(15)) < p.rows;
      const uint32_t s = inside ? fp4_block_scale(m, S) : 0u;
      const float f = s_mult[s];
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) mul2_rn(v[i][k], v[i + 1][k], f, f, y[i], y[i + 1]);
      if (lane < 16) {  // block `warp` of transposed row c8 + k
        const int r = c8 + k;
        s_scale[1][(warp >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (warp & 3)] = uint8_t(s);
      }
      s_col[c8 + k][(r8 >> 3) ^ ((c8 >> 5) << 1)] = fp4_codes(y);
    }
  }
  __syncthreads();
  // the tile's scales: two tiles of the layout along k for each direction, if both are there
  const int which = t >> 6, unit = t & 63;
  if (t < 128) {
    const int64_t tile_cols = scale_tile_cols(((which == 0 ? p.cols : p.rows) + 15) / 16);
    const int64_t r128 = which == 0 ? rb : cb, at = 2 * (which == 0 ? cb : rb) + (unit >> 5);
    uint8_t* s = which == 0 ? p.s_r : p.s_c;
    if ((which == 0 ? kRow : kCol) && at < tile_cols)
      *reinterpret_cast<uint4*>(s + (r128 * tile_cols + at) * 512 + (unit & 31) * 16) = *reinterpret_cast<const uint4*>(&s_scale[which][unit * 16]);
  }
  if constexpr (kCol) {
    const int width = p.rows - rb * kTile < kTile ? int(p.rows - rb * kTile + 1) / 2 : kTile / 2;  // bytes of a transposed row
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = (t >> 2) + 64 * h, u = t & 3;
      if (cb * kTile + j >= p.cols) continue;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = s_col[j][(4 * u + k) ^ ((j >> 5) << 1)];
      uint8_t* q = p.q_c + (cb * kTile + j) * p.ld_c + rb * (kTile / 2) + 16 * u;
      if (p.vec_c && 16 * u + 16 <= width) {
        *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (16 * u + k < width) q[k] = uint8_t(w[k >> 2] >> (8 * (k & 3)));
      }
    }
  }
}

// ------------------------------------------------------------------------------ values
// A thread restores blocks of 16: 8 bytes of codes and one scale.
template <class T>
__global__ void __launch_bounds__(kThreads) k_fp4_restore(const __grid_constant__ Fp4RestoreParams p) {
  grid_dependency_sync();
  const float r = __frcp_rn(fp4_tensor_scale(*p.amax));
  const int64_t nb = (p.cols + 15) / 16, per_row = (nb + 31) / 32, tile_cols = scale_tile_cols(nb);
  const int64_t row = (blockIdx.x / per_row) * 8 + (threadIdx.x >> 5), b = (blockIdx.x % per_row) * 32 + (threadIdx.x & 31);
  if (row >= p.rows || b >= nb) return;
  const int n = p.cols - 16 * b < 16 ? int(p.cols - 16 * b) : 16;
  const uint8_t* q = p.q + row * p.ld_q + 8 * b;
  uint32_t w[2] = {0, 0};
  if (p.vec_q && n == 16) {
    const uint2 c = *reinterpret_cast<const uint2*>(q);
    w[0] = c.x;
    w[1] = c.y;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (2 * k < n) w[k >> 2] |= uint32_t(q[k]) << (8 * (k & 3));
  }
  const float s = fp4_scale_value(p.s[scale_at(row, b, tile_cols)] & 0x7fu);
  float v[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t h;
    asm("{ .reg .b8 c; cvt.u8.u32 c, %1; cvt.rn.f16x2.e2m1x2 %0, c; }" : "=r"(h) : "r"(w[k >> 2] >> (8 * (k & 3)) & 0xffu));
    v[2 * k] = __fmul_rn(__fmul_rn(f16_lo(h), s), r);  // the first product is exact
    v[2 * k + 1] = __fmul_rn(__fmul_rn(f16_hi(h), s), r);
  }
  char* out = static_cast<char*>(p.out) + (row * p.ld_o + 16 * b) * T::kBytes;
  if (p.vec_out && n == 16) {
#pragma unroll
    for (int k = 0; k < 16; k += 16 / T::kBytes) {
      if constexpr (T::kBytes == 4)
        *reinterpret_cast<float4*>(out + 4 * k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      else
        *reinterpret_cast<uint4*>(out + 2 * k) = make_uint4(bf16x2_rn(v[k], v[k + 1]), bf16x2_rn(v[k + 2], v[k + 3]),
                                                            bf16x2_rn(v[k + 4], v[k + 5]), bf16x2_rn(v[k + 6], v[k + 7]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k < n) store_bits<T>(out, k, T::kBytes == 4 ? __float_as_uint(v[k]) : bf16x2_rn(v[k], 0.0f));
  }
}

// ------------------------------------------------------------------------------ weights
// Codes [rows][cols] as they lie densely to rows with the contraction along them: as they are, or (kTurn) transposed.
// The same tile and threads as the quantisation's; once per refresh of a weight, so loads are by the byte.
template <bool kTurn>
__global__ void __launch_bounds__(kThreads) k_fp4_lay_out(const __grid_constant__ Fp4LayOutParams p) {
  __shared__ __align__(16) uint32_t s_col[kTile][17];
  grid_dependency_sync();
  const int64_t tiles_c = (p.cols + kTile - 1) / kTile;
  const int64_t rb = blockIdx.x / tiles_c, cb = blockIdx.x - rb * tiles_c;
  const int t = threadIdx.x, lane = t & 31, r8 = (t >> 5) * 16 + (lane >> 4) * 8, c8 = (lane & 15) * 8;
  const int64_t row = rb * kTile + r8, col = cb * kTile + c8;
  uint32_t w[8];  // eight codes of eight rows
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = 0;
    if (row + i >= p.rows) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (col + 2 * k < p.cols) w[i] |= uint32_t(p.q[(row + i) * p.ld_q + (col >> 1) + k]) << (8 * k);
    if constexpr (!kTurn) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + 2 * k < p.cols) p.out[(row + i) * p.ld_o + (col >> 1) + k] = uint8_t(w[i] >> (8 * k));
    }
  }
  if constexpr (kTurn) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t q = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) q |= (w[i] >> (4 * k) & 15u) << (4 * i);
      s_col[c8 + k][(r8 >> 3) ^ ((c8 >> 5) << 1)] = q;
    }
    __syncthreads();
    const int width = p.rows - rb * kTile < kTile ? int(p.rows - rb * kTile + 1) / 2 : kTile / 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = (t >> 2) + 64 * h, u = t & 3;
      if (cb * kTile + j >= p.cols) continue;
      uint8_t* o = p.out + (cb * kTile + j) * p.ld_o + rb * (kTile / 2) + 16 * u;
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (16 * u + k < width) o[k] = uint8_t(s_col[j][(4 * u + (k >> 2)) ^ ((j >> 5) << 1)] >> (8 * (k & 3)));
    }
  }
}

int64_t tiles(int64_t rows, int64_t cols) { return ((rows + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile); }

template <class T>
cudaError_t quantize(const Fp4QuantizeParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned(tiles(p.rows, p.cols)));
  if (p.q_r != nullptr && p.q_c != nullptr) return launch_kernel(k_fp4_quantize<T, true, true>, grid, dim3(kThreads), 0, stream, p);
  if (p.q_r != nullptr) return launch_kernel(k_fp4_quantize<T, true, false>, grid, dim3(kThreads), 0, stream, p);
  return launch_kernel(k_fp4_quantize<T, false, true>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_tensor_amax(const Fp4AmaxParams& p, int dtype, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t items = (p.cols + 8 * kThreads - 1) / (8 * kThreads) * p.rows, most = 8 * int64_t(dev.sms);
  const dim3 grid(unsigned(items < most ? items : most));
  return dtype == 0 ? launch_kernel(k_tensor_amax<F32T>, grid, dim3(kThreads), 0, stream, p)
                    : launch_kernel(k_tensor_amax<BF16T>, grid, dim3(kThreads), 0, stream, p);
}

cudaError_t launch_fp4_quantize(const Fp4QuantizeParams& p, int dtype, cudaStream_t stream) {
  return dtype == 0 ? quantize<F32T>(p, stream) : quantize<BF16T>(p, stream);
}

cudaError_t launch_fp4_restore(const Fp4RestoreParams& p, int dtype, cudaStream_t stream) {
  const int64_t nb = (p.cols + 15) / 16;
  const dim3 grid(unsigned((p.rows + 7) / 8 * ((nb + 31) / 32)));
  return dtype == 0 ? launch_kernel(k_fp4_restore<F32T>, grid, dim3(kThreads), 0, stream, p)
                    : launch_kernel(k_fp4_restore<BF16T>, grid, dim3(kThreads), 0, stream, p);
}

cudaError_t launch_fp4_lay_out(const Fp4LayOutParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned(tiles(p.rows, p.cols)));
  return p.transpose ? launch_kernel(k_fp4_lay_out<true>, grid, dim3(kThreads), 0, stream, p)
                     : launch_kernel(k_fp4_lay_out<false>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace mxfp8
