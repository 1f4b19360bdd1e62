// Layer norm of the rows of a matrix, and its gradients.
//
//   forward    mean = sum x / c,  var = sum (x - mean)^2 / c,  rstd = (var + eps)^-1/2
//              y = (x - mean) rstd w + b
//   backward   xh = (x - mean) rstd,  g = dy w
//              dx = rstd (g - sum g / c - xh sum(g xh) / c)
//              dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Everything between load and store is F32: sums, statistics and the sums over rows; dx and y
// are rounded once.  The variance is the mean squared deviation from the mean (a second pass
// over registers), not a difference of moments, which would cancel for rows far from zero.
//
// Both directions are streaming passes bound by HBM.  A row belongs to one group of threads, which
// holds it in registers between its reductions, so each value is read once: a warp per row
// for up to 1024 columns, else a block per row.  In the backward pass a thread keeps the
// running dw and db of its columns in registers over all rows of its block; a block leaves one
// row of partial sums, and a second kernel adds the partial rows in their order, so
// the sums do not depend on the run.
#include "common.cuh"
#include "linear.h"

namespace mxfp8 {
namespace {

// Eight consecutive values as floats.
struct Eight {
  float v[8];
};

__device__ __forceinline__ void unpack_bf16(const uint4& c, Eight& e) {
  e.v[0] = bf16_lo(c.x); e.v[1] = bf16_hi(c.x); e.v[2] = bf16_lo(c.y); e.v[3] = bf16_hi(c.y);
  e.v[4] = bf16_lo(c.z); e.v[5] = bf16_hi(c.z); e.v[6] = bf16_lo(c.w); e.v[7] = bf16_hi(c.w);
}

// Elements [0, n) of p as floats, zeros past them.
template <class T>
__device__ __forceinline__ Eight load_eight(const void* base, int64_t at, int n, bool vec) {
  const char* p = static_cast<const char*>(base) + at * T::kBytes;
  Eight e;
  if (vec && n >= 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    if constexpr (T::kBytes == 4) {
      const uint4 b = *reinterpret_cast<const uint4*>(p + 16);
      e.v[0] = __uint_as_float(a.x); e.v[1] = __uint_as_float(a.y); e.v[2] = __uint_as_float(a.z);
      e.v[3] = __uint_as_float(a.w); e.v[4] = __uint_as_float(b.x); e.v[5] = __uint_as_float(b.y);
      e.v[6] = __uint_as_float(b.z); e.v[7] = __uint_as_float(b.w);
    } else {
      unpack_bf16(a, e);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = k < n ? load_bits<T>(p, k) : 0u;
      e.v[k] = T::kBytes == 4 ? __uint_as_float(b) : __uint_as_float(b << 16);
    }
  }
  return e;
}

// The same of a weight or bias, of either type.
__device__ __forceinline__ Eight load_param(const void* base, int bf16, int64_t at, int n, bool vec) {
  return bf16 ? load_eight<BF16T>(base, at, n, vec) : load_eight<F32T>(base, at, n, vec);
}

template <class T>
__device__ __forceinline__ void store_eight(void* base, int64_t at, const Eight& e, int n, bool vec) {
  char* p = static_cast<char*>(base) + at * T::kBytes;
  uint32_t w[T::kBytes * 2];
  if constexpr (T::kBytes == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(e.v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = bf16x2_rn(e.v[2 * k], e.v[2 * k + 1]);
  }
  if (vec && n >= 8) {
#pragma unroll
    for (int k = 0; k < T::kBytes * 2; k += 4)
      *reinterpret_cast<uint4*>(p + 4 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) store_bits<T>(p, k, T::kBytes == 4 ? w[k % (T::kBytes * 2)] : w[k >> 1] >> (16 * (k & 1)));
  }
}

// E4M3 codes [0, n) of p as floats times f.
__device__ __forceinline__ Eight load_codes(const uint8_t* p, int n, bool vec, float f) {
  uint2 q = make_uint2(0, 0);
  if (vec && n >= 8) {
    q = *reinterpret_cast<const uint2*>(p);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = k < n ? p[k] : 0u;
      if (k < 4) q.x |= b << (8 * k); else q.y |= b << (8 * (k - 4));
    }
  }
  Eight e;
  const uint32_t pair[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair[k])));
    e.v[2 * k] = f16_lo(h) * f;
    e.v[2 * k + 1] = f16_hi(h) * f;
  }
  return e;
}

// 2^(s - 127) of the rowwise checkpoint scale of (row, column); NaN for 255.
__device__ __forceinline__ float checkpoint_scale(const uint8_t* s, int64_t row, int64_t col, int64_t cols) {
  const int64_t b = col / kCkptBlock, tcols = scale_tile_cols((cols + kCkptBlock - 1) / kCkptBlock);
  const uint32_t v = s[((row >> 7) * tcols + (b >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (b & 3)];
  return __uint_as_float(v == 255u ? 0x7fc00000u : (v == 0u ? 0x00400000u : v << 23));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFullMask, v, off);
  return v;
}

// Sums of N values over the group that owns a row: the warp, or (kBlock) the whole block, whose
// warps meet in `buf` (a row of 32 per value).  `buf` alternates between two halves, so one
// barrier per sum keeps a warp from overwriting what another still reads.
template <bool kBlock, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* buf, int& half) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if constexpr (kBlock) {
    float* b = buf + half * (N * 32);
    half ^= 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) b[k * 32 + warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < nw ? b[k * 32 + lane] : 0.0f);
  }
}

__device__ __forceinline__ int valid(int64_t cols, int64_t col) {
  return cols - col >= 8 ? 8 : (cols > col ? int(cols - col) : 0);
}

// ------------------------------------------------------------------------------ forward
// A row in registers: NV pieces of 8 columns per thread.
template <class T, bool kBlock, int NV>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) k_norm_forward(const __grid_constant__ NormForwardParams p,
                                                                      int wbf16) {
  __shared__ float buf[2][32];
  grid_dependency_sync();
  const int width = kBlock ? blockDim.x : 32;
  const int lane = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int64_t row = kBlock ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.rows) return;  // whole warps only
  int half = 0;
  Eight x[NV];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = int64_t(lane + i * width) * 8;
    x[i] = load_eight<T>(p.x, row * p.ld_x + col, valid(p.cols, col), p.vec);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += x[i].v[k];
  group_sum<kBlock>(s, &buf[0][0], half);
  const float mean = s[0] / float(p.cols);
  s[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int n = valid(p.cols, int64_t(lane + i * width) * 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[i].v[k] = k < n ? x[i].v[k] - mean : 0.0f;
      s[0] += x[i].v[k] * x[i].v[k];
    }
  }
  group_sum<kBlock>(s, &buf[0][0], half);
  const float rstd = __frsqrt_rn(s[0] / float(p.cols) + p.eps);
  if (lane == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = int64_t(lane + i * width) * 8;
    const int n = valid(p.cols, col);
    if (n == 0) continue;
    const Eight w = load_param(p.weight, wbf16, col, n, p.vec);
    Eight y;
    if (p.bias != nullptr) {
      const Eight b = load_param(p.bias, wbf16, col, n, p.vec);
#pragma unroll
      for (int k = 0; k < 8; ++k) y.v[k] = x[i].v[k] * rstd * w.v[k] + b.v[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) y.v[k] = x[i].v[k] * rstd * w.v[k];
    }
    store_eight<T>(p.y, row * p.ld_y + col, y, n, p.vec);
  }
}

// Rows too long for registers: three passes over the row, the later ones mostly from L2.
template <class T>
__global__ void __launch_bounds__(1024) k_norm_forward_long(const __grid_constant__ NormForwardParams p, int wbf16) {
  __shared__ float buf[2][32];
  grid_dependency_sync();
  const int64_t row = blockIdx.x;
  int half = 0;
  const int64_t step = int64_t(blockDim.x) * 8;
  float s[1] = {0.0f};
  for (int64_t col = int64_t(threadIdx.x) * 8; col < p.cols; col += step) {
    const Eight x = load_eight<T>(p.x, row * p.ld_x + col, valid(p.cols, col), p.vec);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += x.v[k];
  }
  group_sum<true>(s, &buf[0][0], half);
  const float mean = s[0] / float(p.cols);
  s[0] = 0.0f;
  for (int64_t col = int64_t(threadIdx.x) * 8; col < p.cols; col += step) {
    const int n = valid(p.cols, col);
    const Eight x = load_eight<T>(p.x, row * p.ld_x + col, n, p.vec);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = k < n ? x.v[k] - mean : 0.0f;
      s[0] += d * d;
    }
  }
  group_sum<true>(s, &buf[0][0], half);
  const float rstd = __frsqrt_rn(s[0] / float(p.cols) + p.eps);
  if (threadIdx.x == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
  for (int64_t col = int64_t(threadIdx.x) * 8; col < p.cols; col += step) {
    const int n = valid(p.cols, col);
    const Eight x = load_eight<T>(p.x, row * p.ld_x + col, n, p.vec);
    const Eight w = load_param(p.weight, wbf16, col, n, p.vec);
    Eight y;
#pragma unroll
    for (int k = 0; k < 8; ++k) y.v[k] = (x.v[k] - mean) * rstd * w.v[k];
    if (p.bias != nullptr) {
      const Eight b = load_param(p.bias, wbf16, col, n, p.vec);
#pragma unroll
      for (int k = 0; k < 8; ++k) y.v[k] += b.v[k];
    }
    store_eight<T>(p.y, row * p.ld_y + col, y, n, p.vec);
  }
}

// ------------------------------------------------------------------------------ backward
// The saved input: values, or the codes of a checkpoint.
template <class T, bool kCodes>
__device__ __forceinline__ Eight load_input(const NormBackwardParams& p, int64_t row, int64_t col, int n) {
  if constexpr (kCodes) {
    const float f = n > 0 ? checkpoint_scale(p.x_scale, row, col, p.cols) : 0.0f;
    return load_codes(static_cast<const uint8_t*>(p.x) + row * p.ld_x + col, n, p.vec, f);
  } else {
    return load_eight<T>(p.x, row * p.ld_x + col, n, p.vec);
  }
}

template <class T, bool kCodes, bool kBlock, int NV>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) k_norm_backward(const __grid_constant__ NormBackwardParams p,
                                                                       int wbf16) {
  __shared__ float buf[2][2 * 32];
  extern __shared__ float s_acc[];  // warp per row: [8 warps][cols of dw, then db], padded to 8
  grid_dependency_sync();
  const int width = kBlock ? blockDim.x : 32;
  const int lane = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  int half = 0;
  const float inv = 1.0f / float(p.cols);
  float dw[NV][8], db[NV][8];
  Eight w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t col = int64_t(lane + i * width) * 8;
    w[i] = load_param(p.weight, wbf16, col, valid(p.cols, col), p.vec);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = db[i][k] = 0.0f;
  }
  const int64_t first = kBlock ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 8 + warp;
  const int64_t step = kBlock ? int64_t(gridDim.x) : int64_t(gridDim.x) * 8;
  for (int64_t row = first; row < p.rows; row += step) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    Eight dy[NV], xh[NV];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = int64_t(lane + i * width) * 8;
      const int n = valid(p.cols, col);
      dy[i] = load_eight<T>(p.dy, row * p.ld_dy + col, n, p.vec);
      xh[i] = load_input<T, kCodes>(p, row, col, n);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // columns past the last: dy = w = 0, so nothing enters the sums
        xh[i].v[k] = (xh[i].v[k] - mean) * rstd;
        const float g = dy[i].v[k] * w[i].v[k];
        s[0] += g;
        s[1] += g * xh[i].v[k];
        dw[i][k] += dy[i].v[k] * xh[i].v[k];
        db[i][k] += dy[i].v[k];
      }
    }
    group_sum<kBlock>(s, &buf[0][0], half);
    const float mg = s[0] * inv, mgx = s[1] * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = int64_t(lane + i * width) * 8;
      const int n = valid(p.cols, col);
      if (n == 0) continue;
      Eight dx;
#pragma unroll
      for (int k = 0; k < 8; ++k) dx.v[k] = rstd * (dy[i].v[k] * w[i].v[k] - mg - xh[i].v[k] * mgx);
      store_eight<T>(p.dx, row * p.ld_dx + col, dx, n, p.vec);
    }
  }
  // one row of partial sums per block: [blocks][2][cols]
  float* out = p.workspace + int64_t(blockIdx.x) * 2 * p.cols;
  if constexpr (kBlock) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t col = int64_t(lane + i * width) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (col + k < p.cols) {
          out[col + k] = dw[i][k];
          out[p.cols + col + k] = db[i][k];
        }
      }
    }
  } else {
    const int pc = int((p.cols + 7) / 8 * 8);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (lane + i * 32) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (col < pc) {
          s_acc[warp * 2 * pc + col + k] = dw[i][k];
          s_acc[warp * 2 * pc + pc + col + k] = db[i][k];
        }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * pc; c += blockDim.x) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v += s_acc[k * 2 * pc + c];
      const int col = c < pc ? c : c - pc;
      if (col < p.cols) out[(c < pc ? 0 : p.cols) + col] = v;
    }
  }
}

// Rows too long for registers: two passes over the row; the block's partial sums live in
// its workspace row (each entry touched by one thread only).
template <class T, bool kCodes>
__global__ void __launch_bounds__(1024) k_norm_backward_long(const __grid_constant__ NormBackwardParams p, int wbf16) {
  __shared__ float buf[2][2 * 32];
  grid_dependency_sync();
  int half = 0;
  const float inv = 1.0f / float(p.cols);
  float* out = p.workspace + int64_t(blockIdx.x) * 2 * p.cols;
  const int64_t step = int64_t(blockDim.x) * 8;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const bool first = row == blockIdx.x;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s[2] = {0.0f, 0.0f};
    for (int64_t col = int64_t(threadIdx.x) * 8; col < p.cols; col += step) {
      const int n = valid(p.cols, col);
      const Eight dy = load_eight<T>(p.dy, row * p.ld_dy + col, n, p.vec);
      const Eight x = load_input<T, kCodes>(p, row, col, n);
      const Eight w = load_param(p.weight, wbf16, col, n, p.vec);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = (x.v[k] - mean) * rstd, g = dy.v[k] * w.v[k];
        s[0] += g;
        s[1] += g * xh;
        if (k < n) {
          out[col + k] = dy.v[k] * xh + (first ? 0.0f : out[col + k]);
          out[p.cols + col + k] = dy.v[k] + (first ? 0.0f : out[p.cols + col + k]);
        }
      }
    }
    group_sum<true>(s, &buf[0][0], half);
    const float mg = s[0] * inv, mgx = s[1] * inv;
    for (int64_t col = int64_t(threadIdx.x) * 8; col < p.cols; col += step) {
      const int n = valid(p.cols, col);
      const Eight dy = load_eight<T>(p.dy, row * p.ld_dy + col, n, p.vec);
      const Eight x = load_input<T, kCodes>(p, row, col, n);
      const Eight w = load_param(p.weight, wbf16, col, n, p.vec);
      Eight dx;
#pragma unroll
      for (int k = 0; k < 8; ++k) dx.v[k] = rstd * (dy.v[k] * w.v[k] - mg - (x.v[k] - mean) * rstd * mgx);
      store_eight<T>(p.dx, row * p.ld_dx + col, dx, n, p.vec);
    }
  }
}

// Adds the partial rows in their order: a block owns 32 entries of [2][cols], its 8 warps an
// eighth of the rows each, added up through shared memory.
__global__ void __launch_bounds__(256) k_norm_partials(const float* __restrict__ part, int nparts, int64_t cols,
                                                       float* dweight, float* dbias) {
  __shared__ float s[8][32];
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t e = int64_t(blockIdx.x) * 32 + lane;
  const int lo = nparts * warp / 8, hi = nparts * (warp + 1) / 8;
  float v = 0.0f;
  if (e < 2 * cols) {
#pragma unroll 8
    for (int r = lo; r < hi; ++r) v += part[int64_t(r) * 2 * cols + e];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && e < 2 * cols) {
    v = s[0][lane];
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][lane];
    if (e < cols) dweight[e] = v;
    else if (dbias != nullptr) dbias[e - cols] = v;
  }
}

// How a row is spread: a warp per row up to 1024 columns, else a block per row with nv pieces of 8
// columns per thread; 0: the row does not fit in registers.
struct Spread {
  bool block;
  int nv, threads;
};
Spread spread_of(int64_t cols, int max_nv) {
  const int64_t pieces = (cols + 7) / 8;
  if (pieces <= 128) {
    const int nv = pieces <= 32 ? 1 : (pieces <= 64 ? 2 : 4);
    return {false, nv, 256};
  }
  for (int nv = 1; nv <= max_nv; nv *= 2) {
    const int64_t t = (pieces + nv - 1) / nv;
    if (t <= (nv == max_nv ? 1024 : 512)) return {true, nv, int((t + 31) / 32 * 32)};
  }
  return {true, 0, 1024};
}

template <class T>
cudaError_t forward(const NormForwardParams& p, int wdtype, cudaStream_t stream) {
  const Spread s = spread_of(p.cols, 4);
  const dim3 block(s.threads);
  if (!s.block) {
    const dim3 grid(static_cast<unsigned>((p.rows + 7) / 8));
    if (s.nv == 1) return launch_kernel(k_norm_forward<T, false, 1>, grid, block, 0, stream, p, wdtype);
    if (s.nv == 2) return launch_kernel(k_norm_forward<T, false, 2>, grid, block, 0, stream, p, wdtype);
    return launch_kernel(k_norm_forward<T, false, 4>, grid, block, 0, stream, p, wdtype);
  }
  const dim3 grid(static_cast<unsigned>(p.rows));
  if (s.nv == 1) return launch_kernel(k_norm_forward<T, true, 1>, grid, block, 0, stream, p, wdtype);
  if (s.nv == 2) return launch_kernel(k_norm_forward<T, true, 2>, grid, block, 0, stream, p, wdtype);
  if (s.nv == 4) return launch_kernel(k_norm_forward<T, true, 4>, grid, block, 0, stream, p, wdtype);
  return launch_kernel(k_norm_forward_long<T>, grid, block, 0, stream, p, wdtype);
}

template <class T, bool kCodes>
cudaError_t backward(const NormBackwardParams& p, int wdtype, cudaStream_t stream) {
  const Spread s = spread_of(p.cols, 2);
  const dim3 block(s.threads), grid(static_cast<unsigned>(norm_partials(p.rows, p.cols)));
  cudaError_t e;
  if (!s.block) {
    const size_t smem = size_t(8) * 2 * size_t((p.cols + 7) / 8 * 8) * 4;
    auto run = [&](auto kernel) {
      const cudaError_t a = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, 65536);
      return a != cudaSuccess ? a : launch_kernel(kernel, grid, block, smem, stream, p, wdtype);
    };
    e = s.nv == 1 ? run(k_norm_backward<T, kCodes, false, 1>)
                  : (s.nv == 2 ? run(k_norm_backward<T, kCodes, false, 2>) : run(k_norm_backward<T, kCodes, false, 4>));
  } else if (s.nv == 1) {
    e = launch_kernel(k_norm_backward<T, kCodes, true, 1>, grid, block, 0, stream, p, wdtype);
  } else if (s.nv == 2) {
    e = launch_kernel(k_norm_backward<T, kCodes, true, 2>, grid, block, 0, stream, p, wdtype);
  } else {
    e = launch_kernel(k_norm_backward_long<T, kCodes>, grid, block, 0, stream, p, wdtype);
  }
  if (e != cudaSuccess) return e;
  const dim3 rgrid(static_cast<unsigned>((2 * p.cols + 31) / 32));
  return launch_kernel(k_norm_partials, rgrid, dim3(256), 0, stream, static_cast<const float*>(p.workspace),
                       int(grid.x), p.cols, p.dweight, p.dbias);
}

}  // namespace

int64_t norm_partials(int64_t rows, int64_t cols) {
  const int64_t blocks = spread_of(cols, 2).block ? rows : (rows + 7) / 8;
  return blocks < kNormMaxPartials ? blocks : kNormMaxPartials;
}

cudaError_t launch_norm_forward(const NormForwardParams& p, int dtype, int wdtype, const DeviceInfo&,
                                cudaStream_t stream) {
  return dtype == 0 ? forward<F32T>(p, wdtype, stream) : forward<BF16T>(p, wdtype, stream);
}

cudaError_t launch_norm_backward(const NormBackwardParams& p, int dtype, int wdtype, const DeviceInfo&,
                                 cudaStream_t stream) {
  const bool codes = p.x_scale != nullptr;
  if (dtype == 0) return codes ? backward<F32T, true>(p, wdtype, stream) : backward<F32T, false>(p, wdtype, stream);
  return codes ? backward<BF16T, true>(p, wdtype, stream) : backward<BF16T, false>(p, wdtype, stream);
}

}  // namespace mxfp8
