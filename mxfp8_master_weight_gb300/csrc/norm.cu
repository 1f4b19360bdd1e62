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
// Both directions read every value once.  Many rows of up to 8192 columns go through rings of bulk copies
// in persistent blocks (below); few rows, or longer ones, belong to one group of threads each, which
// holds the row in registers between its reductions: a warp for up to 1024 columns, else a block; beyond
// 32768 columns (16384 backward) the row is read again, mostly from L2.  In the backward pass a
// thread keeps the running dw and db of its columns in registers over all rows of its block; a block
// leaves one row of partial sums, and a second kernel adds the partial rows in their order, so the
// sums do not depend on the run.
//
// Measured at 16384 x 6144: forward BF16 62 us (6.5 TB/s, bound by HBM), backward BF16 99 us (6.1 TB/s), from
// an 8-bit checkpoint 95 us for 504 MB: there decoding and two passes of arithmetic over the row take 56 %
// of the issue slots at 16 warps per SM.  1 x 4096 forward: 4.6 us, the time of a call.  Beyond 8192 columns, 4096 x
// 12288 BF16: forward 80 us (2.5 TB/s), backward 185, from a checkpoint 198; a block owns a row and has nothing
// under way for the next one, and at 1024 threads the backward kernel spills 212 to 348 bytes per thread.
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "linear.h"
#include "status.h"
#include "tensor_core.cuh"

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
__device__ __forceinline__ Eight load_codes(const uint8_t* p, int n, bool vec, float f = 1.0f) {
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

// 2^(v - 127); NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t v) {
  return __uint_as_float(v == 255u ? 0x7fc00000u : (v == 0u ? 0x00400000u : v << 23));
}
// That of the rowwise checkpoint scale of (row, column).
__device__ __forceinline__ float checkpoint_scale(const uint8_t* s, int64_t row, int64_t col, int64_t cols) {
  const int64_t b = col / kCkptBlock, tcols = scale_tile_cols((cols + kCkptBlock - 1) / kCkptBlock);
  return scale_value(s[((row >> 7) * tcols + (b >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (b & 3)]);
}

// Two F32 operations in one instruction.
struct Two {
  uint64_t v;
  __device__ __forceinline__ Two() {}
  __device__ __forceinline__ Two(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ explicit Two(float both) : Two(both, both) {}
  __device__ __forceinline__ void get(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};
__device__ __forceinline__ Two operator*(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
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
// The columns of a thread's pieces.  Where the columns are a multiple of 8: 8 neighbours per piece,
// one or two 16-byte loads of an aligned row.  Else (rows then start anywhere): neighbours across
// the threads, so that single loads and stores still fill whole sectors.  The choice goes by the
// shape alone, so that few rows give the same bits whatever the alignment of a buffer.
template <bool kVec>
struct Columns {
  int64_t cols;
  int lane, width;
  bool aligned;
  __device__ __forceinline__ int64_t at(int i, int k) const {
    return kVec ? int64_t(lane + i * width) * 8 + k : int64_t(i * 8 + k) * width + lane;
  }
  __device__ __forceinline__ bool in(int i, int k) const { return at(i, k) < cols; }
  template <class T>
  __device__ __forceinline__ Eight load(const void* base, int64_t row, int i) const {
    if constexpr (kVec) {
      return load_eight<T>(base, row + at(i, 0), valid(cols, at(i, 0)), aligned);
    } else {
      Eight e;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t b = in(i, k) ? load_bits<T>(base, row + at(i, k)) : 0u;
        e.v[k] = T::kBytes == 4 ? __uint_as_float(b) : __uint_as_float(b << 16);
      }
      return e;
    }
  }
  __device__ __forceinline__ Eight param(const void* base, int bf16, int i) const {
    return bf16 ? load<BF16T>(base, 0, i) : load<F32T>(base, 0, i);
  }
  template <class T>
  __device__ __forceinline__ void store(void* base, int64_t row, int i, const Eight& e) const {
    if constexpr (kVec) {
      store_eight<T>(base, row + at(i, 0), e, valid(cols, at(i, 0)), aligned);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (in(i, k)) store_bits<T>(base, row + at(i, k), T::kBytes == 4 ? __float_as_uint(e.v[k]) : bf16x2_rn(e.v[k], 0.0f));
    }
  }
};

// A row in registers: NV pieces of 8 columns per thread.
template <class T, bool kBlock, bool kVec, int NV>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) k_norm_forward(const __grid_constant__ NormForwardParams p,
                                                                      int wbf16) {
  __shared__ float buf[2][32];
  grid_dependency_sync();
  const Columns<kVec> c{p.cols, int(kBlock ? threadIdx.x : threadIdx.x & 31), int(kBlock ? blockDim.x : 32), p.vec != 0};
  const int64_t row = kBlock ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.rows) return;  // whole warps only
  int half = 0;
  Eight x[NV];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = c.template load<T>(p.x, row * p.ld_x, i);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += x[i].v[k];
  group_sum<kBlock>(s, &buf[0][0], half);
  const float mean = s[0] / float(p.cols);
  s[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[i].v[k] = c.in(i, k) ? x[i].v[k] - mean : 0.0f;
      s[0] += x[i].v[k] * x[i].v[k];
    }
  }
  group_sum<kBlock>(s, &buf[0][0], half);
  const float rstd = __frsqrt_rn(s[0] / float(p.cols) + p.eps);
  if (c.lane == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!c.in(i, 0)) continue;
    const Eight w = c.param(p.weight, wbf16, i);
    Eight b = {}, y;
    if (p.bias != nullptr) b = c.param(p.bias, wbf16, i);
#pragma unroll
    for (int k = 0; k < 8; ++k) y.v[k] = x[i].v[k] * rstd * w.v[k] + b.v[k];
    c.template store<T>(p.y, row * p.ld_y, i, y);
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

template <class T, bool kCodes, bool kVec>
__device__ __forceinline__ Eight load_input(const NormBackwardParams& p, const Columns<kVec>& c, int64_t row, int i) {
  if constexpr (kVec) {
    return load_input<T, kCodes>(p, row, c.at(i, 0), valid(p.cols, c.at(i, 0)));
  } else if constexpr (kCodes) {
    const uint8_t* q = static_cast<const uint8_t*>(p.x) + row * p.ld_x;
    Eight e;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const bool in0 = c.in(i, k), in1 = c.in(i, k + 1);
      const uint32_t two = (in0 ? q[c.at(i, k)] : 0u) | (in1 ? uint32_t(q[c.at(i, k + 1)]) << 8 : 0u);
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
      e.v[k] = in0 ? f16_lo(h) * checkpoint_scale(p.x_scale, row, c.at(i, k), p.cols) : 0.0f;
      e.v[k + 1] = in1 ? f16_hi(h) * checkpoint_scale(p.x_scale, row, c.at(i, k + 1), p.cols) : 0.0f;
    }
    return e;
  } else {
    return c.template load<T>(p.x, row * p.ld_x, i);
  }
}

template <class T, bool kCodes, bool kBlock, bool kVec, int NV>
__global__ void __launch_bounds__(kBlock ? (NV == 1 ? 512 : 1024) : 256)
    k_norm_backward(const __grid_constant__ NormBackwardParams p, int wbf16) {
  __shared__ float buf[2][2 * 32];
  extern __shared__ float s_acc[];  // warp per row: [8 warps][dw of the columns, then db]
  grid_dependency_sync();
  const Columns<kVec> c{p.cols, int(kBlock ? threadIdx.x : threadIdx.x & 31), int(kBlock ? blockDim.x : 32), p.vec != 0};
  const int warp = threadIdx.x >> 5;
  int half = 0;
  const float inv = 1.0f / float(p.cols);
  float dw[NV][8], db[NV][8];
  Eight w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i] = c.param(p.weight, wbf16, i);
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
      dy[i] = c.template load<T>(p.dy, row * p.ld_dy, i);
      xh[i] = load_input<T, kCodes, kVec>(p, c, row, i);
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
      if (!c.in(i, 0)) continue;
      Eight dx;
#pragma unroll
      for (int k = 0; k < 8; ++k) dx.v[k] = rstd * (dy[i].v[k] * w[i].v[k] - mg - xh[i].v[k] * mgx);
      c.template store<T>(p.dx, row * p.ld_dx, i, dx);
    }
  }
  // one row of partial sums per block: [blocks][2][cols]
  float* out = p.workspace + int64_t(blockIdx.x) * 2 * p.cols;
  const int cols = int(p.cols);
  float* mine = kBlock ? out : s_acc + warp * 2 * cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (c.in(i, k)) {
        mine[c.at(i, k)] = dw[i][k];
        mine[cols + c.at(i, k)] = db[i][k];
      }
    }
  }
  if constexpr (!kBlock) {
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * cols; e += blockDim.x) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v += s_acc[k * 2 * cols + e];
      out[e] = v;
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

// ------------------------------------------------------------------------------ rings
// Many rows of up to 8192 columns: persistent blocks, each with a ring of rows in shared memory
// that thread 0 (with the statistics: warp 0) keeps full with copies in the background, whatever the
// warps wait for.  A thread owns fixed columns, NV pieces of 8, and keeps what belongs to a column
// (weight, bias, running gradients) in registers over all rows.  A row takes two barriers (one
// backward) of its block; the first of them also says that a slot has been read, and it is refilled.
// Several blocks per SM fill each other's waits, so the blocks are as small as a row allows: TH threads.
constexpr int kRingBytes = 216 * 1024;  // shared memory of an SM that its blocks take
// Rows under way: three per block cover the latency; more bytes than this per SM (23 MB in all) make HBM
// slower (16384 x 6144 backward BF16 with three rows, 147 KB, 99 us, with four 111 us; F32 from codes with two
// rows, 123 KB, 155 us, with three 171 us).  A single block per SM takes what fits (8192 x 8192 BF16 backward
// 80 us with three, 71 with six).
constexpr int kRingFlight = 150 * 1024;
constexpr int kRingMaxSlots = 8;
constexpr int kRingHead = 384;          // barriers and sums

struct Ring {
  int32_t slots, slot_bytes, second;  // rows in flight; bytes of a slot; offset of the second operand
  int32_t side;                       // offset of a row's mean, rstd and scales
  uint32_t smem;
};
// first, second: bytes of a row of each operand (multiples of 16); side: a multiple of 16; blocks: per SM.
Ring ring_of(int64_t first, int64_t second, int side, int blocks) {
  Ring r{};
  r.second = int32_t((first + 127) / 128 * 128);
  r.side = int32_t(r.second + (second + 127) / 128 * 128);
  r.slot_bytes = r.side + side;
  const int fit = (kRingBytes / blocks - 1024 - kRingHead) / r.slot_bytes;  // 1 KB per block is the system's
  const int flight = blocks == 1 ? kRingMaxSlots : kRingFlight / (blocks * r.slot_bytes);
  const int most = blocks == 1 ? kRingMaxSlots : 3;
  r.slots = flight < 2 ? 2 : (flight < most ? flight : most);
  if (fit < r.slots) r.slots = fit;
  r.smem = uint32_t(kRingBytes / blocks - 1024);  // all of it: with room for one more block on an SM another had one less
  return r;
}

struct RingHead {
  uint64_t full[kRingMaxSlots];
  float sums[2][2][16];
};
static_assert(sizeof(RingHead) <= kRingHead, "ring head");

// Sums of N values over the TH threads that own a row.
template <int TH, int N>
__device__ __forceinline__ void ring_sum(float (&v)[N], RingHead* h, int& half) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if constexpr (TH > 32) {
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) h->sums[half][k][threadIdx.x >> 5] = v[k];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(TH) : "memory");
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < TH / 32; w += 2) {
        const float2 a = *reinterpret_cast<const float2*>(&h->sums[half][k][w]);
        t += a.x + a.y;
      }
      v[k] = t;
    }
    half ^= 1;
  }
}

// What thread 0 fetches: rows blockIdx.x, blockIdx.x + gridDim.x, ... of one or two operands, in
// that order, into the slots in turn.  Rows that do not start on 16 bytes (kVec false) land as many bytes
// into their slot as they start into their first 16-byte unit; the units at a row's ends are copied
// whole, but for those that reach past the matrix, whose bytes the thread copies.
struct RingFeed {
  RingHead* h;
  char* slots;
  const char *a, *b;
  int64_t a_pitch, b_pitch, row, rows;
  uint32_t a_bytes, b_bytes, issued;
  struct Units {
    uintptr_t from, to;
  };
  // The whole units of a row of `bytes` (64 at least) that lie inside the matrix; copies the other bytes.
  __device__ __forceinline__ Units ends(char* slot, const char* m, int64_t pitch, uint32_t bytes) const {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(m), p = lo + row * pitch, end = p + bytes;
    const uintptr_t hi = lo + (rows - 1) * pitch + bytes, origin = p & ~uintptr_t(15);
    Units u{origin, (end + 15) & ~uintptr_t(15)};
    if (u.from < lo) u.from = (p + 15) & ~uintptr_t(15);
    if (u.to > hi) u.to = end & ~uintptr_t(15);
    for (uintptr_t q = p; q < u.from; ++q) slot[q - origin] = *reinterpret_cast<const char*>(q);
    for (uintptr_t q = u.to; q < end; ++q) slot[q - origin] = *reinterpret_cast<const char*>(q);
    return u;
  }
  // The next row into slot s.
  template <bool kVec>
  __device__ __forceinline__ void next(const Ring& ring, uint32_t s) {
    if (row >= rows) return;
    char* slot = slots + s * ring.slot_bytes;
    const uint32_t bar = tc::smem_addr(&h->full[s]), dst = tc::smem_addr(slot);
    if constexpr (kVec) {
      tc::mbar_expect(bar, a_bytes);  // the forward pass: one operand
      tc::bulk_load(dst, a + row * a_pitch, a_bytes, bar);
    } else {
      auto copy = [&](uint32_t to, const char* m, int64_t pitch, const Units& u) {
        const uintptr_t origin = reinterpret_cast<uintptr_t>(m + row * pitch) & ~uintptr_t(15);
        tc::bulk_load(to + uint32_t(u.from - origin), reinterpret_cast<const void*>(u.from), uint32_t(u.to - u.from), bar);
      };
      const Units ua = ends(slot, a, a_pitch, a_bytes);
      Units ub{0, 0};
      if (b_bytes != 0) ub = ends(slot + ring.second, b, b_pitch, b_bytes);
      tc::mbar_expect(bar, uint32_t(ua.to - ua.from) + uint32_t(ub.to - ub.from));
      copy(dst, a, a_pitch, ua);
      if (b_bytes != 0) copy(dst + ring.second, b, b_pitch, ub);
    }
    ++issued;
    row += gridDim.x;
  }
  // The same by a warp, rows on 16 bytes, with what belongs to a row beside its values: its mean and rstd and
  // (`words` of four) its scales, one word per lane.
  struct Side {
    const float *mean, *rstd;
    const uint8_t* scale;
    int64_t row_tiles;
    int words;
  };
  __device__ __forceinline__ void next(const Ring& ring, uint32_t s, const Side& side) {
    if (row >= rows) return;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t bar = tc::smem_addr(&h->full[s]), dst = tc::smem_addr(slots + s * ring.slot_bytes);
    if (lane == 0) {
      tc::mbar_expect(bar, a_bytes + b_bytes);
      tc::bulk_load(dst, a + row * a_pitch, a_bytes, bar);
      tc::bulk_load(dst + ring.second, b + row * b_pitch, b_bytes, bar);
    }
    if (int(lane) < side.words)  // 16 at most
      tc::copy_word(dst + ring.side + 16 + 4 * lane,
                    side.scale + (row >> 7) * side.row_tiles + (lane * 512 + (uint32_t(row) & 31) * 16 + ((uint32_t(row) >> 3) & 12)));
    if (lane >= 30) tc::copy_word(dst + ring.side + 4 * (lane - 30), (lane == 30 ? side.mean : side.rstd) + row);
    tc::copied_words_arrive(bar);
    ++issued;
    row += gridDim.x;
  }
  __device__ __forceinline__ void settle(const Ring& ring) const {
    tc::settle_copies(tc::smem_addr(h->full), uint32_t(ring.slots), issued);
  }
};

// Barriers and the first fills.
template <bool kVec>
__device__ __forceinline__ void ring_start(RingFeed& feed, uint32_t* gave_up, const Ring& ring) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < ring.slots; ++i) tc::mbar_init(tc::smem_addr(&feed.h->full[i]), 1);
    *gave_up = 0;
    tc::mbar_init_fence();
    for (int i = 0; i < ring.slots; ++i) feed.next<kVec>(ring, i);
  }
  __syncthreads();
}
__device__ __forceinline__ void ring_start(RingFeed& feed, uint32_t* gave_up, const Ring& ring, const RingFeed::Side& side) {
  if (threadIdx.x < 32) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < ring.slots; ++i) tc::mbar_init(tc::smem_addr(&feed.h->full[i]), 1 + 32);
      *gave_up = 0;
      tc::mbar_init_fence();
    }
    __syncwarp();
    for (int i = 0; i < ring.slots; ++i) feed.next(ring, i, side);
  }
  __syncthreads();
}

// Column of element k of piece i: eight neighbours (kVec), or neighbours across a warp, whose piece spans
// 256 columns: two blocks of a checkpoint, k < 4 and k >= 4.
template <bool kVec, int TH>
__device__ __forceinline__ int ring_col(int i, int k) {
  return kVec ? (int(threadIdx.x) + i * TH) * 8 + k
              : (int(threadIdx.x >> 5) + i * (TH / 32)) * 256 + k * 32 + int(threadIdx.x & 31);
}
// A piece of a row in shared memory; zeros past the row.
template <class T, bool kVec, int TH>
__device__ __forceinline__ Eight ring_piece(const char* row, int i, int cols) {
  if constexpr (kVec) {
    return load_eight<T>(row, ring_col<true, TH>(i, 0), ring_col<true, TH>(i, 0) < cols ? 8 : 0, true);
  } else {
    Eight e;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = ring_col<false, TH>(i, k);
      const uint32_t b = c < cols ? load_bits<T>(row, c) : 0u;
      e.v[k] = T::kBytes == 4 ? __uint_as_float(b) : __uint_as_float(b << 16);
    }
    return e;
  }
}
template <bool kVec, int TH>
__device__ __forceinline__ Eight ring_param(const void* base, int bf16, int i, int cols) {
  if constexpr (kVec) {
    const int col = ring_col<true, TH>(i, 0);
    return load_param(base, bf16, col, valid(cols, col), true);
  } else {
    const char* p = static_cast<const char*>(base);
    return bf16 ? ring_piece<BF16T, false, TH>(p, i, cols) : ring_piece<F32T, false, TH>(p, i, cols);
  }
}
template <class T, bool kVec, int TH>
__device__ __forceinline__ void ring_store(void* base, int64_t row, int i, int cols, const Eight& e) {
  if constexpr (kVec) {
    if (ring_col<true, TH>(i, 0) < cols) store_eight<T>(base, row + ring_col<true, TH>(i, 0), e, 8, true);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = ring_col<false, TH>(i, k);
      if (c < cols) store_bits<T>(base, row + c, T::kBytes == 4 ? __float_as_uint(e.v[k]) : bf16x2_rn(e.v[k], 0.0f));
    }
  }
}
// Bytes that a row starts into its first 16-byte unit, which is where its slot holds it.
template <bool kVec>
__device__ __forceinline__ int ring_offset(const void* base, int64_t byte) {
  return kVec ? 0 : int((reinterpret_cast<uintptr_t>(base) + byte) & 15);
}

template <class T, bool kVec, int TH, int NV, int BLOCKS>
__global__ void __launch_bounds__(TH, BLOCKS)
    k_norm_forward_ring(const __grid_constant__ NormForwardParams p, int wbf16, Ring ring, unsigned* given_up) {
  extern __shared__ __align__(128) char smem[];
  __shared__ uint32_t s_gave_up;
  volatile uint32_t* gave_up = &s_gave_up;
  RingHead* h = reinterpret_cast<RingHead*>(smem);
  char* slots = smem + kRingHead;
  grid_dependency_sync();
  RingFeed feed{h, slots, static_cast<const char*>(p.x), nullptr, p.ld_x * T::kBytes, 0, blockIdx.x, p.rows,
                uint32_t(p.cols * T::kBytes), 0, 0};
  ring_start<kVec>(feed, &s_gave_up, ring);
  const int t = threadIdx.x;
  {
    const int cols = int(p.cols);
    const float count = float(cols), inv = 1.0f / count;
    Eight w[NV], b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      w[i] = ring_param<kVec, TH>(p.weight, wbf16, i, cols);
      b[i] = {};
      if (p.bias != nullptr) b[i] = ring_param<kVec, TH>(p.bias, wbf16, i, cols);
    }
    int s = 0, half = 0;
    uint32_t phase = 0;
    bool good = true;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
      // A thread whose wait was given up still goes through the barriers of this row and the ones after, so
      // that no other waits for it, but writes no more rows or statistics and fetches nothing: its slot's copy
      // may yet land, and a barrier takes no second arrival for the same copy.  (What the rest of the block
      // writes, and the sums over rows, are then invalid: the call is reported.)
      good &= tc::mbar_wait(tc::smem_addr(&h->full[s]), phase, gave_up);
      const char* src = slots + s * ring.slot_bytes + ring_offset<kVec>(p.x, row * p.ld_x * T::kBytes);
      Eight x[NV];
      float sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i] = ring_piece<T, kVec, TH>(src, i, cols);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[0] += x[i].v[k];
      }
      ring_sum<TH>(sum, h, half);
      if (t == 0 && good) feed.next<kVec>(ring, s);  // every thread has the row in registers
      // A product with 1 / cols alone rounds twice: the mean of a constant row would be off by a last place and
      // its deviations not zero.  Adding what is left of the sum, over cols, makes an exact quotient exact
      // (dividing: 16384 x 6144 BF16 64.8 us for 62.3; neither 62.1).  Of an infinite sum NaN is left: fminf makes it a number,
      // and the mean stays infinite.
      const float near = sum[0] * inv;
      const float mean = __fmaf_rn(fminf(__fmaf_rn(-count, near, sum[0]), FLT_MAX), inv, near);
      sum[0] = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[i].v[k] = ring_col<kVec, TH>(i, kVec ? 0 : k) < cols ? x[i].v[k] - mean : 0.0f;
          sum[0] += x[i].v[k] * x[i].v[k];
        }
      }
      ring_sum<TH>(sum, h, half);
      const float rstd = __frsqrt_rn(sum[0] * inv + p.eps);
      if (t == 0 && good) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        Eight y;
#pragma unroll
        for (int k = 0; k < 8; ++k) y.v[k] = x[i].v[k] * rstd * w[i].v[k] + b[i].v[k];
        if (good) ring_store<T, kVec, TH>(p.y, row * p.ld_y, i, cols, y);
      }
      if (++s == ring.slots) {
        s = 0;
        phase ^= 1;
      }
    }
  }
  __syncthreads();
  if (t == 0 && *gave_up != 0) {
    feed.settle(ring);
    tc::report_given_up(given_up);
  }
}

// The two passes over a row take xh = (x - mean) rstd in two forms, neither of which costs an instruction more
// than a product would:
//   sums   d = x - mean, one rounding of a difference that may cancel.  With t = dy d the sums are t w (times
//          rstd once per row) and t rstd, both fused.
//   dx     BF16 and codes: x rstd - m with m = mean rstd rounded.  What m's rounding left out, the same for the whole
//          row and up to |mean| rstd 2^-24, goes into the row's constant.  F32: d rstd.
// (x rstd - m alone in both had xh = 2.7e-3 for 0 in a constant row of 1000.  d rstd in both: 16384 x 6144 BF16
// from codes 97.9 us for 94.7, 16384 x 4096 BF16 70.5 for 68.5.)  Codes come with their scale f, a power of two:
// x stands for x f.
template <class T, bool kCodes, bool kVec, int TH, int NV, int BLOCKS>
__global__ void __launch_bounds__(TH, BLOCKS)
    k_norm_backward_ring(const __grid_constant__ NormBackwardParams p, int wbf16, Ring ring, unsigned* given_up) {
  extern __shared__ __align__(128) char smem[];
  __shared__ uint32_t s_gave_up;
  // kVec false: a row's scales, by block.  Three rows: the next one's are written before the barrier
  // that a row's readers have yet to reach, when none can still be two rows behind.
  __shared__ float s_scale[kCodes && !kVec ? 3 : 1][64];
  volatile uint32_t* gave_up = &s_gave_up;
  RingHead* h = reinterpret_cast<RingHead*>(smem);
  char* slots = smem + kRingHead;
  constexpr int kXBytes = kCodes ? 1 : T::kBytes;
  constexpr bool kFused = kCodes || T::kBytes == 2;
  grid_dependency_sync();
  RingFeed feed{h, slots, static_cast<const char*>(p.dy), static_cast<const char*>(p.x), p.ld_dy * T::kBytes,
                p.ld_x * kXBytes, blockIdx.x, p.rows, uint32_t(p.cols * T::kBytes), uint32_t(p.cols * kXBytes), 0};
  const int64_t row_tiles = scale_tile_cols((p.cols + kCkptBlock - 1) / kCkptBlock) * 512;
  const RingFeed::Side side{p.mean, p.rstd, p.x_scale, row_tiles, kCodes ? int(row_tiles / 512) : 0};
  if constexpr (kVec) ring_start(feed, &s_gave_up, ring, side);
  else ring_start<false>(feed, &s_gave_up, ring);
  const int t = threadIdx.x;
  {
    const int cols = int(p.cols);
    const float inv = 1.0f / float(cols);
    Two dw[NV][4], db[NV][4], w[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Eight e = ring_param<kVec, TH>(p.weight, wbf16, i, cols);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[i][k] = Two(e.v[2 * k], e.v[2 * k + 1]);
        dw[i][k] = db[i][k] = Two(0.0f);
      }
    }
    // kVec: a row's statistics and scales come with it.  Else they are fetched a whole row ahead, the scales
    // two: their latency passes behind the rows before
    struct Stats {
      float mean, rstd;
      uint32_t scale;  // of block t
    };
    const int blocks = (cols + kCkptBlock - 1) / kCkptBlock;
    const int at = kCodes && !kVec && t < blocks ? (t >> 2) * 512 + (t & 3) : -1;  // byte of the scale inside a row's tiles
    auto fetch = [&](int64_t row, Stats& st) {
      if (row >= p.rows) return;
      st.mean = p.mean[row];
      st.rstd = p.rstd[row];
      if (kCodes && at >= 0) st.scale = p.x_scale[(row >> 7) * row_tiles + (row & 31) * 16 + ((row >> 5) & 3) * 4 + at];
    };
    Stats next = {};
    if constexpr (!kVec) fetch(blockIdx.x, next);
    int third = 0;
    uint32_t later = 0;  // the scale of block t two rows ahead
    if constexpr (kCodes && !kVec) {
      if (t < 64) s_scale[0][t] = scale_value(next.scale);
      Stats st = {};
      fetch(blockIdx.x + int64_t(gridDim.x), st);
      later = st.scale;
      __syncthreads();
    }
    int s = 0, half = 0;
    uint32_t phase = 0;
    bool good = true;  // as in the forward pass
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
      Stats now = next;
      if constexpr (!kVec) fetch(row + gridDim.x, next);
      const float* scales = s_scale[kCodes && !kVec ? third : 0];
      if constexpr (kCodes && !kVec) {
        if (++third == 3) third = 0;
        if (t < 64) s_scale[third][t] = scale_value(later);
        Stats st = {};
        fetch(row + 2 * int64_t(gridDim.x), st);
        later = st.scale;
      }
      good &= tc::mbar_wait(tc::smem_addr(&h->full[s]), phase, gave_up);
      const char* slot = slots + s * ring.slot_bytes;
      const char* dy_row = slot + ring_offset<kVec>(p.dy, row * p.ld_dy * T::kBytes);
      const char* x_row = slot + ring.second + ring_offset<kVec>(p.x, row * p.ld_x * kXBytes);
      float scale[NV];  // of a piece's codes
      if constexpr (kVec) {
        const float2 st = *reinterpret_cast<const float2*>(slot + ring.side);
        now.mean = st.x;
        now.rstd = st.y;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        scale[i] = 1.0f;
        if constexpr (kCodes && kVec) scale[i] = scale_value(reinterpret_cast<const uint8_t*>(slot + ring.side + 16)[(t + i * TH) / (kCkptBlock / 8)]);
      }
      const float m = __fmul_rn(now.mean, now.rstd);
      const float rest = kFused ? -__fmaf_rn(now.mean, now.rstd, -m) : 0.0f;
      const Two r2(now.rstd), minus_mean(-now.mean), shift(-m);
      // the piece's dy and x, as pairs, and the scales of x
      auto piece = [&](int i, Two (&dy)[4], Two (&xs)[4], float (&f)[2]) {
        const Eight e = ring_piece<T, kVec, TH>(dy_row, i, cols);
        Eight x;
        if constexpr (kCodes && kVec) {
          x = load_codes(reinterpret_cast<const uint8_t*>(x_row) + ring_col<true, TH>(i, 0), 8, true);
        } else if constexpr (kCodes) {
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const int c0 = ring_col<false, TH>(i, k), c1 = ring_col<false, TH>(i, k + 1);
            const uint32_t two = (c0 < cols ? uint8_t(x_row[c0]) : 0u) | (c1 < cols ? uint32_t(uint8_t(x_row[c1])) << 8 : 0u);
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(two)));
            x.v[k] = f16_lo(h2);
            x.v[k + 1] = f16_hi(h2);
          }
        } else {
          x = ring_piece<T, kVec, TH>(x_row, i, cols);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dy[k] = Two(e.v[2 * k], e.v[2 * k + 1]);
          xs[k] = Two(x.v[2 * k], x.v[2 * k + 1]);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) f[b] = kCodes && !kVec ? scales[ring_col<false, TH>(i, 0) / kCkptBlock + b] : scale[i];
      };
      Two s0(0.0f), s1(0.0f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (ring_col<kVec, TH>(i, 0) >= cols) continue;
        Two dy[4], x[4];  // past the row dy is 0, and adds nothing
        float f[2];
        piece(i, dy, x, f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const Two d = kCodes ? fma2(x[k], Two(f[k >> 1]), minus_mean) : x[k] + minus_mean;
          const Two t = dy[k] * d;
          s0 = fma2(dy[k], w[i][k], s0);
          s1 = fma2(t, w[i][k], s1);
          dw[i][k] = fma2(t, r2, dw[i][k]);
          db[i][k] = db[i][k] + dy[k];
        }
      }
      float sum[2], lo, hi;
      s0.get(lo, hi);
      sum[0] = lo + hi;
      s1.get(lo, hi);
      sum[1] = lo + hi;
      ring_sum<TH>(sum, h, half);
      if (row != blockIdx.x && good) {  // every thread is past the row before
        const uint32_t before = s == 0 ? ring.slots - 1 : s - 1;
        if constexpr (kVec) {
          if (t < 32) feed.next(ring, before, side);
        } else {
          if (t == 0) feed.next<false>(ring, before);
        }
      }
      // dx = rstd g - rstd mean(g) - xh rstd mean(g xh)
      const float by_xh = -now.rstd * (sum[1] * now.rstd * inv);
      const Two c0(__fmaf_rn(rest, by_xh, -now.rstd * (sum[0] * inv))), c1(by_xh);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (ring_col<kVec, TH>(i, 0) >= cols) continue;
        Two dy[4], x[4];
        float f[2];
        piece(i, dy, x, f);
        Eight dx;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const Two xh = kFused ? fma2(x[k], Two(f[k >> 1] * now.rstd), shift) : (x[k] + minus_mean) * r2;
          fma2(xh, c1, fma2(dy[k] * w[i][k], r2, c0)).get(dx.v[2 * k], dx.v[2 * k + 1]);
        }
        if (good) ring_store<T, kVec, TH>(p.dx, row * p.ld_dx, i, cols, dx);
      }
      if (++s == ring.slots) {
        s = 0;
        phase ^= 1;
      }
    }
    float* out = p.workspace + int64_t(blockIdx.x) * 2 * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Eight a, c;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dw[i][k].get(a.v[2 * k], a.v[2 * k + 1]);
        db[i][k].get(c.v[2 * k], c.v[2 * k + 1]);
      }
      ring_store<F32T, kVec, TH>(out, 0, i, cols, a);
      ring_store<F32T, kVec, TH>(out + cols, 0, i, cols, c);
    }
  }
  __syncthreads();
  if (t == 0 && *gave_up != 0) {
    feed.settle(ring);
    tc::report_given_up(given_up);
  }
}

// Adds the partial rows in their order: a block owns 32 entries of [2][cols], each of its 32 warps a
// 32nd of the rows, added up through shared memory.
__global__ void __launch_bounds__(1024) k_norm_partials(const float* __restrict__ part, int nparts, int64_t cols,
                                                        float* dweight, float* dbias) {
  __shared__ float s[32][33];
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t e = int64_t(blockIdx.x) * 32 + lane;
  const int lo = nparts * warp / 32, hi = nparts * (warp + 1) / 32;
  float v = 0.0f;
  if (e < 2 * cols) {
#pragma unroll 8
    for (int r = lo; r < hi; ++r) v += part[int64_t(r) * 2 * cols + e];
  }
  s[warp][lane] = v;
  __syncthreads();
  v = warp_sum(s[lane][warp]);  // this warp: entry `warp` of the block
  const int64_t mine = int64_t(blockIdx.x) * 32 + warp;
  if (lane == 0 && mine < 2 * cols) {
    if (mine < cols) dweight[mine] = v;
    else if (dbias != nullptr) dbias[mine - cols] = v;
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

// Whether rows of `cols` columns go through a ring: enough of them for the prologue of a persistent
// block to pay (odd widths: backward 1001x1023 F32 9.8 us, direct 7.3; 4096x1001 13.7 and 16.4), and rows of
// 64 bytes or more.
bool ring_rows(int64_t rows, int64_t cols, bool odd, const DeviceInfo& dev) {
  return cols <= 8192 && (cols % 16 == 0 || cols >= 64) && rows >= (odd ? 12 : 4) * int64_t(dev.sms);
}

template <class T, bool kVec, int TH, int NV, int BLOCKS>
cudaError_t forward_ring(const NormForwardParams& p, int wdtype, const DeviceInfo& dev, unsigned* given_up,
                         cudaStream_t stream) {
  const Ring ring = ring_of(p.cols * T::kBytes + (kVec ? 0 : 30), 0, 0, BLOCKS);
  auto kernel = k_norm_forward_ring<T, kVec, TH, NV, BLOCKS>;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(ring.smem));
  if (e != cudaSuccess) return e;
  const int64_t most = BLOCKS * dev.sms;
  return launch_kernel(kernel, dim3(unsigned(p.rows < most ? p.rows : most)), dim3(TH), ring.smem, stream, p, wdtype,
                       ring, given_up);
}

template <class T>
cudaError_t forward(const NormForwardParams& p, int wdtype, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t pieces = (p.cols + 7) / 8;
  auto launch = [&](auto kernel, int64_t blocks, int threads) {
    return launch_kernel(kernel, dim3(unsigned(blocks)), dim3(threads), 0, stream, p, wdtype);
  };
  if (ring_rows(p.rows, p.cols, p.cols % 8 != 0, dev) && (p.cols % 8 != 0 || p.vec)) {
    unsigned* given_up = nullptr;
    const cudaError_t e = given_up_address(dev.device, &given_up);
    if (e != cudaSuccess) return e;
    if (p.cols % 8 != 0) {
      if (pieces <= 64) return forward_ring<T, false, 64, 1, 12>(p, wdtype, dev, given_up, stream);
      if (pieces <= 128) return forward_ring<T, false, 128, 1, 6>(p, wdtype, dev, given_up, stream);
      if (pieces <= 256) return forward_ring<T, false, 256, 1, 4>(p, wdtype, dev, given_up, stream);
      if (pieces <= 384) return forward_ring<T, false, 192, 2, 4>(p, wdtype, dev, given_up, stream);
      if (pieces <= 512) return forward_ring<T, false, 256, 2, 3>(p, wdtype, dev, given_up, stream);
      if (pieces <= 768) return forward_ring<T, false, 256, 3, 2>(p, wdtype, dev, given_up, stream);
      return forward_ring<T, false, 256, 4, 2>(p, wdtype, dev, given_up, stream);
    }
    if (pieces <= 32) return forward_ring<T, true, 32, 1, 24>(p, wdtype, dev, given_up, stream);
    if (pieces <= 64) return forward_ring<T, true, 32, 2, 20>(p, wdtype, dev, given_up, stream);
    if (pieces <= 128) return forward_ring<T, true, 64, 2, 12>(p, wdtype, dev, given_up, stream);
    if (pieces <= 256) return forward_ring<T, true, 128, 2, 6>(p, wdtype, dev, given_up, stream);
    if (pieces <= 512) return forward_ring<T, true, 256, 2, T::kBytes == 2 ? 3 : 2>(p, wdtype, dev, given_up, stream);
    if (pieces <= 768) return forward_ring<T, true, 256, 3, 2>(p, wdtype, dev, given_up, stream);
    return forward_ring<T, true, 256, 4, 2>(p, wdtype, dev, given_up, stream);
  }
  auto direct = [&](auto vec) {
    constexpr bool kVec = decltype(vec)::value;
    if (pieces <= 32) return launch(k_norm_forward<T, false, kVec, 1>, (p.rows + 7) / 8, 256);
    if (pieces <= 64) return launch(k_norm_forward<T, false, kVec, 2>, (p.rows + 7) / 8, 256);
    if (pieces <= 128) return launch(k_norm_forward<T, false, kVec, 4>, (p.rows + 7) / 8, 256);
    auto threads = [&](int nv) { return int(((pieces + nv - 1) / nv + 31) / 32 * 32); };
    if (pieces <= 512) return launch(k_norm_forward<T, true, kVec, 1>, p.rows, threads(1));
    if (pieces <= 1024) return launch(k_norm_forward<T, true, kVec, 2>, p.rows, threads(2));
    return launch(k_norm_forward<T, true, kVec, 4>, p.rows, threads(4));
  };
  if (pieces <= 4096) return p.cols % 8 == 0 ? direct(std::true_type{}) : direct(std::false_type{});
  return launch_kernel(k_norm_forward_long<T>, dim3(unsigned(p.rows)), dim3(1024), 0, stream, p, wdtype);
}

template <class T, bool kCodes, bool kVec, int TH, int NV, int BLOCKS>
cudaError_t backward_ring(const NormBackwardParams& p, int wdtype, const DeviceInfo& dev, unsigned* given_up,
                          unsigned* blocks, cudaStream_t stream) {
  constexpr int kPad = kVec ? 0 : 30;
  const Ring ring = ring_of(p.cols * T::kBytes + kPad, p.cols * (kCodes ? 1 : T::kBytes) + kPad,
                            kVec ? (kCodes ? 16 + 64 : 16) : 0, BLOCKS);
  auto kernel = k_norm_backward_ring<T, kCodes, kVec, TH, NV, BLOCKS>;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(ring.smem));
  if (e != cudaSuccess) return e;
  const int64_t most = BLOCKS * dev.sms, room = norm_partials(p.rows, p.cols);
  *blocks = unsigned(most < room ? most : room);
  return launch_kernel(kernel, dim3(*blocks), dim3(TH), ring.smem, stream, p, wdtype, ring, given_up);
}

template <class T, bool kCodes>
cudaError_t backward(const NormBackwardParams& p, int wdtype, const DeviceInfo& dev, cudaStream_t stream) {
  const Spread s = spread_of(p.cols, 2);
  const int64_t pieces = (p.cols + 7) / 8, room = norm_partials(p.rows, p.cols), work = s.block ? p.rows : (p.rows + 7) / 8;
  unsigned blocks = unsigned(work < room ? work : room);
  const dim3 block(s.threads), grid(blocks);
  // codes: 8-byte units serve the direct kernels, the ring copies 16
  const bool odd = p.cols % (kCodes ? 16 : 8) != 0, units = p.vec && !odd && (!kCodes || p.ld_x % 16 == 0) &&
                     reinterpret_cast<uintptr_t>(p.x) % 16 == 0;
  cudaError_t e;
  if ((units || odd) && ring_rows(p.rows, p.cols, odd, dev)) {
    unsigned* given_up = nullptr;
    e = given_up_address(dev.device, &given_up);
    if (e != cudaSuccess) return e;
    if (odd) {
      // by figures: 16384 x 3001 BF16 77 us (256 threads, two blocks 89), F32 93 with two blocks, 103 with
      // three; 16384 x 6143 from codes 143 us (512 threads, one block 255, most of it scales per element)
      e = pieces <= 64    ? backward_ring<T, kCodes, false, 64, 1, 8>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 128 ? (kCodes || T::kBytes == 2 ? backward_ring<T, kCodes, false, 64, 2, 8>(p, wdtype, dev, given_up, &blocks, stream)
                                                      : backward_ring<T, kCodes, false, 128, 1, 5>(p, wdtype, dev, given_up, &blocks, stream))
          : pieces <= 256 ? backward_ring<T, kCodes, false, 256, 1, 3>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 384 ? backward_ring<T, kCodes, false, 192, 2, kCodes || T::kBytes == 2 ? 3 : 2>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 512 ? backward_ring<T, kCodes, false, 256, 2, 2>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 768 ? backward_ring<T, kCodes, false, 256, 3, 2>(p, wdtype, dev, given_up, &blocks, stream)
                          : backward_ring<T, kCodes, false, 512, 2, 1>(p, wdtype, dev, given_up, &blocks, stream);
    } else {
      // blocks per SM: BF16 rows are bound by arithmetic and its waits, which more warps fill; F32 rows by
      // the bytes under way, which fewer and deeper rings keep up (16384 x 4096 with two and with three
      // blocks: BF16 72.9 and 65.3 us, from codes 82.0 and 75.7; F32 100.8 and 108.5)
      constexpr bool kNarrow = T::kBytes == 2;
      e = pieces <= 32    ? backward_ring<T, kCodes, true, 32, 1, 20>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 64  ? backward_ring<T, kCodes, true, 32, 2, kNarrow ? 20 : 16>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 128 ? backward_ring<T, kCodes, true, 64, 2, kNarrow ? 12 : 8>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 256 ? backward_ring<T, kCodes, true, 128, 2, kNarrow ? 6 : 4>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 512 ? backward_ring<T, kCodes, true, 256, 2, kNarrow ? 3 : 2>(p, wdtype, dev, given_up, &blocks, stream)
          : pieces <= 768 ? backward_ring<T, kCodes, true, 256, 3, 2>(p, wdtype, dev, given_up, &blocks, stream)
                          : backward_ring<T, kCodes, true, 512, 2, 1>(p, wdtype, dev, given_up, &blocks, stream);
    }
  } else if (s.nv == 0) {
    e = launch_kernel(k_norm_backward_long<T, kCodes>, grid, block, 0, stream, p, wdtype);
  } else {
    auto direct = [&](auto vec) {
      constexpr bool kVec = decltype(vec)::value;
      auto run = [&](auto kernel, size_t smem) {
        const cudaError_t a = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, 65536);
        return a != cudaSuccess ? a : launch_kernel(kernel, grid, block, smem, stream, p, wdtype);
      };
      if (s.block)
        return s.nv == 1 ? run(k_norm_backward<T, kCodes, true, kVec, 1>, 0) : run(k_norm_backward<T, kCodes, true, kVec, 2>, 0);
      const size_t smem = size_t(8) * 2 * size_t(p.cols) * 4;
      if (s.nv == 1) return run(k_norm_backward<T, kCodes, false, kVec, 1>, smem);
      if (s.nv == 2) return run(k_norm_backward<T, kCodes, false, kVec, 2>, smem);
      return run(k_norm_backward<T, kCodes, false, kVec, 4>, smem);
    };
    e = p.cols % 8 == 0 ? direct(std::true_type{}) : direct(std::false_type{});
  }
  if (e != cudaSuccess) return e;
  const dim3 rgrid(static_cast<unsigned>((2 * p.cols + 31) / 32));
  return launch_kernel(k_norm_partials, rgrid, dim3(1024), 0, stream, static_cast<const float*>(p.workspace),
                       int(blocks), p.cols, p.dweight, p.dbias);
}

}  // namespace

// As many as the blocks of a ring, of BF16 rows, that run at once on 152 SMs.
int64_t norm_partials(int64_t rows, int64_t cols) {
  const int64_t most = cols <= 512 ? 3040 : (cols <= 1024 ? 1824 : (cols <= 2048 ? 912 : (cols <= 4096 ? 456 : 304)));
  return rows < most ? rows : most;
}

cudaError_t launch_norm_forward(const NormForwardParams& p, int dtype, int wdtype, const DeviceInfo& dev,
                                cudaStream_t stream) {
  return dtype == 0 ? forward<F32T>(p, wdtype, dev, stream) : forward<BF16T>(p, wdtype, dev, stream);
}

cudaError_t launch_norm_backward(const NormBackwardParams& p, int dtype, int wdtype, const DeviceInfo& dev,
                                 cudaStream_t stream) {
  const bool codes = p.x_scale != nullptr;
  if (dtype == 0)
    return codes ? backward<F32T, true>(p, wdtype, dev, stream) : backward<F32T, false>(p, wdtype, dev, stream);
  return codes ? backward<BF16T, true>(p, wdtype, dev, stream) : backward<BF16T, false>(p, wdtype, dev, stream);
}

}  // namespace mxfp8
