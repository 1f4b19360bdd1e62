// RMS norm of the rows of a residual stream, and its gradients.
//
//   forward    s = x + residual,  rstd = (sum s^2 / c + eps)^-1/2,  y = s rstd w
//   backward   xh = s rstd,  g = dy w
//              ds = rstd (g - xh sum(g xh) / c) + dsum,   dw = sum over rows of dy xh
//
// y leaves as values, as E4M3 codes with one E8M0 scale per 128 values of a row, or both, and its largest magnitude may
// be folded into one word for a 4-bit quantisation that follows.  Everything between load and store is F32; s, y and ds
// are rounded once, and y and its codes come from the unrounded s.
//
// Both directions read every value once.  Many rows of 257 to 8192 columns go through rings of bulk copies in persistent
// blocks (below); others belong to one group of threads each, which holds the row in registers between the sum and the
// outputs: a warp for up to 256 columns, else a block; beyond 32768 columns (16384 backward) the row is read again,
// mostly from L2.  In the backward pass a thread keeps the running dw of its columns in registers over all rows of its block; a block
// leaves one row of partial sums, and a second kernel adds the partial rows in their order, so the sums do not depend on
// the run.
//
// Measured at 16384 x 6144 BF16 with the residual (floor at 6.8 TB/s): forward with codes 117 us (104), with values 137 (119);
// backward with the stream's gradient 130 (119), without 97 (89): bound by HBM, the forward pass with codes also by
// instructions (57 % of the issue slots at 16 warps per SM).  F32: 230 (193), 261 (237), 261 (237), 205 (178).  16384 x 6143 BF16:
// 193, 151, 146, 119; this path takes an element per load and store, also of codes, whose rows could take wider ones.
// 1 x 4096: 3.0 with codes, 2.5 with values, 3.7 backward, each one launch.
// Without a ring, where a block waits for its row and nothing is fetched behind it, codes / values / backward: 8192 x 12288 BF16 285,
// 267, 289 (104, 119, 119), 8192 x 16384 318, 294, 315 (138, 158, 158), where the backward pass also spills (136 to 196 bytes at 64
// registers); 16384 x 6144 in rows that start off 16 bytes 405, 564, 442, eight single elements per thread side by side.
#include <cfloat>
#include <type_traits>

#include "fp4.cuh"
#include "launch.h"
#include "norm_impl.cuh"

namespace mxfp8 {
namespace {

// The columns of a thread's pieces: eight neighbours where the columns are a multiple of 8, else neighbours across a warp,
// whose piece spans 256 columns; 128 columns, a block of codes, are 16 lanes or half of a warp's piece (k < 4, k >= 4).
template <bool kVec>
struct RowColumns {
  int64_t cols;
  int t, width;  // of the row's threads
  bool aligned;
  __device__ __forceinline__ int64_t at(int i, int k) const {
    return kVec ? int64_t(t + i * width) * 8 + k : int64_t((t >> 5) + i * (width >> 5)) * 256 + k * 32 + (t & 31);
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

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// |y| as it is stored, as F32 bits.
template <class T>
__device__ __forceinline__ uint32_t stored_bits(float v) {
  return T::kBytes == 4 ? abs_bits(v) : (bf16x2_rn(0.0f, v) & 0x7fff0000u);
}

__device__ __forceinline__ uint2 encode8(const Eight& y, float f) {
  float p[8];
#pragma unroll
  for (int k = 0; k < 8; k += 2) mul2_rn(y.v[k], y.v[k + 1], f, f, p[k], p[k + 1]);
  return make_uint2(e4m3x2_rn_sat(p[0], p[1]) | (e4m3x2_rn_sat(p[2], p[3]) << 16),
                    e4m3x2_rn_sat(p[4], p[5]) | (e4m3x2_rn_sat(p[6], p[7]) << 16));
}

// The scale byte of block b of a row; behind a row's last block the padding up to a whole group of four.
__device__ __forceinline__ void store_scale(const RmsForwardParams& p, int64_t row, int64_t b, uint32_t byte) {
  const int64_t blocks = (p.cols + kCkptBlock - 1) / kCkptBlock;
  uint8_t* s = p.scale + scale_at(row, b, scale_tile_cols(blocks));
  *s = uint8_t(byte);
  if (b == blocks - 1)
    for (int i = int(b & 3) + 1; i < 4; ++i) *++s = 0;
}

// Zeros in the scales of the rows behind the last one, up to a whole tile: by the threads of the last row.
__device__ __forceinline__ void pad_scales(const RmsForwardParams& p, int t, int width) {
  const uint32_t tile_cols = uint32_t(scale_tile_cols((p.cols + kCkptBlock - 1) / kCkptBlock));
  const uint32_t words = uint32_t((p.rows + 127) / 128 * 128 - p.rows) * tile_cols;  // one per row and tile of four blocks
  for (uint32_t i = uint32_t(t); i < words; i += uint32_t(width)) {
    const uint32_t row = i / tile_cols, tile = i - row * tile_cols;
    *reinterpret_cast<uint32_t*>(p.scale + scale_at(p.rows + row, 4 * int64_t(tile), tile_cols)) = 0u;
  }
}

// Codes of a thread's piece of eight neighbours; the 16 lanes of a block of 128 all take part.
__device__ __forceinline__ void store_codes(const RmsForwardParams& p, int64_t row, int64_t col, const Eight& y) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, abs_bits(y.v[k]));
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) m = max(m, __shfl_xor_sync(kFullMask, m, off));
  const int n = valid(p.cols, col);
  if (n == 0) return;
  const uint32_t s = e8m0_from_bits<F32T>(m);
  if ((col & 127) == 0) store_scale(p, row, col >> 7, s);
  const uint2 q = encode8(y, scale_multiplier(s));
  uint8_t* dst = p.codes + row * p.ld_q + col;
  if (p.vec_q && n == 8) {
    *reinterpret_cast<uint2*>(dst) = q;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) dst[k] = uint8_t((k < 4 ? q.x : q.y) >> (8 * (k & 3)));
  }
}
// The same of a piece that lies across a warp: two blocks.
__device__ __forceinline__ void store_codes_across(const RmsForwardParams& p, int64_t row, int64_t col0, int lane, const Eight& y) {
  uint32_t s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max(m, abs_bits(y.v[4 * h + k]));
    s[h] = e8m0_from_bits<F32T>(__reduce_max_sync(kFullMask, m));
    if (lane == 0 && col0 + 128 * h < p.cols) store_scale(p, row, (col0 >> 7) + h, s[h]);
  }
  uint8_t* dst = p.codes + row * p.ld_q + col0 + lane;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t q = e4m3x2_rn_sat(y.v[k] * scale_multiplier(s[k >> 2]), 0.0f);
    if (col0 + 32 * k + lane < p.cols) dst[32 * k] = uint8_t(q);
  }
}

// Folds a warp's largest |y| into the output word, which most often holds more already.
__device__ __forceinline__ void fold_amax(float* amax, uint32_t m) {
  m = canonical_nan<F32T>(__reduce_max_sync(kFullMask, m));
  if ((threadIdx.x & 31) == 0 && m > __ldcg(reinterpret_cast<const uint32_t*>(amax))) atomicMax(reinterpret_cast<uint32_t*>(amax), m);
}

// ------------------------------------------------------------------------------ forward
template <class T, bool kBlock, bool kVec, int NV>
__global__ void __launch_bounds__(kBlock ? 1024 : 256)
    k_rms_forward(const __grid_constant__ RmsForwardParams p, int wbf16) {
  __shared__ float buf[2][32];
  grid_dependency_sync();
  const RowColumns<kVec> c{p.cols, int(kBlock ? threadIdx.x : threadIdx.x & 31), int(kBlock ? blockDim.x : 32), p.vec != 0};
  const int64_t row = kBlock ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.rows) return;  // whole warps only
  int half = 0;
  Eight x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = c.template load<T>(p.x, row * p.ld_x, i);
  if (p.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Eight r = c.template load<T>(p.residual, row * p.ld_r, i);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i].v[k] += r.v[k];
    }
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += x[i].v[k] * x[i].v[k];
  group_sum<kBlock>(s, &buf[0][0], half);
  const float rstd = __frsqrt_rn(s[0] / float(p.cols) + p.eps);
  if (c.t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (p.sum != nullptr) c.template store<T>(p.sum, row * p.ld_s, i, x[i]);
    const Eight w = c.param(p.weight, wbf16, i);
    Eight y;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y.v[k] = c.in(i, k) ? x[i].v[k] * rstd * w.v[k] : 0.0f;
      top = max(top, stored_bits<T>(y.v[k]));
    }
    if (p.y != nullptr) c.template store<T>(p.y, row * p.ld_y, i, y);
    if (p.codes != nullptr) {
      if constexpr (kVec) store_codes(p, row, c.at(i, 0), y);
      else store_codes_across(p, row, c.at(i, 0) - (c.t & 31), c.t & 31, y);
    }
  }
  if (p.amax != nullptr) fold_amax(p.amax, top);
  if (p.codes != nullptr && row == p.rows - 1) pad_scales(p, c.t, c.width);
}

// Rows too long for registers: two passes over the row, the second mostly from L2.
template <class T>
__global__ void __launch_bounds__(1024) k_rms_forward_long(const __grid_constant__ RmsForwardParams p, int wbf16) {
  __shared__ float buf[2][32];
  grid_dependency_sync();
  const int64_t row = blockIdx.x, step = int64_t(blockDim.x) * 8;
  int half = 0;
  auto load = [&](int64_t col) {
    const int n = valid(p.cols, col);
    Eight x = load_eight<T>(p.x, row * p.ld_x + col, n, p.vec);
    if (p.residual != nullptr) {
      const Eight r = load_eight<T>(p.residual, row * p.ld_r + col, n, p.vec);
#pragma unroll
      for (int k = 0; k < 8; ++k) x.v[k] += r.v[k];
    }
    return x;
  };
  float s[1] = {0.0f};
  for (int64_t col = int64_t(threadIdx.x) * 8; col < p.cols; col += step) {
    const Eight x = load(col);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] += x.v[k] * x.v[k];
  }
  group_sum<true>(s, &buf[0][0], half);
  const float rstd = __frsqrt_rn(s[0] / float(p.cols) + p.eps);
  if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  uint32_t top = 0;
  for (int64_t base = 0; base < p.cols; base += step) {  // all threads: blocks of codes share their lanes
    const int64_t col = base + int64_t(threadIdx.x) * 8;
    const int n = valid(p.cols, col);
    const Eight x = load(col), w = load_param(p.weight, wbf16, col, n, p.vec);
    if (p.sum != nullptr) store_eight<T>(p.sum, row * p.ld_s + col, x, n, p.vec);
    Eight y;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y.v[k] = k < n ? x.v[k] * rstd * w.v[k] : 0.0f;
      top = max(top, stored_bits<T>(y.v[k]));
    }
    if (p.y != nullptr) store_eight<T>(p.y, row * p.ld_y + col, y, n, p.vec);
    if (p.codes != nullptr) store_codes(p, row, col, y);
  }
  if (p.amax != nullptr) fold_amax(p.amax, top);
  if (p.codes != nullptr && row == p.rows - 1) pad_scales(p, threadIdx.x, blockDim.x);
}

// ------------------------------------------------------------------------------ backward
template <class T, bool kBlock, bool kVec, int NV>
__global__ void __launch_bounds__(kBlock ? 1024 : 256)
    k_rms_backward(const __grid_constant__ RmsBackwardParams p, int wbf16) {
  __shared__ float buf[2][32];
  extern __shared__ float s_acc[];  // warp per row: [8 warps][dw of the columns]
  grid_dependency_sync();
  const RowColumns<kVec> c{p.cols, int(kBlock ? threadIdx.x : threadIdx.x & 31), int(kBlock ? blockDim.x : 32), p.vec != 0};
  const int warp = threadIdx.x >> 5;
  int half = 0;
  const float inv = 1.0f / float(p.cols);
  float dw[NV][8];
  Eight w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i] = c.param(p.weight, wbf16, i);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = 0.0f;
  }
  const int64_t first = kBlock ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 8 + warp;
  const int64_t step = kBlock ? int64_t(gridDim.x) : int64_t(gridDim.x) * 8;
  for (int64_t row = first; row < p.rows; row += step) {
    const float rstd = p.rstd[row];
    Eight dy[NV], xh[NV];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      dy[i] = c.template load<T>(p.dy, row * p.ld_dy, i);
      xh[i] = c.template load<T>(p.x, row * p.ld_x, i);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // columns past the last hold zeros
        xh[i].v[k] *= rstd;
        const float t = dy[i].v[k] * xh[i].v[k];
        s[0] += t * w[i].v[k];
        dw[i][k] += t;
      }
    }
    group_sum<kBlock>(s, &buf[0][0], half);
    const float along = s[0] * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!c.in(i, 0)) continue;
      Eight dx, ds = {};
      if (p.dsum != nullptr) ds = c.template load<T>(p.dsum, row * p.ld_ds, i);
#pragma unroll
      for (int k = 0; k < 8; ++k) dx.v[k] = rstd * (dy[i].v[k] * w[i].v[k] - xh[i].v[k] * along) + ds.v[k];
      c.template store<T>(p.dx, row * p.ld_dx, i, dx);
    }
  }
  // one row of partial sums per block: [blocks][cols]
  float* out = p.workspace + int64_t(blockIdx.x) * p.cols;
  const int cols = int(p.cols);
  float* mine = kBlock ? out : s_acc + warp * cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c.in(i, k)) mine[c.at(i, k)] = dw[i][k];
  }
  if constexpr (!kBlock) {
    __syncthreads();
    for (int e = threadIdx.x; e < cols; e += blockDim.x) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v += s_acc[k * cols + e];
      out[e] = v;
    }
  }
}

// Rows too long for registers: two passes over the row; the block's partial sums live in its workspace row (each
// entry touched by one thread only).
template <class T>
__global__ void __launch_bounds__(1024) k_rms_backward_long(const __grid_constant__ RmsBackwardParams p, int wbf16) {
  __shared__ float buf[2][32];
  grid_dependency_sync();
  int half = 0;
  const float inv = 1.0f / float(p.cols);
  float* out = p.workspace + int64_t(blockIdx.x) * p.cols;
  const int64_t step = int64_t(blockDim.x) * 8;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const bool first = row == blockIdx.x;
    const float rstd = p.rstd[row];
    float s[1] = {0.0f};
    for (int64_t col = int64_t(threadIdx.x) * 8; col < p.cols; col += step) {
      const int n = valid(p.cols, col);
      const Eight dy = load_eight<T>(p.dy, row * p.ld_dy + col, n, p.vec);
      const Eight x = load_eight<T>(p.x, row * p.ld_x + col, n, p.vec);
      const Eight w = load_param(p.weight, wbf16, col, n, p.vec);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float t = dy.v[k] * (x.v[k] * rstd);
        s[0] += t * w.v[k];
        if (k < n) out[col + k] = t + (first ? 0.0f : out[col + k]);
      }
    }
    group_sum<true>(s, &buf[0][0], half);
    const float along = s[0] * inv;
    for (int64_t col = int64_t(threadIdx.x) * 8; col < p.cols; col += step) {
      const int n = valid(p.cols, col);
      const Eight dy = load_eight<T>(p.dy, row * p.ld_dy + col, n, p.vec);
      const Eight x = load_eight<T>(p.x, row * p.ld_x + col, n, p.vec);
      const Eight w = load_param(p.weight, wbf16, col, n, p.vec);
      Eight dx, ds = {};
      if (p.dsum != nullptr) ds = load_eight<T>(p.dsum, row * p.ld_ds + col, n, p.vec);
#pragma unroll
      for (int k = 0; k < 8; ++k) dx.v[k] = rstd * (dy.v[k] * w.v[k] - x.v[k] * rstd * along) + ds.v[k];
      store_eight<T>(p.dx, row * p.ld_dx + col, dx, n, p.vec);
    }
  }
}

// Adds the partial rows in their order: a block owns 32 columns, each of its 32 warps a 32nd of the rows, added up
// through shared memory.
__global__ void __launch_bounds__(1024) k_rms_partials(const float* __restrict__ part, int nparts, int64_t cols, float* dweight) {
  __shared__ float s[32][33];
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t e = int64_t(blockIdx.x) * 32 + lane;
  const int lo = nparts * warp / 32, hi = nparts * (warp + 1) / 32;
  float v = 0.0f;
  if (e < cols) {
#pragma unroll 8
    for (int r = lo; r < hi; ++r) v += part[int64_t(r) * cols + e];
  }
  s[warp][lane] = v;
  __syncthreads();
  v = warp_sum(s[lane][warp]);  // this warp: column `warp` of the block
  const int64_t mine = int64_t(blockIdx.x) * 32 + warp;
  if (lane == 0 && mine < cols) dweight[mine] = v;
}

// ------------------------------------------------------------------------------ rings
// Many rows of up to 8192 columns: persistent blocks, each with a ring of rows in shared memory that thread 0 keeps
// full with bulk copies, whatever the warps wait for.  A thread owns fixed columns, NV pieces of 8, and keeps what belongs to
// a column (weight, running gradient) in registers over all rows.  A row takes one barrier of its block.
//
// What thread 0 fetches: rows blockIdx.x, blockIdx.x + gridDim.x, ... of up to three matrices of one type into the slots
// in turn, one behind the other.  Rows that do not start on 16 bytes (kVec false) land as many bytes into their place as
// they start into their first 16-byte unit; the units at a row's ends are copied whole, but for those that reach past the
// matrix, whose bytes the thread copies.
struct RowFeed {
  RingHead* h;
  char* slots;
  const char* m[3];
  int64_t pitch[3];
  int64_t row, rows;
  uint32_t bytes, place, count, issued;  // bytes of a row; of its place in a slot; matrices
  template <bool kVec>
  __device__ __forceinline__ void next(const Ring& ring, uint32_t s) {
    if (row >= rows) return;
    char* slot = slots + s * ring.slot_bytes;
    const uint32_t bar = tc::smem_addr(&h->full[s]), dst = tc::smem_addr(slot);
    if constexpr (kVec) {
      tc::mbar_expect(bar, bytes * count);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < int(count)) tc::bulk_load(dst + i * place, m[i] + row * pitch[i], bytes, bar);
    } else {
      RingFeed::Units u[3];
      uint32_t total = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (i >= int(count)) continue;
        const RingFeed one{nullptr, nullptr, nullptr, nullptr, 0, 0, row, rows, 0, 0, 0};
        u[i] = one.ends(slot + i * place, m[i], pitch[i], bytes);
        total += uint32_t(u[i].to - u[i].from);
      }
      tc::mbar_expect(bar, total);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (i >= int(count)) continue;
        const uintptr_t origin = reinterpret_cast<uintptr_t>(m[i] + row * pitch[i]) & ~uintptr_t(15);
        tc::bulk_load(dst + i * place + uint32_t(u[i].from - origin), reinterpret_cast<const void*>(u[i].from),
                      uint32_t(u[i].to - u[i].from), bar);
      }
    }
    ++issued;
    row += gridDim.x;
  }
  template <bool kVec>
  __device__ __forceinline__ void start(const Ring& ring, uint32_t* gave_up) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < ring.slots; ++i) tc::mbar_init(tc::smem_addr(&h->full[i]), 1);
      *gave_up = 0;
      tc::mbar_init_fence();
      for (int i = 0; i < ring.slots; ++i) next<kVec>(ring, i);
    }
    __syncthreads();
  }
  // Where the current row of matrix i lies in its slot.
  template <bool kVec>
  __device__ __forceinline__ const char* at(const char* slot, int i, int64_t r) const {
    return slot + i * place + ring_offset<kVec>(m[i], r * pitch[i]);
  }
};

// Ring of `count` rows of `bytes` each per slot.
Ring rows_ring(int64_t bytes, int count, int blocks) {
  const int64_t place = (bytes + 127) / 128 * 128;
  return ring_of(bytes, place * (count - 1), 0, blocks);
}

__device__ __forceinline__ void as_pairs(const Eight& e, Two (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = Two(e.v[2 * k], e.v[2 * k + 1]);
}
__device__ __forceinline__ float sum_of(Two a) {
  float lo, hi;
  a.get(lo, hi);
  return lo + hi;
}

template <class T, bool kVec, int TH, int NV, int BLOCKS>
__global__ void __launch_bounds__(TH, BLOCKS)
    k_rms_forward_ring(const __grid_constant__ RmsForwardParams p, int wbf16, Ring ring, unsigned* given_up) {
  extern __shared__ __align__(128) char smem[];
  __shared__ uint32_t s_gave_up;
  volatile uint32_t* gave_up = &s_gave_up;
  RingHead* h = reinterpret_cast<RingHead*>(smem);
  char* slots = smem + kRingHead;
  grid_dependency_sync();
  const bool res = p.residual != nullptr;
  RowFeed feed{h, slots, {static_cast<const char*>(p.x), static_cast<const char*>(p.residual), nullptr},
               {p.ld_x * T::kBytes, p.ld_r * T::kBytes, 0}, int64_t(blockIdx.x), p.rows, uint32_t(p.cols * T::kBytes),
               uint32_t(ring.second), res ? 2u : 1u, 0};
  feed.start<kVec>(ring, &s_gave_up);
  const int t = threadIdx.x, cols = int(p.cols);
  const float inv = 1.0f / float(cols);
  Two w[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) as_pairs(ring_param<kVec, TH>(p.weight, wbf16, i, cols), w[i]);
  int s = 0, half = 0;
  uint32_t phase = 0, top = 0;
  bool good = true;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    // A warp whose wait was given up still goes through the barriers, but writes no more rows and fetches nothing: its
    // slot's copy may yet land, and a barrier takes no second arrival for the same copy.  (A warp as a whole: the lanes of a
    // block of codes share their maximum.)
    good = __all_sync(kFullMask, good & tc::mbar_wait(tc::smem_addr(&h->full[s]), phase, gave_up));
    const char* slot = slots + s * ring.slot_bytes;
    const char *x_row = feed.at<kVec>(slot, 0, row), *r_row = res ? feed.at<kVec>(slot, 1, row) : nullptr;
    Two x[NV][4], sq(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      as_pairs(ring_piece<T, kVec, TH>(x_row, i, cols), x[i]);
      if (res) {
        Two r[4];
        as_pairs(ring_piece<T, kVec, TH>(r_row, i, cols), r);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i][k] = x[i][k] + r[k];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) sq = fma2(x[i][k], x[i][k], sq);
    }
    float sum[1] = {sum_of(sq)};
    ring_sum<TH>(sum, h, half);
    if (t == 0 && good) feed.next<kVec>(ring, s);  // every thread has the row in registers
    const float rstd = __frsqrt_rn(sum[0] * inv + p.eps);
    if (t == 0 && good && p.rstd != nullptr) p.rstd[row] = rstd;
    const Two r2(rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Eight e;
      if (p.sum != nullptr && good) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i][k].get(e.v[2 * k], e.v[2 * k + 1]);
        ring_store<T, kVec, TH>(p.sum, row * p.ld_s, i, cols, e);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) ((x[i][k] * r2) * w[i][k]).get(e.v[2 * k], e.v[2 * k + 1]);
      if (p.y != nullptr && good) ring_store<T, kVec, TH>(p.y, row * p.ld_y, i, cols, e);
      if (p.amax != nullptr) {  // past the row x and w are 0
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, stored_bits<T>(e.v[k]));
      }
      if (p.codes != nullptr && good) {
        if constexpr (kVec) store_codes(p, row, ring_col<true, TH>(i, 0), e);
        else store_codes_across(p, row, ring_col<false, TH>(i, 0) - (t & 31), t & 31, e);
      }
    }
    if (++s == ring.slots) {
      s = 0;
      phase ^= 1;
    }
    if (row == p.rows - 1 && p.codes != nullptr) pad_scales(p, t, TH);
  }
  if (p.amax != nullptr) fold_amax(p.amax, top);
  __syncthreads();
  if (t == 0 && *gave_up != 0) {
    tc::settle_copies(tc::smem_addr(h->full), uint32_t(ring.slots), feed.issued);
    tc::report_given_up(given_up);
  }
}

template <class T, bool kVec, int TH, int NV, int BLOCKS>
__global__ void __launch_bounds__(TH, BLOCKS)
    k_rms_backward_ring(const __grid_constant__ RmsBackwardParams p, int wbf16, Ring ring, unsigned* given_up) {
  extern __shared__ __align__(128) char smem[];
  __shared__ uint32_t s_gave_up;
  volatile uint32_t* gave_up = &s_gave_up;
  RingHead* h = reinterpret_cast<RingHead*>(smem);
  char* slots = smem + kRingHead;
  grid_dependency_sync();
  const bool add = p.dsum != nullptr;
  RowFeed feed{h, slots, {static_cast<const char*>(p.dy), static_cast<const char*>(p.x), static_cast<const char*>(p.dsum)},
               {p.ld_dy * T::kBytes, p.ld_x * T::kBytes, p.ld_ds * T::kBytes}, int64_t(blockIdx.x), p.rows,
               uint32_t(p.cols * T::kBytes), uint32_t(ring.second), add ? 3u : 2u, 0};
  feed.start<kVec>(ring, &s_gave_up);
  const int t = threadIdx.x, cols = int(p.cols);
  const float inv = 1.0f / float(cols);
  Two dw[NV][4], w[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    as_pairs(ring_param<kVec, TH>(p.weight, wbf16, i, cols), w[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[i][k] = Two(0.0f);
  }
  int s = 0, half = 0;
  uint32_t phase = 0;
  bool good = true;  // as in the forward pass
  float next_rstd = p.rstd[blockIdx.x];  // a row ahead: its latency passes behind the row before
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float rstd = next_rstd;
    if (row + gridDim.x < p.rows) next_rstd = p.rstd[row + gridDim.x];
    good &= tc::mbar_wait(tc::smem_addr(&h->full[s]), phase, gave_up);
    const char* slot = slots + s * ring.slot_bytes;
    const char *dy_row = feed.at<kVec>(slot, 0, row), *x_row = feed.at<kVec>(slot, 1, row);
    const char* ds_row = add ? feed.at<kVec>(slot, 2, row) : nullptr;
    const Two r2(rstd);
    Two along(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (ring_col<kVec, TH>(i, 0) >= cols) continue;
      Two dy[4], x[4];  // past the row zeros, which add nothing
      as_pairs(ring_piece<T, kVec, TH>(dy_row, i, cols), dy);
      as_pairs(ring_piece<T, kVec, TH>(x_row, i, cols), x);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const Two d = dy[k] * (x[k] * r2);
        along = fma2(d, w[i][k], along);
        dw[i][k] = dw[i][k] + d;
      }
    }
    float sum[1] = {sum_of(along)};
    ring_sum<TH>(sum, h, half);
    if (row != blockIdx.x && good && t == 0) feed.next<kVec>(ring, s == 0 ? ring.slots - 1 : s - 1);  // every thread is past the row before
    // dx = rstd (dy w) + xh (-rstd mean(g xh)) + dsum
    const Two c(-rstd * (sum[0] * inv));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (ring_col<kVec, TH>(i, 0) >= cols) continue;
      Two dy[4], x[4], ds[4];
      as_pairs(ring_piece<T, kVec, TH>(dy_row, i, cols), dy);
      as_pairs(ring_piece<T, kVec, TH>(x_row, i, cols), x);
      if (add) {
        as_pairs(ring_piece<T, kVec, TH>(ds_row, i, cols), ds);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) ds[k] = Two(0.0f);
      }
      Eight dx;
#pragma unroll
      for (int k = 0; k < 4; ++k) fma2(x[k] * r2, c, fma2(dy[k] * w[i][k], r2, ds[k])).get(dx.v[2 * k], dx.v[2 * k + 1]);
      if (good) ring_store<T, kVec, TH>(p.dx, row * p.ld_dx, i, cols, dx);
    }
    if (++s == ring.slots) {
      s = 0;
      phase ^= 1;
    }
  }
  float* out = p.workspace + int64_t(blockIdx.x) * cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Eight e;
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[i][k].get(e.v[2 * k], e.v[2 * k + 1]);
    ring_store<F32T, kVec, TH>(out, 0, i, cols, e);
  }
  __syncthreads();
  if (t == 0 && *gave_up != 0) {
    tc::settle_copies(tc::smem_addr(h->full), uint32_t(ring.slots), feed.issued);
    tc::report_given_up(given_up);
  }
}

// Whether rows of `cols` columns go through a ring: enough of them for the prologue of a persistent block to pay, and long
// enough that the rows of a block, one after another, keep memory busy (a warp per row / rings, BF16: forward 12867 x 71 8.4 /
// 19.9 us, 16384 x 256 8.3 / 15.6, 16384 x 512 16.8 / 16.4, 16384 x 1024 35.8 / 28.3; backward 12.5 / 22.6, 16.6 / 16.8, 39.0 /
// 19.3, 117 / 28).
bool ring_rows(int64_t rows, int64_t cols, bool odd, const DeviceInfo& dev) {
  return cols > 256 && cols <= 8192 && rows >= (odd ? 12 : 4) * int64_t(dev.sms);
}

template <class T, bool kVec, int TH, int NV, int BLOCKS>
cudaError_t forward_ring(const RmsForwardParams& p, int wdtype, const DeviceInfo& dev, unsigned* given_up, cudaStream_t stream) {
  const Ring ring = rows_ring(p.cols * T::kBytes + (kVec ? 0 : 30), p.residual != nullptr ? 2 : 1, BLOCKS);
  auto kernel = k_rms_forward_ring<T, kVec, TH, NV, BLOCKS>;
  static std::atomic<unsigned long long> done{0};  // ring.smem goes by the template's arguments
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), int(ring.smem), dev.device, &done);
  if (e != cudaSuccess) return e;
  const int64_t most = BLOCKS * dev.sms;
  return launch_kernel(kernel, dim3(unsigned(p.rows < most ? p.rows : most)), dim3(TH), ring.smem, stream, p, wdtype, ring, given_up);
}

template <class T, bool kVec, int TH, int NV, int BLOCKS>
cudaError_t backward_ring(const RmsBackwardParams& p, int wdtype, const DeviceInfo& dev, unsigned* given_up, unsigned* blocks,
                          cudaStream_t stream) {
  const Ring ring = rows_ring(p.cols * T::kBytes + (kVec ? 0 : 30), p.dsum != nullptr ? 3 : 2, BLOCKS);
  auto kernel = k_rms_backward_ring<T, kVec, TH, NV, BLOCKS>;
  static std::atomic<unsigned long long> done{0};  // ring.smem goes by the template's arguments
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), int(ring.smem), dev.device, &done);
  if (e != cudaSuccess) return e;
  const int64_t most = BLOCKS * dev.sms, room = rms_partials(p.rows, p.cols);
  *blocks = unsigned(most < room ? most : room);
  return launch_kernel(kernel, dim3(*blocks), dim3(TH), ring.smem, stream, p, wdtype, ring, given_up);
}

template <class T>
cudaError_t forward(const RmsForwardParams& p, int wdtype, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t pieces = (p.cols + 7) / 8;
  auto launch = [&](auto kernel, int64_t blocks, int threads) {
    return launch_kernel(kernel, dim3(unsigned(blocks)), dim3(threads), 0, stream, p, wdtype);
  };
  auto direct = [&](auto vec) {
    constexpr bool kVec = decltype(vec)::value;
    // a block per row of more than 256 columns: these rows are few (128 x 627 BF16 with a warp each 7.1 us, 64 x 1024 4.9; with a
    // block 2.7 and 2.5)
    if (pieces <= 32) return launch(k_rms_forward<T, false, kVec, 1>, (p.rows + 7) / 8, 256);
    auto threads = [&](int nv) { return int(((pieces + nv - 1) / nv + 31) / 32 * 32); };
    if (pieces <= 1024) return launch(k_rms_forward<T, true, kVec, 1>, p.rows, threads(1));
    if (pieces <= 2048) return launch(k_rms_forward<T, true, kVec, 2>, p.rows, threads(2));
    return launch(k_rms_forward<T, true, kVec, 4>, p.rows, threads(4));
  };
  const bool odd = p.cols % 8 != 0;
  if (ring_rows(p.rows, p.cols, odd, dev) && (odd || p.vec)) {
    unsigned* given_up = nullptr;
    const cudaError_t e = given_up_address(dev.device, &given_up);
    if (e != cudaSuccess) return e;
    auto ring = [&](auto vec) {
      constexpr bool kVec = decltype(vec)::value, kNarrow = T::kBytes == 2;
      if (pieces <= 64) return forward_ring<T, kVec, 64, 1, kNarrow ? 12 : 10>(p, wdtype, dev, given_up, stream);
      if (pieces <= 128) return forward_ring<T, kVec, 128, 1, 6>(p, wdtype, dev, given_up, stream);
      if (pieces <= 256) return forward_ring<T, kVec, 256, 1, 4>(p, wdtype, dev, given_up, stream);
      if (pieces <= 512) return forward_ring<T, kVec, 256, 2, kNarrow ? 3 : 2>(p, wdtype, dev, given_up, stream);
      // an element per load and store waits longer than it computes: 16384 x 6143 BF16 with codes 193 us, with two blocks 224
      if (pieces <= 768) return forward_ring<T, kVec, 256, 3, kNarrow && !kVec ? 3 : 2>(p, wdtype, dev, given_up, stream);
      return forward_ring<T, kVec, 512, 2, 1>(p, wdtype, dev, given_up, stream);
    };
    return odd ? ring(std::false_type{}) : ring(std::true_type{});
  }
  if (pieces <= 4096) return odd ? direct(std::false_type{}) : direct(std::true_type{});
  return launch_kernel(k_rms_forward_long<T>, dim3(unsigned(p.rows)), dim3(1024), 0, stream, p, wdtype);
}

// Blocks per SM without a ring: more rows of partial sums cost more than they save (600 x 1024 BF16 6.6 us, with four 8.1, with one
// 7.5; 1800 x 511 8.8, 7.7, 14.0; 12867 x 71 8.7, 9.8, 11.6).
constexpr int64_t kDirectBlocks = 2;
template <class T>
cudaError_t backward(RmsBackwardParams p, int wdtype, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t pieces = (p.cols + 7) / 8;
  const bool block = pieces > 32;
  const int64_t room = rms_partials(p.rows, p.cols), work = block ? p.rows : (p.rows + 7) / 8;
  const int64_t most = kDirectBlocks * dev.sms < room ? kDirectBlocks * dev.sms : room;
  unsigned blocks = unsigned(work < most ? work : most);
  if (blocks == 1) p.workspace = p.dweight;  // one row of partial sums is the sum: 1 x 4096 3.6 us, with a second launch 5.2
  auto run = [&](auto kernel, int threads, size_t smem) {
    return launch_kernel(kernel, dim3(blocks), dim3(threads), smem, stream, p, wdtype);
  };
  auto direct = [&](auto vec) {
    constexpr bool kVec = decltype(vec)::value;
    auto threads = [&](int nv) { return int(((pieces + nv - 1) / nv + 31) / 32 * 32); };
    if (block) return pieces <= 1024 ? run(k_rms_backward<T, true, kVec, 1>, threads(1), 0) : run(k_rms_backward<T, true, kVec, 2>, threads(2), 0);
    return run(k_rms_backward<T, false, kVec, 1>, 256, size_t(8) * size_t(p.cols) * 4);
  };
  const bool odd = p.cols % 8 != 0;
  cudaError_t e;
  if (ring_rows(p.rows, p.cols, odd, dev) && (odd || p.vec)) {
    unsigned* given_up = nullptr;
    e = given_up_address(dev.device, &given_up);
    if (e != cudaSuccess) return e;
    auto ring = [&](auto vec) {
      constexpr bool kVec = decltype(vec)::value, kNarrow = T::kBytes == 2;
      if (pieces <= 64) return backward_ring<T, kVec, 64, 1, kNarrow ? 12 : 8>(p, wdtype, dev, given_up, &blocks, stream);
      if (pieces <= 128) return backward_ring<T, kVec, 128, 1, kNarrow ? 6 : 5>(p, wdtype, dev, given_up, &blocks, stream);
      if (pieces <= 256) return backward_ring<T, kVec, 256, 1, kNarrow ? 4 : 3>(p, wdtype, dev, given_up, &blocks, stream);
      if (pieces <= 512) return backward_ring<T, kVec, 256, 2, kNarrow ? 3 : 2>(p, wdtype, dev, given_up, &blocks, stream);
      if (pieces <= 768) return backward_ring<T, kVec, kNarrow ? 256 : 384, kNarrow ? 3 : 2, kNarrow ? 2 : 1>(p, wdtype, dev, given_up, &blocks, stream);
      return backward_ring<T, kVec, 512, 2, 1>(p, wdtype, dev, given_up, &blocks, stream);
    };
    e = odd ? ring(std::false_type{}) : ring(std::true_type{});
  } else {
    e = pieces > 2048 ? run(k_rms_backward_long<T>, 1024, 0) : odd ? direct(std::false_type{}) : direct(std::true_type{});
  }
  if (e != cudaSuccess || blocks == 1) return e;
  return launch_kernel(k_rms_partials, dim3(unsigned((p.cols + 31) / 32)), dim3(1024), 0, stream,
                       static_cast<const float*>(p.workspace), int(blocks), p.cols, p.dweight);
}

}  // namespace

// A row of partial sums per block of the backward pass: kDirectBlocks per SM, or those of its rings (of BF16, which has more),
// of 152 SMs.  The pass takes no more blocks than that on any device.
int64_t rms_partials(int64_t rows, int64_t cols) {
  const int64_t per_sm = cols <= 256 ? kDirectBlocks : (cols <= 512 ? 12 : (cols <= 1024 ? 6 : (cols <= 2048 ? 4 : (cols <= 4096 ? 3 : kDirectBlocks))));
  const int64_t most = 152 * per_sm;
  return rows < most ? rows : most;
}

cudaError_t launch_rms_forward(const RmsForwardParams& p, int dtype, int wdtype, const DeviceInfo& dev, cudaStream_t stream) {
  return dtype == 0 ? forward<F32T>(p, wdtype, dev, stream) : forward<BF16T>(p, wdtype, dev, stream);
}

cudaError_t launch_rms_backward(const RmsBackwardParams& p, int dtype, int wdtype, const DeviceInfo& dev, cudaStream_t stream) {
  return dtype == 0 ? backward<F32T>(p, wdtype, dev, stream) : backward<BF16T>(p, wdtype, dev, stream);
}

}  // namespace mxfp8
