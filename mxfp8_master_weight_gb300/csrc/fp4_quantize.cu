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
// leave as whole 64-byte pieces of the transposed rows; scale bytes gather in shared memory, four rows to a word, and are
// turned into the layout's words there.
//
// Measured at 16384 x 6144 BF16 (floor at 6.8 TB/s): largest magnitude 33 us (30, HBM); both operands 69 us (46): about 1250
// instructions per thread of 64 values, which three blocks per SM (80 registers, 48 bytes of them spilled) issue in 62 % of the
// slots: neither the slots nor HBM are full.  One operand 42-45 us (38) with four; values 44 us (38).  16384 x 6143: both 83,
// values of rows that start anywhere 66.  F32 16384 x 6144: both 95 us (76), one 81 (68); 16384 x 6143, an element per load, 133
// and 105; 4096 x 4096 20 and 17.  160 x 96 F32: 2.4, 3.9 and 2.4 us.  A weight of 8192 x 8192 transposed 16 us, copied 11.
#include "fp4.cuh"
#include "linear.h"

namespace mxfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;

// Eight elements as they lie: BF16 pairs, or F32 values.
template <class T>
struct Eight {
  static constexpr int W = T::kBytes * 2;
  uint32_t w[W];
  __device__ __forceinline__ float get(int k) const {
    if constexpr (T::kBytes == 4) return __uint_as_float(w[k]);
    else return (k & 1) ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1]);
  }
};

// Elements [0, n) of p, zeros past them.
template <class T>
__device__ __forceinline__ Eight<T> load8(const char* p, int n, bool vec) {
  Eight<T> v;
  if (vec && n >= 8) {
#pragma unroll
    for (int k = 0; k < Eight<T>::W; k += 4) {
      const uint4 a = ld_stream16(p + 4 * k);
      v.w[k] = a.x; v.w[k + 1] = a.y; v.w[k + 2] = a.z; v.w[k + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < Eight<T>::W; ++k) v.w[k] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k < n) {
        const uint32_t b = load_bits<T>(p, k);
        if constexpr (T::kBytes == 4) v.w[k] = b; else v.w[k >> 1] |= b << (16 * (k & 1));
      }
    }
  }
  return v;
}

// Maxima of |x|; BF16 keeps two to a word, whose signs mean nothing.  A NaN stays one.
template <class T>
__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t w) {
  if constexpr (T::kBytes == 4) {
    return max(m, w & 0x7fffffffu);
  } else {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w));
    return r;
  }
}

// ------------------------------------------------------------------------------ largest magnitude
// Items of a row's 8192 values (a dense matrix is one row), four loads under way per thread; a block folds its items into
// one atomic maximum.  A matrix that one block reads in a few rounds is read by one block, which stores its maximum:
// no word has to be cleared before.
constexpr int kAmaxLoads = 4, kAmaxItem = 8 * kThreads * kAmaxLoads;
template <class T>
__global__ void __launch_bounds__(kThreads) k_tensor_amax(const __grid_constant__ Fp4AmaxParams p) {
  __shared__ uint32_t s_max[kThreads / 32];
  grid_dependency_sync();
  const int64_t per_row = (p.cols + kAmaxItem - 1) / kAmaxItem, items = per_row * p.rows;
  int64_t row = blockIdx.x / per_row, part = blockIdx.x - row * per_row;
  const int64_t step_row = gridDim.x / per_row, step_part = gridDim.x - step_row * per_row;
  uint32_t m = 0;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t col = part * kAmaxItem + 8 * threadIdx.x;
    const char* src = static_cast<const char*>(p.in) + (row * p.ld + col) * T::kBytes;
    Eight<T> v[kAmaxLoads];
#pragma unroll
    for (int l = 0; l < kAmaxLoads; ++l) {
      const int64_t left = p.cols - col - l * 8 * kThreads;
      v[l] = load8<T>(src + l * 8 * kThreads * T::kBytes, left >= 8 ? 8 : (left > 0 ? int(left) : 0), p.vec);
    }
#pragma unroll
    for (int l = 0; l < kAmaxLoads; ++l)
#pragma unroll
      for (int k = 0; k < Eight<T>::W; ++k) m = max_abs<T>(m, v[l].w[k]);
    row += step_row;
    part += step_part;
    if (part >= per_row) {
      part -= per_row;
      ++row;
    }
  }
  if constexpr (T::kBytes == 2) m = max(m << 16 & 0x7fff0000u, m & 0x7fff0000u);
  m = __reduce_max_sync(kFullMask, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, s_max[w]);
    m = canonical_nan<F32T>(m);
    uint32_t* out = reinterpret_cast<uint32_t*>(p.amax);
    if (p.store) *out = m;
    else atomicMax(out, m);
  }
}

// ------------------------------------------------------------------------------ quantisation
// The largest magnitudes of eight blocks as F32 bits: own[i], or those of two threads' halves.  BF16 sends two to a word.
template <class T>
__device__ __forceinline__ void join8(const uint32_t (&own)[8], int lane_mask, uint32_t (&m)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    if constexpr (T::kBytes == 4) {
      m[i] = max(own[i], __shfl_xor_sync(kFullMask, own[i], lane_mask));
      m[i + 1] = max(own[i + 1], __shfl_xor_sync(kFullMask, own[i + 1], lane_mask));
    } else {
      uint32_t two = own[i] | own[i + 1] << 16;
      two = __vmaxu2(two, __shfl_xor_sync(kFullMask, two, lane_mask));
      m[i] = two << 16;
      m[i + 1] = two & 0xffff0000u;
    }
  }
}

// The tile's transposed rows: word w of row j at w ^ (j / 32 * 2), 64 bytes each.
__device__ __forceinline__ void store_turned(const uint32_t (&s_col)[kTile][17], uint8_t* out, int64_t ld, bool vec, uint32_t rb,
                                             uint32_t cb, int64_t rows, int64_t cols) {
  const int64_t rows_left = rows - int64_t(rb) * kTile;
  const int width = rows_left < kTile ? int(rows_left + 1) / 2 : kTile / 2;  // bytes of a transposed row
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = (int(threadIdx.x) >> 2) + 64 * h, u = threadIdx.x & 3;
    if (int64_t(cb) * kTile + j >= cols) continue;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = s_col[j][(4 * u + k) ^ ((j >> 5) << 1)];
    uint8_t* q = out + (int64_t(cb) * kTile + j) * ld + int64_t(rb) * (kTile / 2) + 16 * u;
    if (vec && 16 * u + 16 <= width) {
      *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (16 * u + k < width) q[k] = uint8_t(w[k >> 2] >> (8 * (k & 3)));
    }
  }
}

template <class T, bool kRow, bool kCol>
__global__ void __launch_bounds__(kThreads, T::kBytes == 4 ? 2 : (kRow && kCol ? 3 : 4)) k_fp4_quantize(const __grid_constant__ Fp4QuantizeParams p) {
  constexpr int W = Eight<T>::W;
  __shared__ float s_mult[128];  // by scale byte: a read of it for eight operations of arithmetic
  // scale bytes [direction][block][row], four rows to a word
  __shared__ uint32_t s_scale[2][8][kTile / 4 + 4];
  __shared__ __align__(16) uint32_t s_col[kTile][17];
  grid_dependency_sync();
  const float G = *p.amax, S = fp4_tensor_scale(G);
  const bool tiny = fp4_tiny(G), bad = isnan(S);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t < 128) s_mult[t] = fp4_multiplier(uint32_t(t), S);
  const uint32_t tiles_c = uint32_t((p.cols + kTile - 1) / kTile);
  const uint32_t rb = blockIdx.x / tiles_c, cb = blockIdx.x - rb * tiles_c;
  const int r8 = warp * 16 + (lane >> 4) * 8, c8 = (lane & 15) * 8;
  const int64_t row = int64_t(rb) * kTile + r8, col = int64_t(cb) * kTile + c8;
  const int n = p.cols - col >= 8 ? 8 : (p.cols > col ? int(p.cols - col) : 0);
  const int left = p.rows - row >= 8 ? 8 : (p.rows > row ? int(p.rows - row) : 0);
  Eight<T> v[8];
  const char* src = static_cast<const char*>(p.in) + (row * p.ld + col) * T::kBytes;
  const int64_t pitch = p.ld * T::kBytes;
  // BF16 rows that start anywhere are read by 32-bit words, shifted by half a word where they start inside one; words
  // that would reach past the matrix are left to the loads by the element.
  const bool words = T::kBytes == 2 && !p.vec_in && n == 8 && left == 8 && (row > 0 || col > 0) && (row + 8 < p.rows || col + 8 < p.cols);
  if (words) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(src + i * pitch);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(at & ~uintptr_t(3));
      uint32_t raw[5];
#pragma unroll
      for (int k = 0; k < 4; ++k) raw[k] = w[k];
      raw[4] = w[at & 2 ? 4 : 3];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i].w[k % W] = __funnelshift_r(raw[k], raw[k + 1], at & 2 ? 16 : 0);
    }
  } else if (left == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = load8<T>(src + i * pitch, n, p.vec_in);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = load8<T>(src + i * pitch, i < left ? n : 0, p.vec_in);
  }
  uint32_t rm[8], cm[W];
#pragma unroll
  for (int k = 0; k < W; ++k) cm[k] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      m = max_abs<T>(m, v[i].w[k]);
      cm[k] = max_abs<T>(cm[k], v[i].w[k]);
    }
    rm[i] = T::kBytes == 4 ? m : max(m & 0x7fffu, m >> 16 & 0x7fffu);
  }
  __syncthreads();
  if constexpr (kRow) {
    uint32_t m[8];
    join8<T>(rm, 1, m);
    // blocks past the last column or row hold zeros: their scales are zero too, unless S is NaN
    const bool some = (col & ~int64_t(15)) < p.cols;
    uint8_t* q = p.q_r + row * p.ld_r + (col >> 1);
    uint32_t bytes[2] = {0, 0}, codes[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      uint32_t s2 = fp4_block_scales(__uint_as_float(m[i]), __uint_as_float(m[i + 1]), S, tiny);
      if (bad) s2 = !some || i >= left ? 0 : (i + 1 >= left ? s2 & 0xffu : s2);
      bytes[i >> 2] |= s2 << (16 * (i >> 1 & 1));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t s = s2 >> (8 * h) & 0xffu;
        const float f = s_mult[s];
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) mul2_rn(v[i + h].get(k), v[i + h].get(k + 1), f, f, y[k], y[k + 1]);
        codes[i + h] = fp4_codes(y);
      }
    }
    if (p.vec_r && n == 8 && left == 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) *reinterpret_cast<uint32_t*>(q + i * p.ld_r) = codes[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i < left && 2 * k < n) q[i * p.ld_r + k] = uint8_t(codes[i] >> (8 * k));
      }
    }
    s_scale[0][c8 >> 4][(r8 >> 2) + (lane & 1)] = lane & 1 ? bytes[1] : bytes[0];  // block c8 / 16, four rows by each of its two threads
  }
  if constexpr (kCol) {
    uint32_t own[8], m[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) own[k] = T::kBytes == 4 ? cm[k % W] : (cm[k >> 1] >> (16 * (k & 1))) & 0x7fffu;
    join8<T>(own, 16, m);
    const bool some = (row & ~int64_t(15)) < p.rows;
    uint32_t bytes[2] = {0, 0};
    uint32_t* turned = &s_col[c8][(r8 >> 3) ^ ((c8 >> 5) << 1)];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      uint32_t s2 = fp4_block_scales(__uint_as_float(m[k]), __uint_as_float(m[k + 1]), S, tiny);
      if (bad) s2 = !some || k >= n ? 0 : (k + 1 >= n ? s2 & 0xffu : s2);
      bytes[k >> 2] |= s2 << (16 * (k >> 1 & 1));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t s = s2 >> (8 * h) & 0xffu;
        const float f = s_mult[s];
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) mul2_rn(v[i].get(k + h), v[i + 1].get(k + h), f, f, y[i], y[i + 1]);
        turned[17 * (k + h)] = fp4_codes(y);
      }
    }
    s_scale[1][warp][(c8 >> 2) + (lane >> 4)] = lane & 16 ? bytes[1] : bytes[0];  // block `warp`, likewise
  }
  __syncthreads();
  // The tile's scales: two tiles of the layout along k for each direction, if both are there.  A thread turns four words, of four
  // blocks, into the words of four rows.
  const int which = t >> 6, tile = (t >> 5) & 1, quad = lane;
  if (t < 128) {
    const int64_t tile_cols = scale_tile_cols(((which == 0 ? p.cols : p.rows) + 15) / 16);
    const int64_t r128 = which == 0 ? rb : cb, at = 2 * int64_t(which == 0 ? cb : rb) + tile;
    if ((which == 0 ? kRow : kCol) && at < tile_cols) {
      uint32_t w[4], x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = s_scale[which][4 * tile + j][quad];
      x[0] = __byte_perm(w[0], w[1], 0x5140);  // of rows 0 and 1, blocks 0 and 1
      x[1] = __byte_perm(w[2], w[3], 0x5140);
      x[2] = __byte_perm(w[0], w[1], 0x7362);
      x[3] = __byte_perm(w[2], w[3], 0x7362);
      uint8_t* s = (which == 0 ? p.s_r : p.s_c) + (r128 * tile_cols + at) * 512 + (quad & 7) * 64 + (quad >> 3) * 4;
      *reinterpret_cast<uint32_t*>(s) = __byte_perm(x[0], x[1], 0x5410);
      *reinterpret_cast<uint32_t*>(s + 16) = __byte_perm(x[0], x[1], 0x7632);
      *reinterpret_cast<uint32_t*>(s + 32) = __byte_perm(x[2], x[3], 0x5410);
      *reinterpret_cast<uint32_t*>(s + 48) = __byte_perm(x[2], x[3], 0x7632);
    }
  }
  if constexpr (kCol) {
    store_turned(s_col, p.q_c, p.ld_c, p.vec_c, rb, cb, p.rows, p.cols);
  }
}

// ------------------------------------------------------------------------------ values
// A thread restores blocks of 16, 8 bytes of codes and one scale each, a warp 512 columns of kRestoreRows rows, whose loads
// are all under way at once.  Rows that start anywhere go through the warp's shared memory and out as 32-bit words aligned in
// the output, neighbours across the lanes (BF16: a lone value at either end where the row starts between words).
constexpr int kRestoreRows = 2;  // 16384 x 6144 BF16 43.9 us; one row 45.6, four 46.3
template <class T>
struct RestoreLine {
  static constexpr int kWords = 4 * T::kBytes;  // of a block's values
  uint32_t w[32 * (kWords + 1)];                // a word apart, against bank conflicts
};
template <class T>
__device__ __forceinline__ void restore_row(const Fp4RestoreParams& p, const uint2& codes, uint32_t byte, float r, int64_t row,
                                            uint32_t part, RestoreLine<T>* s_line) {
  constexpr int kWords = RestoreLine<T>::kWords;
  const uint32_t lane = threadIdx.x & 31;
  const int64_t b = int64_t(part) * 32 + lane;
  const int n = p.cols - 16 * b >= 16 ? 16 : (p.cols > 16 * b ? int(p.cols - 16 * b) : 0);
  uint32_t s;  // the scale as two F16: code times scale is exact there (six bits, from 2^-10 to 2688)
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s) : "h"(static_cast<uint16_t>(byte | byte << 8)));
  uint32_t h[8];
  fp4_values(codes.x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
  fp4_values(codes.y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
  float v[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[k]) : "r"(s));
    mul2_rn(f16_lo(h[k]), f16_hi(h[k]), r, r, v[2 * k], v[2 * k + 1]);
  }
  uint32_t o[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) o[k] = T::kBytes == 4 ? __float_as_uint(v[k % 16]) : bf16x2_rn(v[2 * k % 16], v[(2 * k + 1) % 16]);
  char* out = static_cast<char*>(p.out) + (row * p.ld_o + 16 * b) * T::kBytes;
  if (p.vec_out) {
    if (n == 16 && p.vec_out == 2) {
#pragma unroll
      for (int k = 0; k < kWords; k += 8)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + 4 * k), "r"(o[k]), "r"(o[k + 1]),
                     "r"(o[k + 2]), "r"(o[k + 3]), "r"(o[k + 4]), "r"(o[k + 5]), "r"(o[k + 6]), "r"(o[k + 7])
                     : "memory");
    } else if (n == 16) {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) *reinterpret_cast<uint4*>(out + 4 * k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (k < n) store_bits<T>(out, k, T::kBytes == 4 ? o[k % kWords] : o[k >> 1] >> (16 * (k & 1)));
    }
    return;
  }
  uint32_t* line = s_line[threadIdx.x >> 5].w;
#pragma unroll
  for (int k = 0; k < kWords; ++k) line[lane * (kWords + 1) + k] = o[k];
  __syncwarp();
  auto word = [&](int i) { return line[(i / kWords) * (kWords + 1) + i % kWords]; };
  const int64_t first = int64_t(part) * 512;
  const int width = p.cols - first < 512 ? int(p.cols - first) : 512;
  char* start = static_cast<char*>(p.out) + (row * p.ld_o + first) * T::kBytes;
  if constexpr (T::kBytes == 4) {
    for (int i = int(lane); i < width; i += 32) reinterpret_cast<uint32_t*>(start)[i] = word(i);
  } else {
    const int head = int(reinterpret_cast<uintptr_t>(start) >> 1) & 1, pairs = (width - head) / 2;
    uint32_t* words = reinterpret_cast<uint32_t*>(start + 2 * head);
    if (head) {
      for (int i = int(lane); i < pairs; i += 32) words[i] = __funnelshift_r(word(i), 2 * i + 2 < width ? word(i + 1) : 0u, 16);
    } else {
      for (int i = int(lane); i < pairs; i += 32) words[i] = word(i);
    }
    auto half = [&](int i) { return word(i >> 1) >> (16 * (i & 1)) & 0xffffu; };
    uint16_t* ends = reinterpret_cast<uint16_t*>(start);
    if (lane == 0 && head) ends[0] = uint16_t(half(0));
    if (lane == 1 && ((width - head) & 1)) ends[width - 1] = uint16_t(half(width - 1));
  }
  __syncwarp();
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_fp4_restore(const __grid_constant__ Fp4RestoreParams p) {
  __shared__ RestoreLine<T> s_line[kThreads / 32];
  grid_dependency_sync();
  const int64_t nb = (p.cols + 15) / 16, tile_cols = scale_tile_cols(nb);
  const uint32_t per_row = uint32_t((nb + 31) / 32), lane = threadIdx.x & 31;
  const uint32_t rows = blockIdx.x / per_row, part = blockIdx.x - rows * per_row;
  const int64_t row = (int64_t(rows) * (kThreads / 32) + (threadIdx.x >> 5)) * kRestoreRows, b = int64_t(part) * 32 + lane;
  if (row >= p.rows) return;  // whole warps
  const int n = p.cols - 16 * b >= 16 ? 16 : (p.cols > 16 * b ? int(p.cols - 16 * b) : 0);
  uint2 codes[kRestoreRows];
  uint32_t byte[kRestoreRows];
#pragma unroll
  for (int i = 0; i < kRestoreRows; ++i) {
    codes[i] = make_uint2(0, 0);
    byte[i] = 0;
    if (row + i >= p.rows || n == 0) continue;
    const uint8_t* q = p.q + (row + i) * p.ld_q + 8 * b;
    byte[i] = p.s[scale_at(row + i, b, tile_cols)] & 0x7fu;
    if (p.vec_q && n == 16) {
      codes[i] = *reinterpret_cast<const uint2*>(q);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t two = 2 * k < n ? uint32_t(q[k]) << (8 * (k & 3)) : 0u;
        if (k < 4) codes[i].x |= two; else codes[i].y |= two;
      }
    }
  }
  const float r = __frcp_rn(fp4_tensor_scale(*p.amax));
#pragma unroll
  for (int i = 0; i < kRestoreRows; ++i)
    if (row + i < p.rows) restore_row<T>(p, codes[i], byte[i], r, row + i, part, s_line);
}

// ------------------------------------------------------------------------------ weights
// Codes [rows][cols] as they lie densely to rows with the contraction along them: as they are, or (kTurn) transposed.  The
// tile and the threads are the quantisation's.  Dense rows of a width that is no multiple of 8 start on any byte: their eight
// codes are put together from bytes.
__device__ __forceinline__ uint32_t load_codes4(const uint8_t* q, int bytes, bool vec) {
  if (vec && bytes == 4) return *reinterpret_cast<const uint32_t*>(q);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < bytes) w |= uint32_t(q[k]) << (8 * k);
  return w;
}

template <bool kTurn>
__global__ void __launch_bounds__(kThreads) k_fp4_lay_out(const __grid_constant__ Fp4LayOutParams p) {
  __shared__ __align__(16) uint32_t s_col[kTile][17];
  grid_dependency_sync();
  const uint32_t tiles_c = uint32_t((p.cols + kTile - 1) / kTile);
  const uint32_t rb = blockIdx.x / tiles_c, cb = blockIdx.x - rb * tiles_c;
  const int t = threadIdx.x, lane = t & 31, r8 = (t >> 5) * 16 + (lane >> 4) * 8, c8 = (lane & 15) * 8;
  const int64_t row = int64_t(rb) * kTile + r8, col = int64_t(cb) * kTile + c8;
  const int bytes = p.cols - col >= 8 ? 4 : (p.cols > col ? int(p.cols - col) / 2 : 0);
  uint32_t w[8];  // eight codes of eight rows
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = row + i < p.rows ? load_codes4(p.q + (row + i) * p.ld_q + (col >> 1), bytes, p.vec_q) : 0u;
  if constexpr (!kTurn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint8_t* o = p.out + (row + i) * p.ld_o + (col >> 1);
      if (row + i >= p.rows) continue;
      if (p.vec_out && bytes == 4) {
        *reinterpret_cast<uint32_t*>(o) = w[i];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < bytes) o[k] = uint8_t(w[i] >> (8 * k));
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t q = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) q |= (w[i] >> (4 * k) & 15u) << (4 * i);
      s_col[c8 + k][(r8 >> 3) ^ ((c8 >> 5) << 1)] = q;
    }
    __syncthreads();
    store_turned(s_col, p.out, p.ld_o, p.vec_out, rb, cb, p.rows, p.cols);
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

int64_t amax_items(const Fp4AmaxParams& p) { return (p.cols + kAmaxItem - 1) / kAmaxItem * p.rows; }

// One block: rounds of 8192 values, about 0.3 us each, against a cleared word and a second launch.
bool one_block_amax(const Fp4AmaxParams& p) { return amax_items(p) <= 4; }

cudaError_t launch_tensor_amax(const Fp4AmaxParams& p, int dtype, const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t items = amax_items(p), most = 8 * int64_t(dev.sms);
  const dim3 grid(p.store ? 1u : unsigned(items < most ? items : most));
  return dtype == 0 ? launch_kernel(k_tensor_amax<F32T>, grid, dim3(kThreads), 0, stream, p)
                    : launch_kernel(k_tensor_amax<BF16T>, grid, dim3(kThreads), 0, stream, p);
}

cudaError_t launch_fp4_quantize(const Fp4QuantizeParams& p, int dtype, cudaStream_t stream) {
  return dtype == 0 ? quantize<F32T>(p, stream) : quantize<BF16T>(p, stream);
}

cudaError_t launch_fp4_restore(const Fp4RestoreParams& p, int dtype, cudaStream_t stream) {
  const int64_t nb = (p.cols + 15) / 16;
  constexpr int kRows = kThreads / 32 * kRestoreRows;
  const dim3 grid(unsigned((p.rows + kRows - 1) / kRows * ((nb + 31) / 32)));
  return dtype == 0 ? launch_kernel(k_fp4_restore<F32T>, grid, dim3(kThreads), 0, stream, p)
                    : launch_kernel(k_fp4_restore<BF16T>, grid, dim3(kThreads), 0, stream, p);
}

cudaError_t launch_fp4_lay_out(const Fp4LayOutParams& p, cudaStream_t stream) {
  const dim3 grid(unsigned(tiles(p.rows, p.cols)));
  return p.transpose ? launch_kernel(k_fp4_lay_out<true>, grid, dim3(kThreads), 0, stream, p)
                     : launch_kernel(k_fp4_lay_out<false>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace mxfp8
