// 8-bit activation checkpoints: E4M3 codes with one E8M0 scale per 128 values, along the rows
// and along the columns of an activation, from one read; and the values a copy stands for.
//
//   e = floor(log2(max |x| of the block)) - 8 (clamped at -127),  code = E4M3(x * 2^-e),
//   restored = decode(code) * 2^e
//
// The multiplication by a power of two is exact, so a code carries one rounding (nearest-even,
// saturating at 448: a block maximum in [448, 512) * 2^e becomes 448 * 2^e).
//
// Both kernels are streaming passes bound by HBM: save moves 4 (BF16) or 6 (F32) bytes per
// element and two directions, restore 3 or 5.  A block of 256 threads owns one 128x128 tile --
// the smallest piece that holds whole blocks of both directions -- in registers: thread t has
// columns 8 (t % 16) .. + 7 of rows t / 16 + 16 p, p < 8, so a row's maximum is a butterfly over
// 16 lanes, a column's one shuffle and a pass through shared memory, and every code row leaves
// as 128 contiguous bytes.
#include "common.cuh"
#include "linear.h"

namespace mxfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = kCkptBlock;
constexpr int kPasses = 8;   // rows per thread
constexpr int kRowStep = 16; // rows between a thread's passes

// Eight consecutive elements as 32-bit words: BF16 pairs or F32 values; one access of 16 or 32 bytes.
template <class T>
struct Eight {
  static constexpr int W = T::kBytes * 2;
  uint32_t w[W];
  __device__ __forceinline__ float get(int k) const {
    if constexpr (T::kBytes == 4) {
      return __uint_as_float(w[k]);
    } else {
      return (k & 1) ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1]);
    }
  }
};

// Elements [0, n) of p, zeros past them.
template <class T>
__device__ __forceinline__ Eight<T> load_eight(const char* p, int n, bool vec) {
  Eight<T> v;
  if (vec && n >= 8) {
    if constexpr (T::kBytes == 4) {
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                     "=r"(v.w[7])
                   : "l"(p));
    } else {
      const uint4 c = ld_stream16(p);
      v.w[0] = c.x; v.w[1] = c.y; v.w[2] = c.z; v.w[3] = c.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < Eight<T>::W; ++i) v.w[i] = 0;
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

__device__ __forceinline__ void store_codes(uint8_t* p, uint2 q, int n, bool vec) {
  if (vec && n >= 8) {
    *reinterpret_cast<uint2*>(p) = q;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = static_cast<uint8_t>((k < 4 ? q.x : q.y) >> (8 * (k & 3)));
  }
}

template <class T>
__device__ __forceinline__ uint2 encode(const Eight<T>& v, const float (&mult)[8]) {
  float p[8];
#pragma unroll
  for (int k = 0; k < 8; k += 2) mul2_rn(v.get(k), v.get(k + 1), mult[k], mult[k + 1], p[k], p[k + 1]);
  return make_uint2(e4m3x2_rn_sat(p[0], p[1]) | (e4m3x2_rn_sat(p[2], p[3]) << 16),
                    e4m3x2_rn_sat(p[4], p[5]) | (e4m3x2_rn_sat(p[6], p[7]) << 16));
}

// |x| of a pair or value, as the maxima take it: non-negative bit patterns order as their values,
// NaN above infinity.  BF16 keeps two per word.
template <class T>
__device__ __forceinline__ uint32_t abs_bits(uint32_t w) { return w & T::kAbsMask; }
template <class T>
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
  if constexpr (T::kBytes == 4) return max(a, b); else return __vmaxu2(a, b);
}
// Scale byte of one |x| pattern of T.
template <class T>
__device__ __forceinline__ uint32_t scale_of(uint32_t bits) { return e8m0_from_bits<T>(bits); }

// The tile's 128 scales of one direction, which lie 4 bytes apart in one 512-byte scale tile: entry
// r of block `b`.  The last block also zeroes the padding entries up to a whole group of four.
__device__ __forceinline__ void store_scales(uint8_t* s, int64_t r128, int64_t b, int64_t nblocks, int r, uint32_t byte) {
  uint8_t* p = s + (r128 * scale_tile_cols(nblocks) + (b >> 2)) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3);
  *p = static_cast<uint8_t>(byte);
  if (b == nblocks - 1) {
    for (int i = int(b & 3) + 1; i < 4; ++i) *++p = 0;
  }
}

template <class T, bool kRow, bool kCol>
__global__ void __launch_bounds__(kThreads) k_checkpoint_save(const __grid_constant__ CheckpointSaveParams p) {
  constexpr int W = Eight<T>::W, kPerWord = 4 / T::kBytes;
  __shared__ uint32_t s_max[kThreads / 32][kTile / kPerWord];  // per warp: column maxima of |x|
  __shared__ __align__(16) float s_mult[kTile];
  __shared__ uint8_t s_row[kTile];
  grid_dependency_sync();
  const uint32_t tcols = uint32_t((p.cols + kTile - 1) / kTile);
  const uint32_t rb = blockIdx.x / tcols, cb = blockIdx.x % tcols;
  const int t = threadIdx.x, c8 = t % 16 * 8, r0 = t / 16;
  const int64_t col = int64_t(cb) * kTile + c8, row = int64_t(rb) * kTile + r0;
  const int n = int(p.cols - col < 8 ? (p.cols > col ? p.cols - col : 0) : 8);
  const int left = int(p.rows - row < kTile ? (p.rows > row ? p.rows - row : 0) : kTile);  // rows from this thread's first
  Eight<T> v[kPasses];
  const char* src = static_cast<const char*>(p.in) + (row * p.ld + col) * T::kBytes;
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    v[i] = load_eight<T>(src + i * kRowStep * p.ld * T::kBytes, kRowStep * i < left ? n : 0, p.vec_in);
  uint32_t cm[W], rm[kPasses];
#pragma unroll
  for (int k = 0; k < W; ++k) cm[k] = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const uint32_t a = abs_bits<T>(v[i].w[k]);
      if constexpr (kRow) m = max_bits<T>(m, a);
      if constexpr (kCol) cm[k] = max_bits<T>(cm[k], a);
    }
    rm[i] = T::kBytes == 4 ? m : max(m & 0xffffu, m >> 16);
  }
  if constexpr (kRow) {
    // over the row's 16 threads; BF16: two rows per word
    if constexpr (T::kBytes == 2) {
#pragma unroll
      for (int i = 0; i < kPasses; i += 2) {
        uint32_t m = rm[i] | (rm[i + 1] << 16);
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) m = __vmaxu2(m, __shfl_xor_sync(kFullMask, m, off));
        rm[i] = m & 0xffffu;
        rm[i + 1] = m >> 16;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) rm[i] = max(rm[i], __shfl_xor_sync(kFullMask, rm[i], off));
      }
    }
    uint8_t* q = p.q_r + row * p.ld_r + col;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t s = scale_of<T>(rm[i]);
      if (c8 == 0) s_row[r0 + kRowStep * i] = static_cast<uint8_t>(s);
      const float f = scale_multiplier(s);
      const float mult[8] = {f, f, f, f, f, f, f, f};
      if (kRowStep * i < left) store_codes(q + i * kRowStep * p.ld_r, encode<T>(v[i], mult), n, p.vec_r);
    }
  }
  if constexpr (kCol) {
#pragma unroll
    for (int k = 0; k < W; ++k) cm[k] = max_bits<T>(cm[k], __shfl_xor_sync(kFullMask, cm[k], 16));
    if (t % 32 < 16) {
#pragma unroll
      for (int k = 0; k < W; ++k) s_max[t / 32][c8 / kPerWord + k] = cm[k];
    }
  }
  __syncthreads();
  if constexpr (kRow) {  // rows past the last are padding: their maxima are 0, and so is the byte
    if (t >= kTile) store_scales(p.s_r, rb, cb, tcols, t - kTile, s_row[t - kTile]);
  }
  if constexpr (kCol) {
    if (t < kTile) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) m = max_bits<T>(m, s_max[w][t / kPerWord]);
      if constexpr (T::kBytes == 2) m = t & 1 ? m >> 16 : m & 0xffffu;
      const uint32_t s = scale_of<T>(m);
      s_mult[t] = scale_multiplier(s);
      store_scales(p.s_c, cb, rb, (p.rows + kTile - 1) / kTile, t, s);
    }
    __syncthreads();
    float mult[8];
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&s_mult[c8 + k]);
      mult[k] = f.x; mult[k + 1] = f.y; mult[k + 2] = f.z; mult[k + 3] = f.w;
    }
    uint8_t* q = p.q_c + row * p.ld_c + col;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (kRowStep * i < left) store_codes(q + i * kRowStep * p.ld_c, encode<T>(v[i], mult), n, p.vec_c);
  }
}

// 2^(s - 127); NaN for the NaN scale 255.
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : (s == 0u ? 0x00400000u : s << 23));
}

// Two E4M3 codes (low 16 bits) as floats, exactly.
__device__ __forceinline__ void decode2(uint32_t q, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(q)));
  lo = f16_lo(h);
  hi = f16_hi(h);
}

// Eight codes times their factors.
template <class T>
__device__ __forceinline__ Eight<T> decode8(uint2 q, const float (&f)[8]) {
  float y[8];
  decode2(q.x & 0xffffu, y[0], y[1]);
  decode2(q.x >> 16, y[2], y[3]);
  decode2(q.y & 0xffffu, y[4], y[5]);
  decode2(q.y >> 16, y[6], y[7]);
  Eight<T> w;
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    mul2_rn(y[k], y[k + 1], f[k], f[k + 1], y[k], y[k + 1]);
    if constexpr (T::kBytes == 4) {
      w.w[k] = __float_as_uint(y[k]);
      w.w[k + 1] = __float_as_uint(y[k + 1]);
    } else {
      w.w[k / 2] = bf16x2_rn(y[k], y[k + 1]);
    }
  }
  return w;
}

template <class T>
__device__ __forceinline__ void store_eight(char* dst, const Eight<T>& w, int n, bool vec) {
  if (vec && n == 8) {
    if constexpr (T::kBytes == 4) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w.w[0]), "r"(w.w[1]),
                   "r"(w.w[2]), "r"(w.w[3]), "r"(w.w[4]), "r"(w.w[5]), "r"(w.w[6]), "r"(w.w[7])
                   : "memory");
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) store_bits<T>(dst, k, T::kBytes == 4 ? w.w[k % Eight<T>::W] : w.w[k >> 1] >> (16 * (k & 1)));
  }
}

// The kernel issues about 6 instructions per element; addresses and scale bytes are offsets from a
// row's first (measured: with 64-bit indexes per row it issued 19 and took 62 instead of 45.5 us on
// 16384x6144 to BF16).
template <class T, bool kCol>
__global__ void __launch_bounds__(kThreads) k_checkpoint_restore(const __grid_constant__ CheckpointRestoreParams p) {
  grid_dependency_sync();
  const uint32_t tcols = uint32_t((p.cols + kTile - 1) / kTile);
  const uint32_t rb = blockIdx.x / tcols, cb = blockIdx.x % tcols;
  const int t = threadIdx.x, c8 = t % 16 * 8, r0 = t / 16;
  const int64_t col = int64_t(cb) * kTile + c8, row = int64_t(rb) * kTile + r0;
  const int n = int(p.cols - col < 8 ? (p.cols > col ? p.cols - col : 0) : 8);
  const int left = n == 0 ? 0 : int(p.rows - row < kTile ? (p.rows > row ? p.rows - row : 0) : kTile);
  if (left == 0 && p.vec_out) return;  // (else the warp's rows go out together)
  const uint8_t* src = p.q + row * p.ld_q + col;
  const int64_t q_step = kRowStep * p.ld_q, o_step = kRowStep * p.ld_o * T::kBytes;
  char* dst = static_cast<char*>(p.out) + (row * p.ld_o + col) * T::kBytes;
  // the tile's 512 scale bytes: entry (r, b) at (r % 32) * 16 + (r / 32) * 4 + b % 4
  const int64_t blocks = kCol ? (p.rows + kTile - 1) / kTile : tcols;
  const uint32_t entry = kCol ? cb : rb, block = kCol ? rb : cb;
  const uint8_t* s = p.s + (entry * scale_tile_cols(blocks) + (block >> 2)) * 512 + (block & 3);
  uint2 q[kPasses];
  uint32_t byte[8];
  if (p.vec_q && n == 8 && left > kRowStep * (kPasses - 1)) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) q[i] = *reinterpret_cast<const uint2*>(src + i * q_step);
  } else {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      q[i] = make_uint2(0, 0);
      if (kRowStep * i >= left) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t b = k < n ? src[i * q_step + k] : 0u;
        if (k < 4) q[i].x |= b << (8 * k); else q[i].y |= b << (8 * (k - 4));
      }
    }
  }
  // rowwise: the scale of row r0 + 16 i; columnwise: of column c8 + k.  Both lie inside the tile's
  // padding to 128, so all eight may be read.
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = kCol ? c8 + i : r0 + kRowStep * i;
    byte[i] = s[(r & 31) * 16 + (r >> 5) * 4];
  }
  float f[8];
  if constexpr (kCol) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = scale_value(byte[k]);
  }
  if (!p.vec_out) {
    // Rows that start anywhere: a warp's two rows go through its own shared memory, and out again as
    // 32-bit words aligned in the output, neighbours across the lanes (BF16: a lone value at
    // either end where the row starts between words).
    __shared__ __align__(16) char s_rows[kThreads / 32][2][kTile * T::kBytes];
    const int lane = t & 31, width = int(p.cols - int64_t(cb) * kTile < kTile ? p.cols - int64_t(cb) * kTile : kTile);
    const int wrow = r0 & ~1;  // the warp's first row
    const int64_t row1 = int64_t(rb) * kTile + wrow;
    const int wleft = int(p.rows - row1 < kTile ? p.rows - row1 : kTile);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if constexpr (!kCol) {
        const float one = scale_value(byte[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = one;
      }
      const Eight<T> e = decode8<T>(q[i], f);
#pragma unroll
      for (int k = 0; k < Eight<T>::W; k += 4)
        *reinterpret_cast<uint4*>(&s_rows[t / 32][r0 & 1][c8 * T::kBytes + 4 * k]) = make_uint4(e.w[k], e.w[k + 1], e.w[k + 2], e.w[k + 3]);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (kRowStep * i + h >= wleft) break;
        const char* line = s_rows[t / 32][h];
        char* o = static_cast<char*>(p.out) + ((row1 + kRowStep * i + h) * p.ld_o + int64_t(cb) * kTile) * T::kBytes;
        if constexpr (T::kBytes == 4) {
#pragma unroll
          for (int c = 0; c < kTile; c += 32)
            if (c + lane < width) reinterpret_cast<uint32_t*>(o)[c + lane] = reinterpret_cast<const uint32_t*>(line)[c + lane];
        } else {
          const int head = int(reinterpret_cast<uintptr_t>(o) >> 1) & 1;
          const uint16_t* l = reinterpret_cast<const uint16_t*>(line) + head;
          uint32_t* words = reinterpret_cast<uint32_t*>(o + 2 * head);
          const int n2 = (width - head) / 2;
#pragma unroll
          for (int c = 0; c < kTile / 2; c += 32)
            if (c + lane < n2) words[c + lane] = l[2 * (c + lane)] | uint32_t(l[2 * (c + lane) + 1]) << 16;
          if (lane == 0 && head) *reinterpret_cast<uint16_t*>(o) = *reinterpret_cast<const uint16_t*>(line);
          if (lane == 1 && ((width - head) & 1)) reinterpret_cast<uint16_t*>(o)[width - 1] = reinterpret_cast<const uint16_t*>(line)[width - 1];
        }
      }
      __syncwarp();
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (kRowStep * i >= left) break;
    if constexpr (!kCol) {
      const float one = scale_value(byte[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = one;
    }
    store_eight<T>(dst + i * o_step, decode8<T>(q[i], f), n, p.vec_out);
  }
}

int64_t tiles(int64_t rows, int64_t cols) {
  return ((rows + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile);
}

template <class T>
cudaError_t save(const CheckpointSaveParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(tiles(p.rows, p.cols)));
  if (p.q_r != nullptr && p.q_c != nullptr)
    return launch_kernel(k_checkpoint_save<T, true, true>, grid, dim3(kThreads), 0, stream, p);
  if (p.q_r != nullptr)
    return launch_kernel(k_checkpoint_save<T, true, false>, grid, dim3(kThreads), 0, stream, p);
  return launch_kernel(k_checkpoint_save<T, false, true>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_checkpoint_save(const CheckpointSaveParams& p, int dtype, cudaStream_t stream) {
  return dtype == 0 ? save<F32T>(p, stream) : save<BF16T>(p, stream);
}

cudaError_t launch_checkpoint_restore(const CheckpointRestoreParams& p, int dtype, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(tiles(p.rows, p.cols)));
  auto run = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kThreads), 0, stream, p); };
  if (dtype == 0) return p.colwise ? run(k_checkpoint_restore<F32T, true>) : run(k_checkpoint_restore<F32T, false>);
  return p.colwise ? run(k_checkpoint_restore<BF16T, true>) : run(k_checkpoint_restore<BF16T, false>);
}

}  // namespace mxfp8
