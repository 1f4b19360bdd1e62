// Pieces that the norms of a row share: values of a row in eights, sums over a row's threads, a thread's columns, and
// rings of rows in shared memory.
#pragma once

#include "common.cuh"
#include "linear.h"
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

// ------------------------------------------------------------------------------ a thread's columns
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

}  // namespace
}  // namespace mxfp8
