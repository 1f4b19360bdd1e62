// Operands whose base or row stride is not a multiple of 16 bytes, which no single TMA map can describe.
//
// Every 16th row of such a matrix does lie at a multiple of 16 bytes from the one before, so 16 maps
// describe it: map s has the rows 16 q + s, from the 16-byte unit that holds their first byte, at
// the stride 16 ld.  A box of 128 stored rows by 128 bytes is fetched as 16 boxes of 8 rows by 160 bytes
// (zeros past the matrix, as always) into a ring of raw boxes, and groups of four warps write
// it into the stage as a single map would have: shifted to its first byte, under the 128-byte swizzle.
// A lane makes one 32-bit word at a time from two neighbours; the eight rows of a step take their
// 16-byte units in turns, so that with 160 bytes per raw row neither reads nor writes ask a bank twice
// (16-byte reads and writes of whole units: 248 instead of 228 us in the case below).
// Box corners are multiples of 64 rows and 64 bytes, so a lane's rows keep their place in a 16-byte
// unit over the whole matrix.  (A box cannot start at a row's first byte instead: its innermost coordinate
// times the element size has to be a multiple of 16 bytes.)  (The first unit may start up to 15 bytes before the matrix: inside
// its allocation, which starts at a multiple of 16.)
//
// What bounds it: the raw boxes' way through shared memory, about as much again as the stages' own
// (1.0 us per 128 values of k of a 256 x 256 tile, 0.3 aligned).  Tried first: a bulk copy per row (128
// per box, about 30 cycles each) and cp.async of the units (an SM keeps too few of them under way; in
// the writing warps, the proxy fence waits for them): 8192 x 5001 x 3001 with one operand off 16 bytes 490 and 264 us,
// with maps 232-235 us; with both off 16 bytes 320.
#pragma once

#include <type_traits>

#include <cuda.h>

#include "gemm_impl.cuh"

namespace mxfp8 {

constexpr int kResidues = 16;
constexpr int kRawRow = 160;
constexpr int kRawPart = 8 * kRawRow;            // rows of one residue
constexpr int kRawBox = kResidues * kRawPart;

// A box: the stored row and byte of its corner, the rows it needs, where it goes.
struct RealignItem {
  int32_t row0, col;
  int32_t rows;    // 128, or fewer for narrow tiles
  bool narrow;     // rows of 64 bytes under the 64-byte swizzle
  int32_t live;    // rows from row0 to the end of the matrix
  uint32_t dst;    // the stage's box in shared memory
  bool second;     // of B
};

// The maps of both operands' residues.
struct Residues {
  CUtensorMap residues[2 * kResidues];
};

// A position in a ring of `size` slots, and how often the ring has been round (its parity).
struct RingAt {
  uint32_t slot, parity;
  __device__ __forceinline__ void on(uint32_t by, uint32_t size) {
    slot += by;
    while (slot >= size) {
      slot -= size;
      parity ^= 1;
    }
  }
};

// What is realigned, in registers: both operands' shapes, and which of them.
struct RealignShape {
  int32_t rows_a, rows_b;  // stored
  bool across_a, across_b, a, b;
  __device__ __forceinline__ explicit RealignShape(const GemmParams& p)
      : rows_a(int32_t(p.a.colwise ? p.k : p.m)), rows_b(int32_t(p.b.colwise ? p.k : p.n)), across_a(p.a.colwise),
        across_b(p.b.colwise), a(!p.a.aligned), b(!p.b.aligned) {}
  // A box of `extent` rows of A or B at (mn, k0).
  __device__ __forceinline__ RealignItem item(bool second, int32_t mn, int32_t k0, int32_t extent, uint32_t dst) const {
    const bool across = second ? across_b : across_a;
    const int32_t row0 = across ? k0 : mn;
    return {row0, across ? mn : k0, across ? 128 : extent, across && extent == 64, (second ? rows_b : rows_a) - row0, dst, second};
  }
  __device__ __forceinline__ uint32_t per_stage() const { return a && b ? 2 : 1; }
};

// The ring: a slot is full when its copies have landed, and empty when the four warps of a group have
// read it.
struct RealignRing {
  char* boxes;
  uint32_t full, empty;  // barriers, one per slot
  int depth;
  __device__ __forceinline__ char* box(uint32_t slot) const { return boxes + slot * kRawBox; }
  __device__ __forceinline__ void init() const {
    for (int i = 0; i < depth; ++i) {
      tc::mbar_init(full + 8 * i, 1);
      tc::mbar_init(empty + 8 * i, 4);
    }
  }
};

// Has the maps that a launch uses fetched at once: one after the other, on first use, they would cost
// a latency of memory each.
__device__ __forceinline__ void prefetch_residues(const CUtensorMap* maps, bool of_a, bool of_b) {
  const int lane = threadIdx.x & 31;
  if (lane < kResidues ? of_a : of_b) tc::prefetch_map(maps + lane);
}

// The fetching thread: every box, in order.  maps: those of A's residues, then B's.
template <class Walk>
__device__ __forceinline__ void realign_fetch(const RealignRing& ring, const CUtensorMap* maps, Walk at,
                                              volatile uint32_t* gave_up) {
  RingAt raw{0, 0};
  uint32_t issued = 0;
  for (; at.valid(); at.next()) {
    const RealignItem it = at.item();
    if (!tc::mbar_wait(ring.empty + 8 * raw.slot, raw.parity ^ 1, gave_up)) break;
    const uint32_t bar = ring.full + 8 * raw.slot, dst = tc::smem_addr(ring.box(raw.slot));
    const CUtensorMap* m = maps + (it.second ? kResidues : 0);
    tc::mbar_expect(bar, kRawBox);
#pragma unroll
    for (int s = 0; s < kResidues; ++s) tc::tma_load_2d(dst + s * kRawPart, m + s, it.col, it.row0 >> 4, bar);
    ++issued;
    raw.on(1, ring.depth);
  }
  if (*gave_up != 0) tc::settle_copies(ring.full, uint32_t(ring.depth), issued);
}

// Lane l of warp w (0 .. 3) of a group writes word l % 4 of the units of rows 16 (l / 4) + s, s = 4 w .. 4 w + 3.
// place: for each s the byte in the raw box, and shift << 16, of that word of unit 0.
template <bool kPlain>
__device__ __forceinline__ void realign_box(uint4 place, uint32_t from, uint32_t dst, int warp, int rows, int live, bool narrow) {
  const int lane = threadIdx.x & 31, q = lane >> 2;
  if (16 * q >= rows) return;
  const uint32_t p[4] = {place.x, place.y, place.z, place.w};
  const uint32_t to = dst + 16 * q * 128 + 4 * (lane & 3);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t src = from + (p[g] & 0xffffu), sh = p[g] >> 16, s = 4 * warp + g;
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = 16 * ((i + q) & 7);
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(lo[i]) : "r"(src + u));
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(hi[i]) : "r"(src + u + 4));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = __funnelshift_r(lo[i], hi[i], sh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = (i + q) & 7, r = 16 * q + s;
      if constexpr (kPlain) {
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + s * 128 + ((u ^ (s & 7)) << 4)), "r"(lo[i]) : "memory");
      } else {
        const uint32_t at = narrow ? dst + r * 64 + ((u ^ (r >> 1 & 3)) << 4) + 4 * (lane & 3) : to + s * 128 + ((u ^ (s & 7)) << 4);
        if (!narrow || u < 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(int(r) < live ? lo[i] : 0u) : "memory");
      }
    }
  }
}
// Boxes with rows of 64 bytes, and those whose matrix has fewer than 16 rows left (residues without rows
// have no map of zeros).  Out of line: inside the loop these cases cost a fifth of the others' rate.
static __device__ __noinline__ void realign_rare_box(uint4 place, uint32_t from, uint32_t dst, int warp, int rows, int live, bool narrow) {
  realign_box<false>(place, from, dst, warp, rows, live, narrow);
}

// One of the four warps of a group.
struct Realigner {
  uint4 a, b;  // places of A and B
  int warp;

  __device__ __forceinline__ uint4 places(const GemmOperand& o) const {
    const int lane = threadIdx.x & 31;
    const uint32_t base = uint32_t(reinterpret_cast<uintptr_t>(o.codes)), ld = uint32_t(o.ld);
    uint32_t p[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t s = 4 * warp + g, off = (base + s * ld) & 15;
      p[g] = (s * kRawPart + (lane >> 2) * kRawRow + (off & ~3u) + 4 * (lane & 3)) | ((off & 3) * 8) << 16;
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
  }

  __device__ __forceinline__ void write(const RealignItem& it, const char* box) const {
    const uint32_t from = tc::smem_addr(box);
    const uint4 place = make_uint4(it.second ? b.x : a.x, it.second ? b.y : a.y, it.second ? b.z : a.z, it.second ? b.w : a.w);
    if (!it.narrow && it.live >= kResidues) realign_box<true>(place, from, it.dst, warp, it.rows, 0, false);
    else realign_rare_box(place, from, it.dst, warp, it.rows, it.live, it.narrow);
  }
};

// A writing warp: its residues of the boxes of every `groups`-th stage, from stage `group` on.  Walk:
// valid(), item(), first() / last() of its stage, next().  `box_free` waits until the stage of the
// walk's item may be written; `box_full` announces it.
template <class Walk, class Free, class Full>
__device__ __forceinline__ void realign_write(const RealignRing& ring, const Realigner& ra, Walk at, uint32_t group,
                                              uint32_t groups, volatile uint32_t* gave_up, Free box_free, Full box_full) {
  const uint32_t per = at.shape.per_stage();
  RingAt raw{0, 0};
  raw.on(per * group, ring.depth);
  for (; at.valid(); at.next()) {
    const RealignItem it = at.item();
    bool good = !at.first() || box_free(at);
    good = good && tc::mbar_wait(ring.full + 8 * raw.slot, raw.parity, gave_up);
    if (!__all_sync(kFullMask, good)) break;
    ra.write(it, ring.box(raw.slot));
    const bool last = at.last();
    if (last) tc::fence_async_proxy();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(ring.empty + 8 * raw.slot);
    if (last) box_full(at);
    raw.on(last ? per * groups - (per - 1) : 1, ring.depth);
  }
}

}  // namespace mxfp8
