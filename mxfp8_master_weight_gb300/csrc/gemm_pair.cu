// Block-scaled product for large outputs: tiles of 256 x 256 by pairs of CTAs.
//
// The two SMs of a pair work on one tile with one stream of matrix instructions (cta_group::2,
// 256 x 256 x 32): each holds 128 rows of A, 128 rows of B and 128 rows of the sums, so a
// stage of 128 values of k costs an SM 33.5 KB of copies for 512 cycles of matrix work.  A
// single-SM tile of 128 x 256 would fetch 50 KB for the same 512 cycles.
//
// Roles in a CTA: warp 0 fetches (one thread, TMA, five stages, or seven where every tile is a half),
// warp 1 of the leading CTA issues scale copies and matrix instructions for both, eight warps
// write the sums out.  With an operand to realign four warps write, and nine others fetch and
// realign.
//
// When the last round of tiles would occupy at most half of the pairs, its tiles are cut into
// halves of 256 x 128, one per pair: 4096^3 has 256 tiles for 76 pairs, 3.5 rounds instead of 4
// (1.6 us less); outputs of few tiles are halves throughout (256 x 4096 x 4096 13.9 -> 10.4 us).
//
// Tensor memory has 512 columns; two buffers of 256 sums and the scales do not fit.  The buffers
// therefore share 32 columns: buffer 0 is columns 0..255, buffer 1 columns 224..479, two sets of
// scales 480..511.  The writers drain the shared columns of a tile first; then the next
// tile's instructions start in the other buffer while they write the rest.
//
// What bounds it: the matrix instructions and what feeds them, and over more than some milliseconds the board's
// power, which sets the clock.  8192^3 takes 302 us in a burst (3.64 PFLOP/s, 0.96 of twice the measured BF16
// rate) and 337 in a loop of half a second (1470 MHz).  4096^3 takes 43 us in a burst on unchanged operands, 46.6
// in a loop (2070 MHz), 48.8 with three sets of operands in turn (1880 MHz), 50-51 with new inputs in every
// pass; the first and last stages of a launch, about 4 us, and the share of the last round that stays empty are
// what it loses of 36.  2048 x 8192 x 8192 with both operands across k and F32 output: 94 us in a loop, 100 with
// the addend (1665 MHz both), 102-105 with the addend and new inputs.
#include <type_traits>

#include <cuda.h>

#include "gemm_impl.cuh"
#include "gemm_maps.h"
#include "gemm_realign.cuh"

namespace mxfp8 {
namespace {

constexpr int kMaxStages = 7;
constexpr int kRawDepth = 3;  // raw boxes
constexpr int kScaleBytes = 3 * kScaleTile;  // of A, and of both 128-row halves of B
// Writers: eight warps; four where eight others realign an operand.
template <bool kRealign>
constexpr int kWriters = kRealign ? 4 : 8;
constexpr int kRealignGroups = 2;  // of four warps, which take the stages in turn
constexpr int kRealignWarps = 4 * kRealignGroups + 1;  // and one that fetches
constexpr int kWriterBytes = 4096;  // a writer's 32 rows of 128 bytes
constexpr int kSmem = 226 * 1024;
// What is left for stages: a stage is A's box, B's box (half a box where every tile is a half) and
// the scales, each kind in an array of its own, which keeps the boxes on 1024-byte boundaries.
template <bool kRealign>
constexpr int kStageRoom = kSmem - 1024 - kWriters<kRealign> * kWriterBytes - (kRealign ? kRawDepth * kRawBox : 0) - 384;
template <bool kRealign>
constexpr int kThreads = 64 + 32 * (kWriters<kRealign> + (kRealign ? kRealignWarps : 0));
constexpr int kSecondBuffer = 224;  // first column of the second buffer of sums
constexpr int kScaleCol = 480;

struct PairParams {
  GemmParams g;
  CUtensorMap a, b, b_half, sa, sb;
  unsigned* given_up;
  int64_t whole, units;  // whole tiles first, then halves
  int32_t stages, b_bytes;
};

struct PairParamsRealign : PairParams, Residues {};

struct Tile {
  int64_t tm, col;  // 256-row block; first column
  bool half;
};
__device__ __forceinline__ Tile tile_of(const PairParams& q, int64_t unit, int64_t tiles_m, int64_t tiles_n) {
  Tile t;
  int64_t tn;
  t.half = unit >= q.whole;
  tile_at(t.half ? q.whole + (unit - q.whole) / 2 : unit, tiles_m, tiles_n, t.tm, tn);
  t.col = tn * 256 + (t.half ? 128 * ((unit - q.whole) & 1) : 0);
  return t;
}

// The boxes that are realigned: all of them for the fetching thread (`stride` 1), for a group of writing
// warps those of every kRealignGroups-th stage.
struct PairWalk {
  const PairParams& q;
  RealignShape shape;
  int64_t unit, step, tiles_m, tiles_n;
  int32_t nk, kb, a_mn, b_mn;  // a_mn, b_mn: first rows of A and B of this CTA
  uint32_t rank, a_box, b_box;
  RingAt stage;
  int32_t stages, stride;
  bool second, half;
  __device__ __forceinline__ bool valid() const { return unit < q.units && nk > 0; }
  __device__ __forceinline__ bool first() const { return second != shape.a; }
  __device__ __forceinline__ bool last() const { return second == shape.b; }
  __device__ __forceinline__ RealignItem item() const {
    return shape.item(second, second ? b_mn : a_mn, kb * kBlockK, second && half ? 64 : 128,
                      second ? b_box + stage.slot * q.b_bytes : a_box + stage.slot * kBoxBytes);
  }
  __device__ __forceinline__ void tile() {
    if (unit >= q.units) return;
    const Tile t = tile_of(q, unit, tiles_m, tiles_n);
    half = t.half;
    a_mn = int32_t(t.tm * 256 + rank * 128);
    b_mn = int32_t(t.col + rank * (half ? 64 : 128));
  }
  __device__ __forceinline__ void skip(int by) {  // `by` stages on
    stage.on(by, stages);
    kb += by;
    if (kb < nk) return;
    for (; kb >= nk && unit < q.units; kb -= nk) unit += step;
    tile();
  }
  __device__ __forceinline__ void next() {
    if (!last()) {
      second = true;
      return;
    }
    second = !shape.a;
    skip(stride);
  }
};

template <bool kRealign>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<kRealign>, 1)
    k_gemm_pair(const __grid_constant__ std::conditional_t<kRealign, PairParamsRealign, PairParams> q) {
  extern __shared__ char raw[];
  const GemmParams& p = q.g;
  // the same offset in both CTAs: their dynamic shared memory starts alike
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  char* b_boxes = smem + q.stages * kBoxBytes;
  char* scales = b_boxes + q.stages * q.b_bytes;
  char* writers = scales + q.stages * kScaleBytes;
  char* raw_boxes = writers + kWriters<kRealign> * kWriterBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(raw_boxes + (kRealign ? kRawDepth * kRawBox : 0));
  uint64_t* raw_bars = bars + 3 * kMaxStages + 3;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw_bars + (kRealign ? 2 * kRawDepth : 0));
  const RealignRing ring{raw_boxes, tc::smem_addr(raw_bars), tc::smem_addr(raw_bars + kRawDepth), kRawDepth};
  volatile uint32_t* gave_up = tmem_slot + 1;
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kMaxStages, sums_full = empty + 8 * kMaxStages,
                 sums_free = sums_full + 16, ready = sums_free + 8;
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = tc::cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.stages; ++s) {
      // the expected copies; realigned, also four warps of the leading CTA and the other one's word
      tc::mbar_init(full + 8 * s, 1 + (kRealign ? 4 + 1 : 0));
      if constexpr (kRealign) tc::mbar_init(ready + 8 * s, 4);
      tc::mbar_init(empty + 8 * s, 1);
    }
    if constexpr (kRealign) ring.init();
    tc::mbar_init(sums_full, 1);
    tc::mbar_init(sums_full + 8, 1);
    tc::mbar_init(sums_free, 2 * kWriters<kRealign>);
    *gave_up = 0;
    tc::mbar_init_fence();
    if (p.k > 0) {
      if (!kRealign || p.a.aligned) tc::prefetch_map(&q.a);
      if (!kRealign || p.b.aligned) {
        tc::prefetch_map(&q.b);
        tc::prefetch_map(&q.b_half);
      }
      tc::prefetch_map(&q.sa);
      tc::prefetch_map(&q.sb);
    }
  }
  if (warp == 1) tc::tmem_alloc<2>(tc::smem_addr(tmem_slot), 512);
  if constexpr (kRealign) {
    if (warp == 2) prefetch_residues(q.residues, !p.a.aligned, !p.b.aligned);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  tc::grid_wait_then_release();
  const uint32_t tmem = *tmem_slot;
  const int64_t tiles_m = (p.m + 255) / 256, tiles_n = (p.n + 255) / 256;
  const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int64_t nk = (p.k + kBlockK - 1) / kBlockK;

  if (warp == 0) {
    if (tc::elect_one()) {
      const uint32_t lead_full = tc::in_cta(full, 0);
      int s = 0;
      uint32_t phase = 1;
      uint32_t issued = 0;
      for (int64_t unit = first; unit < q.units && *gave_up == 0; unit += step) {
        const Tile t = tile_of(q, unit, tiles_m, tiles_n);
        const int am = int(t.tm * 256 + rank * 128), bn = int(t.col + rank * (t.half ? 64 : 128));
        const bool tma_a = !kRealign || p.a.aligned, tma_b = !kRealign || p.b.aligned;
        const uint32_t bytes = (tma_a ? kBoxBytes : 0) + (tma_b ? (t.half ? kBoxBytes / 2 : kBoxBytes) : 0) + kScaleBytes;
        for (int64_t kb = 0; kb < nk; ++kb) {
          if (!tc::mbar_wait(empty + 8 * s, phase, gave_up)) break;
          const uint32_t at_a = tc::smem_addr(smem + s * kBoxBytes), at_b = tc::smem_addr(b_boxes + s * q.b_bytes),
                         at_s = tc::smem_addr(scales + s * kScaleBytes), bar = lead_full + 8 * s;
          const int k0 = int(kb * kBlockK);
          if (rank == 0) tc::mbar_expect(full + 8 * s, 2 * bytes);
          if (tma_a) tc::tma_load_2d_pair(at_a, &q.a, p.a.colwise ? am : k0, p.a.colwise ? k0 : am, bar);
          if (tma_b) tc::tma_load_2d_pair(at_b, t.half ? &q.b_half : &q.b, p.b.colwise ? bn : k0, p.b.colwise ? k0 : bn, bar);
          tc::tma_load_3d_pair(at_s, &q.sa, 0, int(scale_tile_of(kb, p.a.block)), int(2 * t.tm + rank), bar);
          tc::tma_load_3d_pair(at_s + kScaleTile, &q.sb, 0, int(scale_tile_of(kb, p.b.block)), int(t.col >> 7), bar);
          ++issued;
          if (++s == q.stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (*gave_up != 0 && rank == 0) tc::settle_copies(full, uint32_t(q.stages), issued);
    }
  } else if (warp == 1) {
    if (rank == 0 && tc::elect_one()) {
      const uint32_t astep = p.a.colwise ? 4096 : 32;
      int s = 0;
      uint32_t phase = 0, nth = 0, set = 0;
      bool good = true;
      for (int64_t unit = first; unit < q.units && good; unit += step, ++nth) {
        if (nth > 0) good = tc::mbar_wait(sums_free, (nth - 1) & 1, gave_up);
        tc::fence_after_sync();
        const uint32_t d = tmem + (nth & 1 ? kSecondBuffer : 0);
        const bool half = unit >= q.whole, narrow = half && p.b.colwise;  // rows of 64 bytes
        const uint32_t idesc = tc::instr_desc(256, half ? 128 : 256, p.a.colwise, p.b.colwise);
        const uint32_t bstep = narrow ? 2048 : (p.b.colwise ? 4096 : 32);
        for (int64_t kb = 0; kb < nk && good; ++kb) {
          good = tc::mbar_wait(full + 8 * s, phase, gave_up);
          if (!good) break;
          tc::fence_after_sync();
          const uint32_t at_a = tc::smem_addr(smem + s * kBoxBytes), at_b = tc::smem_addr(b_boxes + s * q.b_bytes),
                         at_s = tc::smem_addr(scales + s * kScaleBytes);
          const uint32_t sa = tmem + kScaleCol + 16 * set, sb = sa + 4;
          set ^= 1;
          tc::copy_scales<2>(sa, tc::scale_desc(at_s));
          tc::copy_scales<2>(sb, tc::scale_desc(at_s + kScaleTile));
          tc::copy_scales<2>(sb + 4, tc::scale_desc(at_s + 2 * kScaleTile));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_scaled<2>(d, tc::operand_desc(at_a + j * astep),
                              narrow ? tc::operand_desc64(at_b + j * bstep) : tc::operand_desc(at_b + j * bstep),
                              tc::with_scale_ids(idesc, scale_id_of(kb, j, p.a.block), scale_id_of(kb, j, p.b.block)),
                              sa, sb, kb > 0 || j > 0);
          tc::commit_pair(empty + 8 * s, 3);
          if (++s == q.stages) {
            s = 0;
            phase ^= 1;
          }
        }
        tc::commit_pair(sums_full + 8 * (nth & 1), 3);
      }
    }
    if (kRealign && rank == 1 && tc::elect_one()) {
      // The other CTA's realigned stages, passed on to the leading one: an arrival there is a release
      // to the cluster, which holds a warp up for 800 cycles.
      RingAt at{0, 0};
      bool good = true;
      for (int64_t unit = first; unit < q.units && good; unit += step) {
        for (int64_t kb = 0; kb < nk && good; ++kb) {
          good = tc::mbar_wait(ready + 8 * at.slot, at.parity, gave_up);
          if (good) tc::mbar_arrive_cluster(full + 8 * at.slot, 0);
          at.on(1, q.stages);
        }
      }
    }
  } else if (kRealign && warp >= 2 + kWriters<kRealign>) {
    if constexpr (kRealign) {
      const int w = warp - 2 - kWriters<kRealign>;
      const bool fetches = w >= 4 * kRealignGroups;
      const RealignShape shape(p);
      PairWalk walk{q, shape, first, step, tiles_m, tiles_n, int32_t(nk), 0, 0, 0, rank, tc::smem_addr(smem),
                    tc::smem_addr(b_boxes), {0, 0}, q.stages, fetches ? 1 : kRealignGroups, !shape.a, false};
      walk.tile();
      if (fetches) {
        if (tc::elect_one()) realign_fetch(ring, q.residues, walk, gave_up);
      } else {
        Realigner ra = {};
        ra.warp = w & 3;
        if (shape.a) ra.a = ra.places(p.a);
        if (shape.b) ra.b = ra.places(p.b);
        if (nk > 0) walk.skip(w >> 2);
        const uint32_t announce = rank == 0 ? full : ready;
        realign_write(
            ring, ra, walk, w >> 2, kRealignGroups, gave_up,
            [&](const PairWalk& at) { return tc::mbar_wait(empty + 8 * at.stage.slot, at.stage.parity ^ 1, gave_up); },
            [&](const PairWalk& at) {
              if ((threadIdx.x & 31) == 0) tc::mbar_arrive(announce + 8 * at.stage.slot);
            });
      }
    }
  } else {
    const int side = (warp - 2) >> 2;  // the first or second half of the columns
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    uint32_t nth = 0;
    for (int64_t unit = first; unit < q.units; unit += step, ++nth) {
      const Tile t = tile_of(q, unit, tiles_m, tiles_n);
      const int cols = (t.half ? 512 : 1024) / kWriters<kRealign>;  // this warp's
      const uint32_t buffer = nth & 1;
      // no two tiles' sums are ready at once that this warp has not drained: the next tile's
      // instructions wait for sums_free
      if (!tc::mbar_wait(sums_full + 8 * buffer, (nth >> 1) & 1, gave_up)) break;
      tc::fence_after_sync();
      const int64_t row0 = t.tm * 256 + 128 * rank + 32 * (warp & 3), col0 = t.col + cols * side;
      const uint32_t d = tmem + lanes + (buffer ? kSecondBuffer : 0) + cols * side;
      // the shared columns, the last of buffer 0 and the first of buffer 1, come first; the arrival
      // after the first chunk also says that the warp is done with the tile before
      const int width = p.out_f32 ? 32 : 64, chunks = cols / width;
#pragma unroll 1
      for (int i = 0; i < chunks; ++i) {
        const int c = width * (buffer ? i : chunks - 1 - i);
        int left = i == 0 ? width / 32 : 0;  // loads until the first chunk is drained
        write_rows(p, writers + (warp - 2) * kWriterBytes, row0, col0 + c, [&](int e, float(&v)[32]) {
          if (nk > 0) {
            tc::tmem_load32(d + c + e, v);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0.0f;
          }
          if (left != 0 && --left == 0) {
            tc::fence_before_sync();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) tc::mbar_arrive_cluster_relaxed(sums_free, 0);
          }
        });
      }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  if (threadIdx.x == 0 && *gave_up != 0) tc::report_given_up(q.given_up);
  if (warp == 1) tc::tmem_free<2>(tmem, 512);
}

}  // namespace

cudaError_t launch_gemm_pair(const GemmParams& g, unsigned* given_up, const DeviceInfo& dev, cudaStream_t stream,
                             const char** what) {
  PairParamsRealign q{};
  q.g = g;
  q.given_up = given_up;
  const bool realign = g.k > 0 && !(g.a.aligned && g.b.aligned);
  cudaError_t e = cudaSuccess;
  if (g.k > 0) {
    if (g.a.aligned) e = operand_map(g.a, g.k, 128, &q.a, what);
    if (e == cudaSuccess && g.b.aligned) e = operand_map(g.b, g.k, 128, &q.b, what);
    if (e == cudaSuccess && g.b.aligned) e = half_operand_map(g.b, g.k, &q.b_half, what);
    if (e == cudaSuccess) e = scale_map(g.a, g.k, 1, &q.sa, what);
    if (e == cudaSuccess) e = scale_map(g.b, g.k, 2, &q.sb, what);
  }
  if (e == cudaSuccess && realign && !g.a.aligned) e = residue_maps(g.a, g.k, q.residues, what);
  if (e == cudaSuccess && realign && !g.b.aligned) e = residue_maps(g.b, g.k, q.residues + kResidues, what);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((g.m + 255) / 256) * ((g.n + 255) / 256);
  const int64_t pairs = dev.sms / 2, last = tiles % pairs;
  q.whole = last != 0 && 2 * last <= pairs ? tiles - last : tiles;
  q.units = q.whole + 2 * (tiles - q.whole);
  q.b_bytes = q.whole == 0 ? kBoxBytes / 2 : kBoxBytes;
  const int fit = (realign ? kStageRoom<true> : kStageRoom<false>) / (kBoxBytes + q.b_bytes + kScaleBytes);
  q.stages = fit < kMaxStages ? fit : kMaxStages;
  const unsigned grid = 2 * unsigned(q.units < pairs ? q.units : pairs);
  auto run = [&](auto kernel, int threads, const auto& params) {
    const cudaError_t a = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return a != cudaSuccess ? a : launch_kernel(kernel, dim3(grid), dim3(threads), kSmem, stream, params);
  };
  return realign ? run(k_gemm_pair<true>, kThreads<true>, q)
                 : run(k_gemm_pair<false>, kThreads<false>, static_cast<const PairParams&>(q));
}

}  // namespace mxfp8
