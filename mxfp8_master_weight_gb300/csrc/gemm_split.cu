// Block-scaled product for outputs of few tiles: tiles of 128 x NT by single CTAs, the contraction
// split over the CTAs of a cluster.
//
// A few tokens against a weight read the whole weight for little arithmetic: the product is bound
// by HBM, and what counts is that every SM has copies in flight from the start.  The weight's
// rows take the 128 lanes of the tile (the operands change places when the output has few rows),
// the tokens its NT = 16 .. 128 columns, and 1 to 8 CTAs share a tile, each with its part
// of k.  Their partial sums stay in shared memory; after a cluster barrier each CTA adds its share of
// the columns over the cluster in rank order and writes it.  No workspace, no atomics: the
// result depends on the shape alone.
#include <type_traits>

#include <cuda.h>

#include "gemm_impl.cuh"
#include "gemm_maps.h"
#include "gemm_realign.cuh"

namespace mxfp8 {
namespace {

constexpr int kThreads = 192;  // warp 0 fetches, warp 1 issues, four warps write
constexpr int kMaxSplit = 8;
constexpr int kMaxStages = 8;
constexpr int kRealignWarps = 5;  // four write, one fetches
constexpr int kRawDepth = 2;  // raw boxes

// Stages of a CTA: two CTAs share an SM.  An operand that lies across k has 128 bytes of n per
// row of its box however small NT is.
template <int NT>
constexpr int columns_bytes(bool across) { return across ? kBoxBytes : NT * 128; }
constexpr int kSmemBudget = 112 * 1024;

struct SplitParams {
  GemmParams g;      // A: the 128-row side, B: the NT-column side
  CUtensorMap a, b, sa, sb;
  unsigned* given_up;
  int32_t swapped;   // out[column][row]: the caller's A is B here
  int32_t stages, b_bytes, split;
};

struct SplitParamsRealign : SplitParams, Residues {};

// Writes N neighbouring columns, j .. j + N - 1, of row i of the tile's matrix.
template <int N>
__device__ __forceinline__ void store_columns(const SplitParams& q, int64_t i, int64_t j, const float (&v)[N]) {
  const GemmParams& p = q.g;
  if (i >= p.m) return;
  if (q.swapped) {  // neighbouring lanes hold neighbouring elements of the output row
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (j + e < p.n) store_one(p, j + e, i, v[e] + load_addend(p, j + e, i));
    return;
  }
  if (N % 8 == 0 && p.vec_out && p.addend == nullptr && j + N <= p.n) {
#pragma unroll
    for (int e = 0; e < N; e += 8) {
      if (p.out_f32) {
        float* o = static_cast<float*>(p.out) + i * p.ld_o + j + e;
        *reinterpret_cast<float4*>(o) = make_float4(v[e], v[e + 1 < N ? e + 1 : 0], v[e + 2 < N ? e + 2 : 0], v[e + 3 < N ? e + 3 : 0]);
        *reinterpret_cast<float4*>(o + 4) = make_float4(v[e + 4 < N ? e + 4 : 0], v[e + 5 < N ? e + 5 : 0], v[e + 6 < N ? e + 6 : 0], v[e + 7 < N ? e + 7 : 0]);
      } else {
        uint16_t* o = static_cast<uint16_t*>(p.out) + i * p.ld_o + j + e;
        *reinterpret_cast<uint4*>(o) = make_uint4(bf16x2_rn(v[e], v[e + 1 < N ? e + 1 : 0]), bf16x2_rn(v[e + 2 < N ? e + 2 : 0], v[e + 3 < N ? e + 3 : 0]),
                                                  bf16x2_rn(v[e + 4 < N ? e + 4 : 0], v[e + 5 < N ? e + 5 : 0]), bf16x2_rn(v[e + 6 < N ? e + 6 : 0], v[e + 7 < N ? e + 7 : 0]));
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (j + e < p.n) store_one(p, i, j + e, v[e] + load_addend(p, i, j + e));
}

// Adds N columns from `c` of the tile over the cluster, in rank order, and writes them.
template <int N>
__device__ __forceinline__ void add_and_store(const SplitParams& q, const float* part, int c, int row, int64_t i, int64_t j) {
  float v[N];
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = 0.0f;
  const uint32_t at = tc::smem_addr(part + c * 128 + row);
#pragma unroll
  for (int r = 0; r < kMaxSplit; ++r) {
    if (r < q.split) {
      const uint32_t from = tc::in_cta(at, r);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(from + 512 * e) : "memory");
        v[e] += x;
      }
    }
  }
  store_columns<N>(q, i, j, v);
}

// The boxes that are realigned, in the order of the stages.
struct SplitWalk {
  RealignShape shape;
  int32_t am, bn, kb, k_hi;
  uint32_t a_box, b_box;
  int32_t b_rows, b_bytes, stages;
  RingAt stage;
  bool second;
  __device__ __forceinline__ bool valid() const { return kb < k_hi; }
  __device__ __forceinline__ bool first() const { return second != shape.a; }
  __device__ __forceinline__ bool last() const { return second == shape.b; }
  __device__ __forceinline__ RealignItem item() const {
    return shape.item(second, second ? bn : am, kb * kBlockK, second && !shape.across_b ? b_rows : 128,
                      second ? b_box + stage.slot * b_bytes : a_box + stage.slot * kBoxBytes);
  }
  __device__ __forceinline__ void next() {
    if (!last()) {
      second = true;
      return;
    }
    second = !shape.a;
    ++kb;
    stage.on(1, stages);
  }
};

template <int NT, bool kRealign>
__global__ void __launch_bounds__(kThreads + (kRealign ? 32 * kRealignWarps : 0), 2) k_gemm_split(
    const __grid_constant__ std::conditional_t<kRealign, SplitParamsRealign, SplitParams> q) {
  extern __shared__ char raw[];
  const GemmParams& p = q.g;
  constexpr uint32_t kTmemCols = NT <= 32 ? 64 : (NT <= 64 ? 128 : 256);
  constexpr uint32_t kScaleCol = NT;  // two sets of 4 + 4 columns
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  // boxes of A, boxes of B, scales: an array of each keeps the boxes on 1024-byte boundaries
  char* b_boxes = smem + q.stages * kBoxBytes;
  char* scales = b_boxes + q.stages * q.b_bytes;
  char* raw_boxes = scales + q.stages * 2 * kScaleTile;
  __shared__ uint64_t bars[2 * kMaxStages + 1 + (kRealign ? 2 * kRawDepth : 0)];
  __shared__ uint32_t tmem_slot, s_gave_up;
  volatile uint32_t* gave_up = &s_gave_up;
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kMaxStages, done = empty + 8 * kMaxStages;
  const RealignRing ring{raw_boxes, done + 8, done + 8 + 8 * kRawDepth, kRawDepth};
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = q.split > 1 ? tc::cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.stages; ++s) {
      tc::mbar_init(full + 8 * s, 1 + (kRealign ? 4 : 0));
      tc::mbar_init(empty + 8 * s, 1);
    }
    if constexpr (kRealign) ring.init();
    tc::mbar_init(done, 1);
    s_gave_up = 0;
    tc::mbar_init_fence();
    if (!kRealign || p.a.aligned) tc::prefetch_map(&q.a);
    if (!kRealign || p.b.aligned) tc::prefetch_map(&q.b);
    tc::prefetch_map(&q.sa);
    tc::prefetch_map(&q.sb);
  }
  if (warp == 1) tc::tmem_alloc<1>(tc::smem_addr(&tmem_slot), kTmemCols);
  if constexpr (kRealign) {
    if (warp == 2) prefetch_residues(q.residues, !p.a.aligned, !p.b.aligned);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  tc::grid_wait_then_release();
  const uint32_t tmem = tmem_slot;
  int64_t tm, tn;
  tile_at(blockIdx.x / q.split, (p.m + 127) / 128, (p.n + NT - 1) / NT, tm, tn);
  const int64_t nk = (p.k + kBlockK - 1) / kBlockK;
  const int64_t k_lo = nk * rank / q.split, k_hi = nk * (rank + 1) / q.split;

  if (warp == 0) {
    if (tc::elect_one()) {
      int s = 0;
      uint32_t phase = 1;
      int64_t issued = 0;
      const int am = int(tm * 128), bn = int(tn * NT);
      const bool tma_a = !kRealign || p.a.aligned, tma_b = !kRealign || p.b.aligned;
      for (int64_t kb = k_lo; kb < k_hi; ++kb) {
        if (!tc::mbar_wait(empty + 8 * s, phase, gave_up)) break;
        const uint32_t at_s = tc::smem_addr(scales + s * 2 * kScaleTile), bar = full + 8 * s;
        const int k0 = int(kb * kBlockK);
        tc::mbar_expect(bar, uint32_t((tma_a ? kBoxBytes : 0) + (tma_b ? q.b_bytes : 0) + 2 * kScaleTile));
        if (tma_a) tc::tma_load_2d(tc::smem_addr(smem + s * kBoxBytes), &q.a, p.a.colwise ? am : k0, p.a.colwise ? k0 : am, bar);
        if (tma_b) tc::tma_load_2d(tc::smem_addr(b_boxes + s * q.b_bytes), &q.b, p.b.colwise ? bn : k0, p.b.colwise ? k0 : bn, bar);
        tc::tma_load_3d(at_s, &q.sa, 0, int(scale_tile_of(kb, p.a.block)), int(tm), bar);
        tc::tma_load_3d(at_s + kScaleTile, &q.sb, 0, int(scale_tile_of(kb, p.b.block)), bn >> 7, bar);
        ++issued;
        if (++s == q.stages) {
          s = 0;
          phase ^= 1;
        }
      }
      if (*gave_up != 0) {  // let the copies in flight land (or a bounded time pass) before leaving
        const long long t0 = clock64();
        for (int i = 0; i < q.stages && i < issued; ++i) {
          const int64_t c = issued - 1 - i;
          while (!tc::mbar_try(full + 8 * int(c % q.stages), uint32_t(c / q.stages) & 1) && clock64() - t0 < tc::kWaitCycles) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (tc::elect_one()) {
      const uint32_t idesc = tc::instr_desc(128, NT, p.a.colwise, p.b.colwise);
      const uint32_t astep = p.a.colwise ? 4096 : 32, bstep = p.b.colwise ? 4096 : 32;
      int s = 0;
      uint32_t phase = 0;
      for (int64_t kb = k_lo; kb < k_hi; ++kb) {
        if (!tc::mbar_wait(full + 8 * s, phase, gave_up)) break;
        tc::fence_after_sync();
        const uint32_t at_a = tc::smem_addr(smem + s * kBoxBytes), at_b = tc::smem_addr(b_boxes + s * q.b_bytes),
                       at_s = tc::smem_addr(scales + s * 2 * kScaleTile);
        const uint32_t sa = tmem + kScaleCol + 8 * uint32_t(kb & 1), sb = sa + 4;
        tc::copy_scales<1>(sa, tc::scale_desc(at_s));
        tc::copy_scales<1>(sb, tc::scale_desc(at_s + kScaleTile));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc::mma_scaled<1>(tmem, tc::operand_desc(at_a + j * astep), tc::operand_desc(at_b + j * bstep),
                            tc::with_scale_ids(idesc, scale_id_of(kb, j, p.a.block), scale_id_of(kb, j, p.b.block)), sa,
                            sb, kb > k_lo || j > 0);
        tc::commit(empty + 8 * s);
        if (++s == q.stages) {
          s = 0;
          phase ^= 1;
        }
      }
      tc::commit(done);
    }
  } else if (kRealign && warp >= 6) {
    if constexpr (kRealign) {
      const RealignShape shape(p);
      const SplitWalk walk{shape, int32_t(tm * 128), int32_t(tn * NT), int32_t(k_lo), int32_t(k_hi), tc::smem_addr(smem),
                           tc::smem_addr(b_boxes), p.b.colwise ? 128 : NT, q.b_bytes, q.stages, {0, 0}, !shape.a};
      if (warp >= 10) {
        if (tc::elect_one()) realign_fetch(ring, q.residues, walk, gave_up);
      } else {
        Realigner ra = {};
        ra.warp = warp - 6;
        if (shape.a) ra.a = ra.places(p.a);
        if (shape.b) ra.b = ra.places(p.b);
        realign_write(
            ring, ra, walk, 0, 1, gave_up,
            [&](const SplitWalk& at) { return tc::mbar_wait(empty + 8 * at.stage.slot, at.stage.parity ^ 1, gave_up); },
            [&](const SplitWalk& at) {
              if ((threadIdx.x & 31) == 0) tc::mbar_arrive(full + 8 * at.stage.slot);
            });
      }
    }
  }
  __syncwarp();
  // split: the partial sums, [NT columns][128 rows], over the stages' memory
  float* part = reinterpret_cast<float*>(smem);
  const int row = 32 * (warp & 3) + (threadIdx.x & 31);
  const int64_t i = tm * 128 + row, j = tn * NT;
  const bool writer = warp >= 2 && warp < 6;
  if (writer) {
    tc::mbar_wait(done, 0, gave_up);
    tc::fence_after_sync();
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
      float v[16];
      if (k_hi > k_lo) {
        tc::tmem_load16(tmem + (uint32_t(32 * (warp & 3)) << 16) + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.0f;
      }
      if (q.split == 1) {
        store_columns<16>(q, i, j + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(c + e) * 128 + row] = v[e];
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (q.split > 1) {
    tc::cluster_sync();
    if (writer) {
      const int share = NT / q.split;
      for (int c = share * int(rank); c < share * int(rank + 1);) {
        if (share >= 8) {
          add_and_store<8>(q, part, c, row, i, j + c);
          c += 8;
        } else if (share >= 4) {
          add_and_store<4>(q, part, c, row, i, j + c);
          c += 4;
        } else {
          add_and_store<2>(q, part, c, row, i, j + c);
          c += 2;
        }
      }
    }
  }
  tc::fence_after_sync();
  __syncthreads();
  if (q.split > 1) tc::cluster_sync();  // no CTA leaves while another reads its sums
  if (threadIdx.x == 0 && s_gave_up != 0) tc::report_given_up(q.given_up);
  if (warp == 1) tc::tmem_free<1>(tmem, kTmemCols);
}

template <int NT>
cudaError_t launch(const GemmParams& g, bool swapped, int split, unsigned* given_up, cudaStream_t stream, const char** what) {
  SplitParamsRealign q{};
  q.g = g;
  q.given_up = given_up;
  q.swapped = swapped;
  q.split = split;
  q.b_bytes = columns_bytes<NT>(g.b.colwise != 0);
  const bool realign = !(g.a.aligned && g.b.aligned);
  const int stage = kBoxBytes + q.b_bytes + 2 * kScaleTile, room = kSmemBudget - 1024;
  const int raw = realign ? kRawDepth * kRawBox : 0, fit = (room - raw) / stage;
  q.stages = fit < kMaxStages ? fit : kMaxStages;
  const int smem = 1024 + q.stages * stage + raw;
  cudaError_t e = g.a.aligned ? operand_map(g.a, g.k, 128, &q.a, what) : cudaSuccess;
  if (e == cudaSuccess && g.b.aligned) e = operand_map(g.b, g.k, g.b.colwise ? 128 : NT, &q.b, what);
  if (e == cudaSuccess) e = scale_map(g.a, g.k, 1, &q.sa, what);
  if (e == cudaSuccess) e = scale_map(g.b, g.k, 1, &q.sb, what);
  if (e == cudaSuccess && !g.a.aligned) e = residue_maps(g.a, g.k, q.residues, what);
  if (e == cudaSuccess && !g.b.aligned) e = residue_maps(g.b, g.k, q.residues + kResidues, what);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(((g.m + 127) / 128) * ((g.n + NT - 1) / NT) * split));
  cfg.blockDim = dim3(kThreads + (realign ? 32 * kRealignWarps : 0));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  auto run = [&](auto kernel, const auto& params) {
    const cudaError_t a = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget);
    return a != cudaSuccess ? a : cudaLaunchKernelEx(&cfg, kernel, params);
  };
  return realign ? run(k_gemm_split<NT, true>, q) : run(k_gemm_split<NT, false>, static_cast<const SplitParams&>(q));
}

}  // namespace

cudaError_t launch_gemm_split(const GemmParams& p, unsigned* given_up, const DeviceInfo& dev, cudaStream_t stream,
                              const char** what) {
  // the side with fewer rows takes the columns of the tiles
  GemmParams g = p;
  const bool swapped = p.m < p.n;
  if (swapped) {
    g.a = p.b;
    g.b = p.a;
    g.m = p.n;
    g.n = p.m;
  }
  const int nt = g.n <= 16 ? 16 : (g.n <= 32 ? 32 : (g.n <= 64 ? 64 : 128));
  const int64_t tiles = ((g.m + 127) / 128) * ((g.n + nt - 1) / nt), nk = (g.k + kBlockK - 1) / kBlockK;
  // CTAs for two per SM, each with two stages or more: 64 x 8192 x 8192 takes 21.4 us with one CTA
  // per SM and 18.2 us with two (with four, half of them in a second round, 24.5 us)
  int split = 1;
  while (split < kMaxSplit && tiles * split * 2 <= 2 * dev.sms && nk >= split * 4) split *= 2;
  switch (nt) {
    case 16: return launch<16>(g, swapped, split, given_up, stream, what);
    case 32: return launch<32>(g, swapped, split, given_up, stream, what);
    case 64: return launch<64>(g, swapped, split, given_up, stream, what);
    default: return launch<128>(g, swapped, split, given_up, stream, what);
  }
}

}  // namespace mxfp8
