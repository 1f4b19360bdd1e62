// Block-scaled product for outputs of few tiles: tiles of 128 x NT by single CTAs, the contraction
// split over the CTAs of a cluster.
//
// A few tokens against a weight read the whole weight for little arithmetic: the product is bound
// by HBM, and what counts is that every SM has copies in flight from the start.  The weight's
// rows take the 128 lanes of the tile (the operands change places when the output has few rows),
// the tokens its NT = 16 .. 128 columns, and 1 to 8 CTAs share a tile, each with its part
// of k.  Their partial sums stay in shared memory, laid out as lines of the output; after a cluster
// barrier each CTA adds its share of the lines over the cluster in rank order and writes it.  No
// workspace, no atomics: the result depends on the shape, the alignment and the number of SMs (which sets the
// split) alone.
//
// Measured, launches of a graph that follow one another with three weights in turn: 1 x 4096 x 4096 5.6 us and 64 x
// 4096 x 4096 6.8 (from L2), 1 x 8192 x 8192 14.0 (from HBM, 4.8 TB/s of weight), 64 x 8192 x 8192 16.0; called
// one by one with new inputs, the first 6.2 and the last 17.2-17.5.  Streaming the weight takes 10.3 us of the last two;
// about 4 us are a launch that starts, allocates tensor memory and joins; the others are the stream's: 256
// CTAs on 152 SMs leave 48 SMs with half of the weight that the others have.  Reading the sums four at a time, with every rank's reads under way at once, took 1.6 us
// from the last: a rank's read costs about 0.4 us when the ranks take turns.
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

// Where 16-byte unit u of line r lies: units of eight neighbouring lines that threads write at once
// take different banks.
template <int NT>
__device__ __forceinline__ int unit_at(int r, int u) { return u ^ (NT >= 32 ? r & 7 : (r >> 1) & 3); }

// Adds this CTA's share of the tile's output lines over the S CTAs of the cluster, in rank order, and writes
// them.  The partial sums lie at `part` as lines of the output: 128 lines of NT sums, or with operands
// that changed places NT lines of 128.  A thread keeps W neighbouring columns, four where the output takes
// 16-byte stores, else one, and walks down the lines with kLoads loads under way at once.
template <int NT, int W, int S, int kLoads>
__device__ __forceinline__ void write_lines(const SplitParams& q, uint32_t part, int64_t i0, int64_t j0, int rank, int thread) {
  const GemmParams& p = q.g;
  constexpr int kBatch = kLoads / S;
  const int width = q.swapped ? 128 : NT, shift = 31 - __clz(width / W), step = 128 >> shift;
  const int64_t row0 = q.swapped ? j0 : i0, rows = (q.swapped ? p.n : p.m) - row0;
  const int c = (thread & ((1 << shift) - 1)) * W;
  const int64_t col = (q.swapped ? i0 : j0) + c, cols = (q.swapped ? p.m : p.n) - col;
  if (cols <= 0) return;
  const int per = (q.swapped ? NT : 128) / S;
  int line = per * rank + (thread >> shift);
  const int end = per * (rank + 1) < rows ? per * (rank + 1) : int(rows);
  uint32_t parts[S];
#pragma unroll
  for (int r = 0; r < S; ++r) parts[r] = S > 1 ? tc::in_cta(part, r) : part;
  const int64_t size = p.out_f32 ? 4 : 2;
  char* out = static_cast<char*>(p.out) + ((row0 + line) * p.ld_o + col) * size;
  const float* addend = p.addend == nullptr ? nullptr : p.addend + (row0 + line) * p.ld_c + col;
  for (; line < end; line += step * kBatch) {
    float v[kBatch][W], x[S][kBatch][W];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int at_line = line + step * b;
      const bool live = at_line < end;
      const uint32_t at = 4 * (at_line * width + (q.swapped ? c : 4 * unit_at<NT>(at_line, c >> 2) + (c & 3)));
#pragma unroll
      for (int r = 0; r < S; ++r) {
#pragma unroll
        for (int e = 0; e < W; ++e) x[r][b][e] = 0.0f;
        if constexpr (W == 4)
          asm volatile("{ .reg .pred live; setp.ne.u32 live, %5, 0;\n"
                       "@live ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4]; }"
                       : "+f"(x[r][b][0]), "+f"(x[r][b][1]), "+f"(x[r][b][2]), "+f"(x[r][b][3])
                       : "r"(parts[r] + at), "r"(uint32_t(live)));
        else
          asm volatile("{ .reg .pred live; setp.ne.u32 live, %2, 0;\n"
                       "@live ld.shared::cluster.f32 %0, [%1]; }"
                       : "+f"(x[r][b][0])
                       : "r"(parts[r] + at), "r"(uint32_t(live)));
      }
#pragma unroll
      for (int e = 0; e < W; ++e) v[b][e] = 0.0f;
      if (addend != nullptr) {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (live && e < cols) v[b][e] = addend[e];
        addend += step * p.ld_c;
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b, out += step * p.ld_o * size) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        float sum = x[0][b][e];
#pragma unroll
        for (int r = 1; r < S; ++r) sum += x[r][b][e];
        v[b][e] += sum;
      }
      if (line + step * b >= end) continue;
      if (W == 4 && cols >= W) {
        if (p.out_f32) *reinterpret_cast<float4*>(out) = make_float4(v[b][0], v[b][W > 1 ? 1 : 0], v[b][W > 2 ? 2 : 0], v[b][W > 3 ? 3 : 0]);
        else *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2_rn(v[b][0], v[b][W > 1 ? 1 : 0]), bf16x2_rn(v[b][W > 2 ? 2 : 0], v[b][W > 3 ? 3 : 0]));
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (e >= cols) continue;
          if (p.out_f32) reinterpret_cast<float*>(out)[e] = v[b][e];
          else reinterpret_cast<uint16_t*>(out)[e] = static_cast<uint16_t>(bf16x2_rn(v[b][e], 0.0f));
        }
      }
    }
  }
}

template <int NT, int W, int kLoads>
__device__ __forceinline__ void write_lines(const SplitParams& q, uint32_t part, int64_t i0, int64_t j0, int rank, int thread) {
  if (q.split == 1) write_lines<NT, W, 1, kLoads>(q, part, i0, j0, rank, thread);
  else if (q.split == 2) write_lines<NT, W, 2, kLoads>(q, part, i0, j0, rank, thread);
  else if (q.split == 4) write_lines<NT, W, 4, kLoads>(q, part, i0, j0, rank, thread);
  else write_lines<NT, W, 8, kLoads>(q, part, i0, j0, rank, thread);
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
      uint32_t issued = 0;
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
      if (*gave_up != 0) tc::settle_copies(full, uint32_t(q.stages), issued);
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
  // the sums, as lines of the output, over the stages' memory
  float* part = reinterpret_cast<float*>(smem);
  const bool writer = warp >= 2 && warp < 6;
  if (writer) {
    const int row = 32 * (warp & 3) + (threadIdx.x & 31);
    tc::mbar_wait(done, 0, gave_up);
    tc::fence_after_sync();
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
      float v[16];
      tc::tmem_load16(tmem + (uint32_t(32 * (warp & 3)) << 16) + c, v);
      if (q.swapped) {
#pragma unroll
        for (int e = 0; e < 16; ++e) part[(c + e) * 128 + row] = v[e];
      } else {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<float4*>(part + row * NT + 4 * unit_at<NT>(row, (c + e) >> 2)) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_free<1>(tmem, kTmemCols);
  if (q.split > 1) tc::cluster_sync();
  if (writer) {
    if (p.vec_out) write_lines<NT, 4, kRealign ? 8 : 16>(q, tc::smem_addr(part), tm * 128, tn * NT, int(rank), threadIdx.x - 64);
    else write_lines<NT, 1, kRealign ? 16 : 32>(q, tc::smem_addr(part), tm * 128, tn * NT, int(rank), threadIdx.x - 64);
  }
  __syncwarp();
  if (q.split > 1) tc::cluster_sync();  // no CTA leaves while another reads its sums: a release, behind every load
  if (threadIdx.x == 0 && s_gave_up != 0) tc::report_given_up(q.given_up);
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
  // CTAs that share a tile, each with two stages or more.  Two CTAs per SM where the copies of one do not
  // fill the SM's share of HBM or the realigning warps bound it, else one: 64 x 8192 x 8192 18.1 us with
  // one, 16.7 with two (23 with four, half of them in a second round), 1024 x 1024 x 8192 14.0 and 15.5.
  // Eight to a tile join slower than four; they pay on half of the SMs (64 x 1024 x 4096 6.0 and 6.5 us,
  // 64 x 2048 x 4096 7.4 and 6.5), or with little to join (1 x 4096 x 4096 5.5 and 5.7).
  const int64_t two = nt <= 64 || !(g.a.aligned && g.b.aligned) ? 2 * dev.sms : dev.sms;
  const int64_t eight = nt == 16 ? 2 * dev.sms : dev.sms / 2;
  int split = 1;
  while (split < kMaxSplit && tiles * split * 2 <= (split == 4 ? eight : two) && nk >= split * 4) split *= 2;
  switch (nt) {
    case 16: return launch<16>(g, swapped, split, given_up, stream, what);
    case 32: return launch<32>(g, swapped, split, given_up, stream, what);
    case 64: return launch<64>(g, swapped, split, given_up, stream, what);
    default: return launch<128>(g, swapped, split, given_up, stream, what);
  }
}

}  // namespace mxfp8
