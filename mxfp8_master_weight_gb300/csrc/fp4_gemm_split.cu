// Product of NVFP4 operands for outputs of few tiles: tiles of 128 x NT by single CTAs, the contraction split over the
// CTAs of a cluster.
//
// A few tokens against a weight read the whole weight for little arithmetic, so what counts is that every SM
// has copies in flight from the start.  The weight's rows take the 128 lanes of the tile (the operands change places
// when the output has few rows), the tokens its NT = 16 .. 128 columns, and 1 to 8 CTAs share a tile, each with its
// part of k.  After a cluster barrier each CTA adds its share of the tile's output lines over the cluster in rank order
// and writes them: no workspace, no atomics.  Partial sums of up to 32 columns are sent to the CTA that adds them, into a
// place of their own behind the stages, so that one barrier is between them and the output (1 x 4096 x 4096 4.2 us, with the
// sums read over the cluster 4.9).  Of more columns they stay where they are made, over the stages, and are read by the CTA
// that adds them: a place of their own would cost a stage (64 x 8192 x 8192 11.9 us, 12.2 with it, 12.7 sent over the stages
// behind a barrier more).
//
// What bounds it: a launch that starts, allocates tensor memory and joins takes about 3.5 us (1 x 1024 x 4096); the rest is the
// weight's stream: 1 x 8192 x 8192 8.3 us for 38 MB, 16 x 8192 x 8192 8.8, 1 x 16384 x 4096 8.6 (launches of a graph, three weights
// in turn); called one by one with new inputs 1 x 4096 x 4096 4.6 and 64 x 8192 x 8192 13.0.
#include <cuda.h>

#include "fp4.cuh"
#include "fp4_gemm.h"
#include "gemm_lines.cuh"
#include "gemm_maps.h"
#include "launch.h"

namespace mxfp8 {
namespace {

constexpr int kThreads = 192;  // warp 0 fetches, warp 1 issues, four warps write
constexpr int kMaxSplit = 8;
constexpr int kMaxStages = 8;
constexpr int kScales = 4 * kScaleTile;  // of 128 rows and a stage
constexpr int kSmemBudget = 112 * 1024;  // two CTAs share an SM
template <int NT>
constexpr bool kApart = NT <= 32;        // sums are sent to a place of their own

struct SplitParams {
  Fp4GemmParams f;    // a: the 128-row side, b: the NT-column side
  CUtensorMap a, b, sa, sb;
  unsigned* given_up;
  int32_t swapped;    // out[column][row]: the caller's A is b here
  int32_t stages, split;
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 2) k_fp4_gemm_split(const __grid_constant__ SplitParams q) {
  extern __shared__ char raw[];
  const GemmParams& p = q.f.g;
  constexpr int kBBytes = NT * 128;
  constexpr uint32_t kTmemCols = NT <= 64 ? 128 : 256;  // two sets of 16 + 16 scale columns behind the sums
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  char* b_boxes = smem + q.stages * kBoxBytes;
  char* scales = b_boxes + q.stages * kBBytes;
  __shared__ uint64_t bars[2 * kMaxStages + 1];
  __shared__ uint32_t tmem_slot, s_gave_up;
  volatile uint32_t* gave_up = &s_gave_up;
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kMaxStages, done = empty + 8 * kMaxStages;
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = q.split > 1 ? tc::cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.stages; ++s) {
      tc::mbar_init(full + 8 * s, 1);
      tc::mbar_init(empty + 8 * s, 1);
    }
    tc::mbar_init(done, 1);
    s_gave_up = 0;
    tc::mbar_init_fence();
    tc::prefetch_map(&q.a);
    tc::prefetch_map(&q.b);
    tc::prefetch_map(&q.sa);
    tc::prefetch_map(&q.sb);
  }
  if (warp == 1) tc::tmem_alloc<1>(tc::smem_addr(&tmem_slot), kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (kApart<NT> && q.split > 1) tc::cluster_started();
  tc::grid_wait_then_release();
  const uint32_t tmem = tmem_slot;
  int64_t tm, tn;
  tile_at(blockIdx.x / q.split, (p.m + 127) / 128, (p.n + NT - 1) / NT, tm, tn);
  const int64_t nk = (p.k + kFp4StageK - 1) / kFp4StageK;
  const int64_t k_lo = nk * rank / q.split, k_hi = nk * (rank + 1) / q.split;

  if (warp == 0) {
    if (tc::elect_one()) {
      int s = 0;
      uint32_t phase = 1;
      uint32_t issued = 0;
      const int am = int(tm * 128), bn = int(tn * NT);
      for (int64_t kb = k_lo; kb < k_hi; ++kb) {
        if (!tc::mbar_wait(empty + 8 * s, phase, gave_up)) break;
        const uint32_t at_s = tc::smem_addr(scales + s * 2 * kScales), bar = full + 8 * s;
        tc::mbar_expect(bar, uint32_t(kBoxBytes + kBBytes + 2 * kScales));
        tc::tma_load_2d(tc::smem_addr(smem + s * kBoxBytes), &q.a, int(kb * 128), am, bar);
        tc::tma_load_2d(tc::smem_addr(b_boxes + s * kBBytes), &q.b, int(kb * 128), bn, bar);
        tc::tma_load_3d(at_s, &q.sa, 0, int(4 * kb), int(tm), bar);
        tc::tma_load_3d(at_s + kScales, &q.sb, 0, int(4 * kb), bn >> 7, bar);
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
      constexpr uint32_t idesc = tc::instr_desc4(128, NT);
      int s = 0;
      uint32_t phase = 0;
      for (int64_t kb = k_lo; kb < k_hi; ++kb) {
        if (!tc::mbar_wait(full + 8 * s, phase, gave_up)) break;
        tc::fence_after_sync();
        const uint32_t at_a = tc::smem_addr(smem + s * kBoxBytes), at_b = tc::smem_addr(b_boxes + s * kBBytes),
                       at_s = tc::smem_addr(scales + s * 2 * kScales);
        const uint32_t sa = tmem + NT + 32 * uint32_t(kb & 1), sb = sa + 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tc::copy_scales<1>(sa + 4 * j, tc::scale_desc(at_s + j * kScaleTile));
          tc::copy_scales<1>(sb + 4 * j, tc::scale_desc(at_s + kScales + j * kScaleTile));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc::mma_scaled4<1>(tmem, tc::operand_desc(at_a + 32 * j), tc::operand_desc(at_b + 32 * j), idesc, sa + 4 * j,
                             sb + 4 * j, kb > k_lo || j > 0);
        tc::commit(empty + 8 * s);
        if (++s == q.stages) {
          s = 0;
          phase ^= 1;
        }
      }
      tc::commit(done);
    }
  }
  __syncwarp();
  // The joined sums are multiplied by it, not each part of k: parts that cancel would leave what their roundings differ by,
  // or overflow.
  Fp4Factor factor;
  if (warp >= 2) factor = Fp4Factor(*q.f.a_amax, *q.f.b_amax);
  if constexpr (kApart<NT>) {
    if (q.split > 1) tc::cluster_all_started();
    char* received = scales + q.stages * 2 * kScales;  // [rank][line of this CTA's][column]
    // Lines of the output: 128 of NT sums, or with operands that changed places NT of 128; `per` of them are each CTA's.
    const int width = q.swapped ? 128 : NT, per = (q.swapped ? NT : 128) / q.split, shift_per = 31 - __clz(per);
    if (warp >= 2) {
      const int row = 32 * (warp & 3) + (threadIdx.x & 31);
      const uint32_t mine = tc::smem_addr(received) + 4 * per * width * rank;
      tc::mbar_wait(done, 0, gave_up);
      tc::fence_after_sync();
      if (q.swapped) {
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          float v[16];
          tc::tmem_load16(tmem + (uint32_t(32 * (warp & 3)) << 16) + c, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) {  // 16 lines, of one owner or several
            const int owner = (c + e) >> shift_per;
            tc::store_cluster(tc::in_cta(mine + 4 * ((c + e - owner * per) * 128 + row), owner), v[e]);
          }
        }
      } else {
        const int owner = row >> shift_per, line = row - owner * per;
        const uint32_t to = tc::in_cta(mine + 4 * line * NT, owner);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          float v[16];
          tc::tmem_load16(tmem + (uint32_t(32 * (warp & 3)) << 16) + c, v);
#pragma unroll
          for (int e = 0; e < 16; e += 4) tc::store_cluster4(to + 16 * unit_at<NT>(line, (c + e) >> 2), v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
    }
    tc::fence_before_sync();
    if (q.split > 1) tc::cluster_sync();
    else __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_free<1>(tmem, kTmemCols);
    if (warp >= 2) {
      const int units = width / 4, shift = 31 - __clz(units);
      const int64_t row0 = (q.swapped ? tn * NT : tm * 128) + per * int64_t(rank), col0 = q.swapped ? tm * 128 : tn * NT;
      const int64_t rows = q.swapped ? p.n : p.m, cols = q.swapped ? p.m : p.n;
      const float* sums = reinterpret_cast<const float*>(received);
      for (int u = int(threadIdx.x) - 64; u < per * units; u += 128) {
        const int line = u >> shift, c = (u & (units - 1)) * 4;
        const int64_t r = row0 + line, j = col0 + c;
        if (r >= rows || j >= cols) continue;
        const int at = line * width + (q.swapped ? c : 4 * unit_at<NT>(line, c >> 2));
        float4 v = *reinterpret_cast<const float4*>(sums + at);
        for (int s = 1; s < q.split; ++s) {
          const float4 x = *reinterpret_cast<const float4*>(sums + s * per * width + at);
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
        }
        float e[4] = {v.x, v.y, v.z, v.w};
        factor.apply(e);
        const int n = cols - j < 4 ? int(cols - j) : 4;
        if (p.addend != nullptr) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < n) e[k] += p.addend[r * p.ld_c + j + k];
        }
        if (p.out_f32) {
          float* o = static_cast<float*>(p.out) + r * p.ld_o + j;
          if (p.vec_out && n == 4) {
            *reinterpret_cast<float4*>(o) = make_float4(e[0], e[1], e[2], e[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < n) o[k] = e[k];
          }
        } else {
          uint16_t* o = static_cast<uint16_t*>(p.out) + r * p.ld_o + j;
          const uint2 w = make_uint2(bf16x2_rn(e[0], e[1]), bf16x2_rn(e[2], e[3]));
          if (p.vec_out && n == 4) {
            *reinterpret_cast<uint2*>(o) = w;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < n) o[k] = uint16_t((k < 2 ? w.x : w.y) >> (16 * (k & 1)));
          }
        }
      }
    }
  } else {
    // the sums, as lines of the output, over the stages' memory
    float* part = reinterpret_cast<float*>(smem);
    const bool writer = warp >= 2;
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
      if (p.vec_out) write_lines<NT, 4, 16>(p, factor, q.swapped, q.split, tc::smem_addr(part), tm * 128, tn * NT, int(rank), threadIdx.x - 64);
      else write_lines<NT, 1, 32>(p, factor, q.swapped, q.split, tc::smem_addr(part), tm * 128, tn * NT, int(rank), threadIdx.x - 64);
    }
    __syncwarp();
    if (q.split > 1) tc::cluster_sync();  // no CTA leaves while another reads its sums: a release, behind every load
  }
  if (threadIdx.x == 0 && s_gave_up != 0) tc::report_given_up(q.given_up);
}

template <int NT>
cudaError_t launch(const Fp4GemmParams& f, bool swapped, int split, unsigned* given_up, int device, cudaStream_t stream, const char** what) {
  SplitParams q{};
  q.f = f;
  q.given_up = given_up;
  q.swapped = swapped;
  q.split = split;
  const GemmParams& g = f.g;
  constexpr int stage = kBoxBytes + NT * 128 + 2 * kScales, sums = 128 * NT * 4, apart = kApart<NT> ? sums : 0,
                fit = (kSmemBudget - 1024 - apart) / stage;
  static_assert(fit >= 2 && fit * stage + apart >= sums, "stages");
  q.stages = fit < kMaxStages ? fit : kMaxStages;
  const int smem = 1024 + q.stages * stage + apart;
  cudaError_t e = operand_map(g.a, (g.k + 1) / 2, 128, &q.a, what);
  if (e == cudaSuccess) e = operand_map(g.b, (g.k + 1) / 2, NT, &q.b, what);
  if (e == cudaSuccess) e = scale_map(g.a, g.k, 1, &q.sa, what, 4);
  if (e == cudaSuccess) e = scale_map(g.b, g.k, 1, &q.sb, what, 4);
  static std::atomic<unsigned long long> done{0};
  if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(k_fp4_gemm_split<NT>), kSmemBudget, device, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(((g.m + 127) / 128) * ((g.n + NT - 1) / NT) * split));
  cfg.blockDim = dim3(kThreads);
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
  return cudaLaunchKernelEx(&cfg, k_fp4_gemm_split<NT>, q);
}

}  // namespace

cudaError_t launch_fp4_gemm_split(const Fp4GemmParams& p, unsigned* given_up, const DeviceInfo& dev, cudaStream_t stream,
                                  const char** what) {
  // the side with fewer rows takes the columns of the tiles
  Fp4GemmParams f = p;
  const bool swapped = p.g.m < p.g.n;
  if (swapped) {
    f.g.a = p.g.b;
    f.g.b = p.g.a;
    f.g.m = p.g.n;
    f.g.n = p.g.m;
    f.a_amax = p.b_amax;
    f.b_amax = p.a_amax;
  }
  // 16, 32 and 64 columns are whole outputs (one tile of columns), so a tile of columns starts on a whole scale tile
  const int nt = f.g.n <= 16 ? 16 : (f.g.n <= 32 ? 32 : (f.g.n <= 64 ? 64 : 128));
  const int64_t tiles = ((f.g.m + 127) / 128) * ((f.g.n + nt - 1) / nt), nk = (f.g.k + kFp4StageK - 1) / kFp4StageK;
  // CTAs that share a tile, each with four stages or more.  Two CTAs per SM up to 64 columns (64 x 8192 x 8192 with one 12.8 us, with
  // two 11.9); eight to a tile on half of the SMs, or with few columns to join (1 x 1024 x 4096 4.3 us, four 4.7).
  const int64_t two = nt <= 64 ? 2 * dev.sms : dev.sms, eight = nt == 16 ? 2 * dev.sms : dev.sms / 2;
  int split = 1;
  while (split < kMaxSplit && tiles * split * 2 <= (split == 4 ? eight : two) && nk >= split * 4) split *= 2;
  switch (nt) {
    case 16: return launch<16>(f, swapped, split, given_up, dev.device, stream, what);
    case 32: return launch<32>(f, swapped, split, given_up, dev.device, stream, what);
    case 64: return launch<64>(f, swapped, split, given_up, dev.device, stream, what);
    default: return launch<128>(f, swapped, split, given_up, dev.device, stream, what);
  }
}

}  // namespace mxfp8
