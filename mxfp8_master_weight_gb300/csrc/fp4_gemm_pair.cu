// Product of NVFP4 operands for large outputs: tiles of 256 x 256 by pairs of CTAs.
//
// The two SMs of a pair work on one tile with one stream of matrix instructions (cta_group::2, 256 x 256 x 64): each
// holds 128 rows of A, 128 rows of B and 128 rows of the sums.  A stage is 256 values of k: 16 KB of each operand's
// codes, 2 KB of A's scales and 4 KB of B's (each CTA needs those of all 256 columns).
//
// Roles in a CTA: warp 0 fetches (one thread, TMA), warp 1 of the leading CTA issues scale copies and matrix
// instructions for both, eight warps write the sums out.  When the last round of tiles would occupy at most half of the
// pairs, its tiles are cut into halves of 256 x 128.
//
// Tensor memory has 512 columns; a stage's scales take 48 (16 for A, 32 for B), of which there are two sets, so the two
// buffers of 256 sums share 96 columns: buffer 0 is columns 0..255, buffer 1 columns 160..415.  The writers
// drain the shared columns of a tile first; then the next tile's instructions start in the other buffer.
// Where the output's rows start and end on 16 bytes and nothing is added, the sums leave through TMA from 4 KB of shared memory
// of each writer (16384 x 8192 x 256, all output, 44 us; by the writers' own stores 121); else by their own stores.
//
// What bounds it, with the instruction's form of 64 values of k (sm_103a has one of 96 as well, which is not used here): shared
// memory.  Per stage an SM writes 38 KB (38912 bytes) to it and its matrix instructions read as much, 608 cycles at 128 bytes a
// cycle, where they would compute for 512; a stage takes 654 (with all loads but a quarter of the instructions 522, with the
// instructions alone 564).  Then the board's power: 8192^3 155 us (7.1 PFLOP/s), at 1.83 GHz; 165-172 in loops of a second.  4096^3:
// 26.5 us on three sets of operands in turn, 27.5 with new inputs in every pass: 3.5 rounds of tiles of 5 us, about 1 us
// between two tiles of a pair, start and end.  2048 x 8192 x 8192 with F32 output 51.6 us, 58.8 with an addend and new inputs.
#include <cuda.h>

#include "fp4.cuh"
#include "fp4_gemm.h"
#include "gemm_impl.cuh"
#include "gemm_maps.h"
#include "launch.h"

namespace mxfp8 {
namespace {

constexpr int kMaxStages = 7;
constexpr int kScalesA = 4 * kScaleTile, kScalesB = 8 * kScaleTile, kScaleBytes = kScalesA + kScalesB;
constexpr int kWriters = 8;
constexpr int kWriterBytes = 4096;  // a writer's 32 rows of 128 bytes
constexpr int kThreads = 64 + 32 * kWriters;
constexpr int kSmem = 226 * 1024;
constexpr int kStageRoom = kSmem - 1024 - kWriters * kWriterBytes - 384;
constexpr int kSecondBuffer = 160;  // first column of the second buffer of sums
constexpr int kScaleCol = 416, kScaleSet = 48;
static_assert(kScaleCol + 2 * kScaleSet == 512 && kSecondBuffer + 256 == kScaleCol, "tensor memory");

struct PairParams {
  Fp4GemmParams f;
  CUtensorMap a, b, b_half, sa, sb, out;
  unsigned* given_up;
  int64_t whole, units;  // whole tiles first, then halves
  int32_t stages, b_bytes;
};

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

// How the sums leave: through TMA as BF16 or F32, or by the writers' own stores (an addend, rows that start anywhere).
enum Out { kOutBf16, kOutF32, kOutAny };

template <Out kOut>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_fp4_gemm_pair(const __grid_constant__ PairParams q) {
  extern __shared__ char raw[];
  const GemmParams& p = q.f.g;
  // the same offset in both CTAs: their dynamic shared memory starts alike
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  char* b_boxes = smem + q.stages * kBoxBytes;
  char* scales = b_boxes + q.stages * q.b_bytes;
  char* writers = scales + q.stages * kScaleBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(writers + kWriters * kWriterBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 3);
  volatile uint32_t* gave_up = tmem_slot + 1;
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kMaxStages, sums_full = empty + 8 * kMaxStages,
                 sums_free = sums_full + 16;
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = tc::cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < q.stages; ++s) {
      tc::mbar_init(full + 8 * s, 1);
      tc::mbar_init(empty + 8 * s, 1);
    }
    tc::mbar_init(sums_full, 1);
    tc::mbar_init(sums_full + 8, 1);
    tc::mbar_init(sums_free, 2 * kWriters);
    *gave_up = 0;
    tc::mbar_init_fence();
    if (p.k > 0) {
      tc::prefetch_map(&q.a);
      if (q.whole > 0) tc::prefetch_map(&q.b);
      if (q.whole < q.units) tc::prefetch_map(&q.b_half);
      tc::prefetch_map(&q.sa);
      tc::prefetch_map(&q.sb);
    }
  }
  if (warp == 1) tc::tmem_alloc<2>(tc::smem_addr(tmem_slot), 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  tc::grid_wait_then_release();
  const uint32_t tmem = *tmem_slot;
  const int64_t tiles_m = (p.m + 255) / 256, tiles_n = (p.n + 255) / 256;
  const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int64_t nk = (p.k + kFp4StageK - 1) / kFp4StageK;

  if (warp == 0) {
    if (tc::elect_one()) {
      const uint32_t lead_full = tc::in_cta(full, 0);
      int s = 0;
      uint32_t phase = 1;
      uint32_t issued = 0;
      for (int64_t unit = first; unit < q.units && *gave_up == 0; unit += step) {
        const Tile t = tile_of(q, unit, tiles_m, tiles_n);
        const int am = int(t.tm * 256 + rank * 128), bn = int(t.col + rank * (t.half ? 64 : 128));
        const uint32_t bytes = kBoxBytes + (t.half ? kBoxBytes / 2 : kBoxBytes) + kScaleBytes;
        for (int64_t kb = 0; kb < nk; ++kb) {
          if (!tc::mbar_wait(empty + 8 * s, phase, gave_up)) break;
          const uint32_t at_a = tc::smem_addr(smem + s * kBoxBytes), at_b = tc::smem_addr(b_boxes + s * q.b_bytes),
                         at_s = tc::smem_addr(scales + s * kScaleBytes), bar = lead_full + 8 * s;
          if (rank == 0) tc::mbar_expect(full + 8 * s, 2 * bytes);
          tc::tma_load_2d_pair(at_a, &q.a, int(kb * 128), am, bar);
          tc::tma_load_2d_pair(at_b, t.half ? &q.b_half : &q.b, int(kb * 128), bn, bar);
          tc::tma_load_3d_pair(at_s, &q.sa, 0, int(4 * kb), int(2 * t.tm + rank), bar);
          tc::tma_load_3d_pair(at_s + kScalesA, &q.sb, 0, int(4 * kb), int(t.col >> 7), bar);
          ++issued;
          if (++s == q.stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // Neither CTA leaves before the other one's last arrivals have come in.
      for (int i = 0; i < q.stages && *gave_up == 0; ++i) {
        tc::mbar_wait(empty + 8 * s, phase, gave_up);
        if (++s == q.stages) {
          s = 0;
          phase ^= 1;
        }
      }
      if (*gave_up != 0 && rank == 0) tc::settle_copies(full, uint32_t(q.stages), issued);
    }
  } else if (warp == 1) {
    if (rank == 0 && tc::elect_one()) {
      int s = 0;
      uint32_t phase = 0, nth = 0, set = 0;
      bool good = true;
      for (int64_t unit = first; unit < q.units && good; unit += step, ++nth) {
        if (nth > 0) good = tc::mbar_wait(sums_free, (nth - 1) & 1, gave_up);
        tc::fence_after_sync();
        const uint32_t d = tmem + (nth & 1 ? kSecondBuffer : 0);
        const uint32_t idesc = tc::instr_desc4(256, unit >= q.whole ? 128 : 256);
        for (int64_t kb = 0; kb < nk && good; ++kb) {
          good = tc::mbar_wait(full + 8 * s, phase, gave_up);
          if (!good) break;
          tc::fence_after_sync();
          const uint32_t at_a = tc::smem_addr(smem + s * kBoxBytes), at_b = tc::smem_addr(b_boxes + s * q.b_bytes),
                         at_s = tc::smem_addr(scales + s * kScaleBytes);
          const uint32_t sa = tmem + kScaleCol + kScaleSet * set, sb = sa + 16;
          set ^= 1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            tc::copy_scales<2>(sa + 4 * j, tc::scale_desc(at_s + j * kScaleTile));
            tc::copy_scales<2>(sb + 8 * j, tc::scale_desc(at_s + kScalesA + j * kScaleTile));
            tc::copy_scales<2>(sb + 8 * j + 4, tc::scale_desc(at_s + kScalesA + (4 + j) * kScaleTile));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_scaled4<2>(d, tc::operand_desc(at_a + 32 * j), tc::operand_desc(at_b + 32 * j), idesc, sa + 4 * j,
                               sb + 8 * j, kb > 0 || j > 0);
          tc::commit_pair(empty + 8 * s, 3);
          if (++s == q.stages) {
            s = 0;
            phase ^= 1;
          }
        }
        tc::commit_pair(sums_full + 8 * (nth & 1), 3);
      }
    }
  } else {
    const int side = (warp - 2) >> 2;  // the first or second half of the columns
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const int lane = threadIdx.x & 31;
    const Fp4Factor factor(p.k > 0 ? *q.f.a_amax : 0.0f, p.k > 0 ? *q.f.b_amax : 0.0f);
    uint32_t nth = 0;
    for (int64_t unit = first; unit < q.units; unit += step, ++nth) {
      const Tile t = tile_of(q, unit, tiles_m, tiles_n);
      const uint32_t buffer = nth & 1;
      // no two tiles' sums are ready at once that this warp has not drained: the next tile's
      // instructions wait for sums_free
      if (!tc::mbar_wait(sums_full + 8 * buffer, (nth >> 1) & 1, gave_up)) break;
      tc::fence_after_sync();
      const int64_t row0 = t.tm * 256 + 128 * rank + 32 * (warp & 3);
      const uint32_t d = tmem + lanes + (buffer ? kSecondBuffer : 0);
      // 64 columns at a time, the two sides in turn.  The shared columns, the last of buffer 0 and the first of buffer 1,
      // are in registers after the first 64 of both; the arrival then also says that the warp is done with the
      // tile before.
      const int parts = t.half ? 1 : 2;
#pragma unroll 1
      for (int i = 0; i < parts; ++i) {
        const int c = 64 * (2 * (buffer ? i : parts - 1 - i) + side);
        float v[64];
        if (nk > 0) {
          tc::tmem_load64(d + c, v);
        } else {
#pragma unroll
          for (int k = 0; k < 64; ++k) v[k] = 0.0f;
        }
        if (i == 0) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_cluster_relaxed(sums_free, 0);
        }
        factor.apply(v);
        char* stage = writers + (warp - 2) * kWriterBytes;
        if constexpr (kOut == kOutAny) {
          auto part = [&](int e0) {
            return [&v, e0](int e, float(&o)[32]) {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = v[e0 + e + k];
            };
          };
          write_rows(p, stage, row0, t.col + c, part(0));
          if (p.out_f32) write_rows(p, stage, row0, t.col + c + 32, part(32));
        } else {
          if (row0 >= p.m) continue;
#pragma unroll
          for (int h = 0; h < (kOut == kOutF32 ? 2 : 1); ++h) {
            const int64_t col = t.col + c + 32 * h;
            if (col >= p.n) break;
            if (lane == 0) tc::bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              uint4 w;
              if constexpr (kOut == kOutF32) {
                const float* e = v + 32 * h + 4 * u;
                w = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3]));
              } else {
                const float* e = v + 8 * u;
                w = make_uint4(bf16x2_rn(e[0], e[1]), bf16x2_rn(e[2], e[3]), bf16x2_rn(e[4], e[5]), bf16x2_rn(e[6], e[7]));
              }
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = w;
            }
            tc::fence_async_proxy();
            __syncwarp();
            if (lane == 0) {
              tc::tma_store_2d(&q.out, tc::smem_addr(stage), int(col), int(row0));
              tc::bulk_commit();
            }
          }
        }
      }
    }
    if (kOut != kOutAny && lane == 0) tc::bulk_wait();
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

cudaError_t launch_fp4_gemm_pair(const Fp4GemmParams& f, unsigned* given_up, const DeviceInfo& dev, cudaStream_t stream,
                                 const char** what) {
  PairParams q{};
  q.f = f;
  q.given_up = given_up;
  const GemmParams& g = f.g;
  const int64_t bytes = (g.k + 1) / 2;
  const int64_t tiles = ((g.m + 255) / 256) * ((g.n + 255) / 256);
  const int64_t pairs = dev.sms / 2, last = tiles % pairs;
  q.whole = last != 0 && 2 * last <= pairs ? tiles - last : tiles;
  q.units = q.whole + 2 * (tiles - q.whole);
  q.b_bytes = q.whole == 0 ? kBoxBytes / 2 : kBoxBytes;
  const int fit = kStageRoom / (kBoxBytes + q.b_bytes + kScaleBytes);
  q.stages = fit < kMaxStages ? fit : kMaxStages;
  cudaError_t e = cudaSuccess;
  if (g.k > 0) {
    e = operand_map(g.a, bytes, 128, &q.a, what);
    if (e == cudaSuccess && q.whole > 0) e = operand_map(g.b, bytes, 128, &q.b, what);
    if (e == cudaSuccess && q.whole < q.units) e = operand_map(g.b, bytes, 64, &q.b_half, what);
    if (e == cudaSuccess) e = scale_map(g.a, g.k, 1, &q.sa, what, 4);
    if (e == cudaSuccess) e = scale_map(g.b, g.k, 2, &q.sb, what, 4);
  }
  if (e != cudaSuccess) return e;
  const unsigned grid = 2 * unsigned(q.units < pairs ? q.units : pairs);
  static std::atomic<unsigned long long> told[3];
  auto run = [&](auto kernel, std::atomic<unsigned long long>* done) {
    const cudaError_t r = allow_smem(reinterpret_cast<const void*>(kernel), kSmem, dev.device, done);
    return r != cudaSuccess ? r : launch_kernel(kernel, dim3(grid), dim3(kThreads), kSmem, stream, q);
  };
  // A store through TMA ends a row on 16 bytes: it would write past one that ends elsewhere.
  if (g.addend != nullptr || !g.vec_out || g.n % (g.out_f32 ? 4 : 8) != 0) return run(k_fp4_gemm_pair<kOutAny>, &told[kOutAny]);
  e = output_map(g, &q.out, what);
  if (e != cudaSuccess) return e;
  return g.out_f32 ? run(k_fp4_gemm_pair<kOutF32>, &told[kOutF32]) : run(k_fp4_gemm_pair<kOutBf16>, &told[kOutBf16]);
}

}  // namespace mxfp8
