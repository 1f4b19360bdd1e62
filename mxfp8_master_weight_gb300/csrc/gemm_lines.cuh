// The end of a product whose contraction is split over the CTAs of a cluster: their partial sums, joined and written.
#pragma once

#include "gemm_impl.cuh"

namespace mxfp8 {

// Where 16-byte unit u of line r lies: units of eight neighbouring lines that threads write at once
// take different banks.
template <int NT>
__device__ __forceinline__ int unit_at(int r, int u) { return u ^ (NT >= 32 ? r & 7 : (r >> 1) & 3); }

// Of sums that are the result as they are.
struct NoFactor {
  template <int N>
  __device__ __forceinline__ void apply(float (&)[N]) const {}
};

// Adds this CTA's share of the tile's output lines over the S CTAs of the cluster, in rank order, multiplies the joined sums
// by `factor`, adds the addend and writes them.  The partial sums lie at `part` as lines of the output: 128 lines of NT sums,
// or with operands that changed places NT lines of 128.  A thread keeps W neighbouring columns, four where the output takes
// 16-byte stores, else one, and walks down the lines with kLoads loads under way at once.
template <int NT, int W, int S, int kLoads, class F>
__device__ __forceinline__ void write_lines(const GemmParams& p, const F& factor, bool swapped, uint32_t part, int64_t i0, int64_t j0,
                                            int rank, int thread) {
  constexpr int kBatch = kLoads / S;
  const int width = swapped ? 128 : NT, shift = 31 - __clz(width / W), step = 128 >> shift;
  const int64_t row0 = swapped ? j0 : i0, rows = (swapped ? p.n : p.m) - row0;
  const int c = (thread & ((1 << shift) - 1)) * W;
  const int64_t col = (swapped ? i0 : j0) + c, cols = (swapped ? p.m : p.n) - col;
  if (cols <= 0) return;
  const int per = (swapped ? NT : 128) / S;
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
      const uint32_t at = 4 * (at_line * width + (swapped ? c : 4 * unit_at<NT>(at_line, c >> 2) + (c & 3)));
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
      float sum[W];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        sum[e] = x[0][b][e];
#pragma unroll
        for (int r = 1; r < S; ++r) sum[e] += x[r][b][e];
      }
      factor.apply(sum);
#pragma unroll
      for (int e = 0; e < W; ++e) v[b][e] += sum[e];
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

template <int NT, int W, int kLoads, class F>
__device__ __forceinline__ void write_lines(const GemmParams& p, const F& factor, bool swapped, int split, uint32_t part, int64_t i0,
                                            int64_t j0, int rank, int thread) {
  if (split == 1) write_lines<NT, W, 1, kLoads>(p, factor, swapped, part, i0, j0, rank, thread);
  else if (split == 2) write_lines<NT, W, 2, kLoads>(p, factor, swapped, part, i0, j0, rank, thread);
  else if (split == 4) write_lines<NT, W, 4, kLoads>(p, factor, swapped, part, i0, j0, rank, thread);
  else write_lines<NT, W, 8, kLoads>(p, factor, swapped, part, i0, j0, rank, thread);
}

}  // namespace mxfp8
