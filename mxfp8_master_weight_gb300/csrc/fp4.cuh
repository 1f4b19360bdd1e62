// Scale and code arithmetic of NVFP4 operands (see nvfp4_quantize in the header of the library).
#pragma once

#include <cfloat>

#include "common.cuh"

namespace mxfp8 {

// S of the tensor whose largest magnitude is g: 2688 / g (448 * 6: the largest scale times the largest code),
// 1 for 0, the largest float if the quotient overflows; NaN where g is not finite, so that every scale is.
__device__ __forceinline__ float fp4_tensor_scale(float g) {
  if (g == 0.0f) return 1.0f;
  const float s = __fdiv_rn(2688.0f, g);
  return fabsf(g) <= FLT_MAX ? fminf(s, FLT_MAX) : __uint_as_float(0x7fc00000u);
}

// fp32(a / 6) for a >= 0, correctly rounded: a product with the rounded reciprocal, the exact remainder, one
// correction (P. Markstein, IBM J. Res. Dev. 34(1), 1990); equal to the quotient for 0 and from 2^-124 up to the largest
// float (tests/test_div6_identity.py); NaN for an infinity.  Below 2^-124 the remainder may be subnormal and the result off
// by units in the last place, which only a tensor of largest magnitude under 2^-100 can tell: any other's scales of
// such blocks round to 0.  For those, `tiny` takes the division itself.
__device__ __forceinline__ float fp4_div6(float a, bool tiny) {
  constexpr float kInv6 = 0x1.555556p-3f;
  if (tiny) return __fdiv_rn(a, 6.0f);
  const float q = __fmul_rn(a, kInv6);
  return __fmaf_rn(__fmaf_rn(-6.0f, q, a), kInv6, q);
}
__device__ __forceinline__ bool fp4_tiny(float amax) { return amax < 0x1p-100f; }

// The scale bytes of two blocks of largest magnitudes a and b, b's in the second byte: E4M3(fp32(fp32(a / 6) * S)), NaN
// (0x7F) where the block or S is not finite.
__device__ __forceinline__ uint32_t fp4_block_scales(float a, float b, float tensor_scale, bool tiny) {
  if (tiny) {  // the division of an infinity is one: made NaN, as it comes out below
    a = a <= FLT_MAX ? a : __uint_as_float(0x7fc00000u);
    b = b <= FLT_MAX ? b : __uint_as_float(0x7fc00000u);
  }
  return e4m3x2_rn_sat(__fmul_rn(fp4_div6(a, tiny), tensor_scale), __fmul_rn(fp4_div6(b, tiny), tensor_scale)) & 0x7f7fu;
}

// Value of a non-negative E4M3 byte, exactly; 0x7F is NaN.
__device__ __forceinline__ float fp4_scale_value(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return f16_lo(h);
}

// What a block's values are multiplied by: fp32(S / scale), at most the largest float (a zero stays one); 0 where
// the scale is 0 or NaN.
__device__ __forceinline__ float fp4_multiplier(uint32_t byte, float tensor_scale) {
  return byte == 0u || byte == 0x7fu ? 0.0f : fminf(__fdiv_rn(tensor_scale, fp4_scale_value(byte)), FLT_MAX);
}

// Eight values to E2M1 codes (nearest-even, saturating at 6), the first in the lowest four bits.
__device__ __forceinline__ uint32_t fp4_codes(const float (&v)[8]) {
  uint32_t r;
  asm("{ .reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d}; }"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight E2M1 codes as pairs of F16 values, the first in the low half of r[0].
__device__ __forceinline__ void fp4_values(uint32_t codes, uint32_t (&r)[4]) {
  asm("{ .reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(codes));
}

// What a product's sums are multiplied by: (1 / Sa) (1 / Sb), in two steps where that is too small or too large to be one number:
// as an infinity it would make a NaN of a sum of 0.  The larger factor comes first: where the product overflows both are above 1,
// so the first step overflows only where the result does; where it is too small, what the first step loses the second would too.
struct Fp4Factor {
  float first, then;
  __device__ __forceinline__ Fp4Factor() {}
  __device__ __forceinline__ Fp4Factor(float a_amax, float b_amax) {
    const float ra = __frcp_rn(fp4_tensor_scale(a_amax)), rb = __frcp_rn(fp4_tensor_scale(b_amax)), both = __fmul_rn(ra, rb);
    const bool one = !(both < 0x1p-100f) && !(both > FLT_MAX);  // a NaN is one number
    first = one ? both : fmaxf(ra, rb);
    then = one ? 1.0f : fminf(ra, rb);
  }
  template <int N>
  __device__ __forceinline__ void apply(float (&v)[N]) const {
    if constexpr (N == 1) {
      v[0] = __fmul_rn(v[0], first);
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 2) mul2_rn(v[k], v[k + 1], first, first, v[k], v[k + 1]);
    }
    if (then == 1.0f) return;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __fmul_rn(v[k], then);
  }
};

// Where entry (r, b) of a scale grid with `tile_cols` tiles of 128 x 4 along a row lies.
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t b, int64_t tile_cols) {
  return ((r >> 7) * tile_cols + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

}  // namespace mxfp8
