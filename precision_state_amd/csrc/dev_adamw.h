// dev_adamw.h - gfx950 device helpers of the AdamW plan's kernels: e4m3 moment
// codes, and IEEE square roots and quotients for values of ordinary size.
#pragma once

#include "dev_common.h"

namespace ps {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// e4m3 moments. The block's scale is the smallest power of two s >= 2^-126
// with max <= 448 s (448 = 1.75 * 2^8 is the largest e4m3 value): adding the
// mantissa bits above 1.75 carries into the exponent exactly when the
// mantissa is larger than 1.75. Scaling by a power of two is exact, so a code
// is one rounding of the moment, and the hardware conversion makes it.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void e4m3_scale(uint32_t max_bits, float& s, float& inv) {
  const int e = __builtin_elementwise_max((int)((max_bits + 0x1FFFFFu) >> 23) - 8, 1);
  s = __uint_as_float((uint32_t)e << 23);
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
}

__device__ __forceinline__ void e4m3_unpack4(uint32_t c, float* d) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  d[0] = a.x; d[1] = a.y; d[2] = b.x; d[3] = b.y;
}

__device__ __forceinline__ uint32_t e4m3_pack4(const float* y) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
}

// Codes of x / s, the power-of-two scale s in the conversion.
__device__ __forceinline__ uint32_t e4m3_pack4(const float* x, float s) {
  i16x2 c = {0, 0};
  c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[0], x[1], s, false);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[2], x[3], s, true);
  return __builtin_bit_cast(uint32_t, c);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
  x = row32_max_u32(x);
  const auto p = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return __builtin_elementwise_max((uint32_t)p[0], (uint32_t)p[1]);
}

constexpr float kMinCode = 0x1p-9f;   // smallest e4m3 value above zero

// The random 16 bits of element j (0..3) of a quad, from its 64 bits.
__device__ __forceinline__ uint32_t random16(uint64_t z, int j) { return (uint32_t)(z >> (16 * j)) & 0xFFFFu; }

// y >= 0 cut to 3 mantissa bits after adding 16 random bits below them (one
// instruction: 16 times half of a word of the quad's bits, plus y).
__device__ __forceinline__ float e4m3_cut(float y, uint64_t z, int j) {
  const uint32_t w = (uint32_t)(z >> (32 * (j >> 1)));
  uint32_t u;
  if (j & 1)
    asm("v_mad_u32_u16 %0, %1, 16, %2 op_sel:[1,0,0,0]" : "=v"(u) : "v"(w), "v"(y));
  else
    asm("v_mad_u32_u16 %0, %1, 16, %2" : "=v"(u) : "v"(w), "v"(y));
  return __uint_as_float(u & 0xFFF00000u);
}
// y in [0, 448] cut so to e4m3's values: below 2^-6 they keep the places of 2^-6,
// which adding 2^-6 lines up.
__device__ __forceinline__ float e4m3_stochastic(float y, uint64_t z, int j) {
  return y < 0x1p-6f ? e4m3_cut(y + 0x1p-6f, z, j) - 0x1p-6f : e4m3_cut(y, z, j);
}

// ---------------------------------------------------------------------------
// IEEE square root and quotient without the library's scaling steps.
// ---------------------------------------------------------------------------

// sqrt(v) for v == 0 or v >= 2^-100: one Newton step from the hardware's
// 1/sqrt(v). It is the correctly rounded root for every such fp32 value
// (checked for all of them on the GPU).
__device__ __forceinline__ float sqrt_fast(float v) {
  // the order of bits as integers is that of the values; their maximum needs no quieting
  const float y = __builtin_amdgcn_rsqf(__uint_as_float((uint32_t)__builtin_elementwise_max((int)__float_as_uint(v), 27 << 23)));
  const float s = v * y;
  return __builtin_fmaf(__builtin_fmaf(-s, s, v), 0.5f * y, s);
}

// a / d by Markstein's iterations (IBM J. Res. Dev. 34, 1990): a reciprocal
// refined once, a quotient that its remainder brings within one ulp, and the
// exact remainder of that one. These are the steps of a correctly rounded
// quotient without the scaling that keeps them in the normal range; for d in
// [2^-60, 2^60] and a == 0 or |a| in [2^-60, 2^60] none leaves it (the sign of
// a zero apart).
__device__ __forceinline__ float div_fast(float a, float d) {
  const float y0 = __builtin_amdgcn_rcpf(d);
  const float y = __builtin_fmaf(__builtin_fmaf(-d, y0, 1.0f), y0, y0);
  float q = a * y;
  q = __builtin_fmaf(__builtin_fmaf(-d, q, a), y, q);
  return __builtin_fmaf(__builtin_fmaf(-d, q, a), y, q);
}

}  // namespace ps
