// The 4-bit row format (include/rkv.h): e2m1 codes in blocks of 16 with a 5-exponent, 3-mantissa-bit
// scale, and the conversions that the append and the decode share.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace rkv {

constexpr uint32_t kMaxScaleByte = 226;     // 10240; six times it still fits fp16
constexpr float kMaxCodeValue = 61440.0f;   // 6 * 10240

// A scale byte as an fp16 number: the format is the upper half of fp16 without its sign.
__device__ __forceinline__ __half scale_half(uint32_t b) {
  return __ushort_as_half((unsigned short)(b << 7));
}
__device__ __forceinline__ float scale_float(uint32_t b) { return __half2float(scale_half(b)); }

// max|x| / 6 rounded to the nearest scale, ties to even, as its byte. amax is a bf16 number in
// [0, 61440]: 8 significant bits against the 5 of a midpoint between scales, so the one rounding
// of the fp32 division cannot move the quotient across or onto a midpoint that it does not hit
// exactly (their relative distance is at least 2^-12).
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const float x = __fdiv_rn(amax, 6.0f);
  uint32_t b;
  if (x < 6.103515625e-05f) {  // below 2^-14 the scales are multiples of 2^-17
    b = (uint32_t)__float2int_rn(x * 131072.0f);
  } else {
    const uint32_t u = __float_as_uint(x);
    b = ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112u << 3);
  }
  return min(b, kMaxScaleByte);
}

// Two numbers already divided by their scale -> a byte of codes (lo in the low half), round to
// nearest even, saturating.
__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tcvt.u32.u8 %0, c;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// The four bytes of codes in w as fp16 pairs (low half of a byte -> low half of the pair).
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// x / s for a scale s with reciprocal r (both 0 for a zero scale): the quotient of the first
// product is corrected once by its exact remainder, so a quotient that is itself a number of few
// bits (a tie between two codes) comes out exactly. Any other is at least 2^-8 away from a tie,
// relatively (8 bits of x against 7 of a tie times a scale), and the error here is below 2^-22.
__device__ __forceinline__ float over_scale(float x, float s, float r) {
  const float q = x * r;
  return fmaf(-fmaf(q, s, -x), r, q);  // (in this order a zero keeps its sign)
}

// 16 bf16 values (8 words) -> 8 bytes of codes and the scale byte.
__device__ __forceinline__ uint2 quantise16(const uint32_t (&in)[8], uint32_t* sb) {
  uint32_t w[8];
  // NaN -> +0, then the clip; on packed pairs (hequ2 masks a lane that is not equal to itself)
  const __nv_bfloat162 lim = __float2bfloat162_rn(kMaxCodeValue);
  const __nv_bfloat162 nlim = __float2bfloat162_rn(-kMaxCodeValue);
  __nv_bfloat162 mx = __float2bfloat162_rn(0.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&in[i]);
    const uint32_t ok = __heq2_mask(x, x);
    w[i] = in[i] & ok;
    x = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
    x = __hmax2(__hmin2(x, lim), nlim);
    w[i] = *reinterpret_cast<const uint32_t*>(&x);
    mx = __hmax2(mx, __habs2(x));
  }
  const float amax = fmaxf(__low2float(mx), __high2float(mx));
  const uint32_t b = scale_byte(amax);
  const float s = scale_float(b);
  const float r = b ? __frcp_rn(s) : 0.0f;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = codes_of(over_scale(bf16_lo(w[i]), s, r), over_scale(bf16_hi(w[i]), s, r));
  *sb = b;
  return make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24),
                    c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
}

// The bf16 values (8 words) that a block of codes stands for.
__device__ __forceinline__ void values16(uint2 codes, uint32_t sb, uint32_t (&out)[8]) {
  uint32_t h[8];
  uint32_t a[4], b[4];
  codes_to_half2(codes.x, a);
  codes_to_half2(codes.y, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = a[i];
    h[4 + i] = b[i];
  }
  const float s = scale_float(sb);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    out[i] = pack_bf16x2(f.x * s, f.y * s);
  }
}

}  // namespace rkv
