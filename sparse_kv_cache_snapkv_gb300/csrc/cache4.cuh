// The 4-bit row format (include/rkv.h): e2m1 codes in blocks of 16 with a 5-exponent, 3-mantissa-bit
// scale, and the conversions that the append and the decode share.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "tensor_core.cuh"

namespace rkv {

constexpr uint32_t kMaxScaleByte = 226;     // 10240; six times it still fits fp16
constexpr float kMaxCodeValue = 61440.0f;   // 6 * 10240

// A scale byte as an fp16 number: the format is the upper half of fp16 without its sign.
__device__ __forceinline__ __half scale_half(uint32_t b) {
  return __ushort_as_half((unsigned short)(b << 7));
}
__device__ __forceinline__ float scale_float(uint32_t b) { return __half2float(scale_half(b)); }

// a / b by an approximate reciprocal r of b: the first product's quotient corrected once by its exact
// remainder. A quotient that is itself a number of few bits comes out exactly (and a zero keeps its
// sign); any other is within 2^-22, relatively.
__device__ __forceinline__ float corrected_quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(-fmaf(q, b, -a), r, q);
}

// max|x| / 6 rounded to the nearest scale, ties to even, as its byte. amax is a bf16 number in
// [0, 61440]: 8 significant bits against the 5 of a midpoint between scales, so a quotient that is
// no midpoint is at least 2^-12 away from one, relatively, and one that is comes out exactly.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const float x = corrected_quotient(amax, 6.0f, 1.0f / 6.0f);
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

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// NaN -> +0, values beyond +-61440 clipped to it, on a packed pair.
__device__ __forceinline__ uint32_t sane_pair(uint32_t w) {
  const __nv_bfloat162 lim = __float2bfloat162_rn(kMaxCodeValue);
  const __nv_bfloat162 nlim = __float2bfloat162_rn(-kMaxCodeValue);
  __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w);
  w &= __heq2_mask(x, x);
  x = __hmax2(__hmin2(*reinterpret_cast<const __nv_bfloat162*>(&w), lim), nlim);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// 16 bf16 values (8 words) -> 8 bytes of codes and the scale byte. x / scale decides between two codes
// exactly: a tie is a quotient of few bits, and any other is at least 2^-8 from one (8 bits of x
// against the 7 of a code midpoint times a scale).
__device__ __forceinline__ uint2 quantise16(const uint32_t (&in)[8], uint32_t* sb) {
  uint32_t w[8], mx = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = in[i];
    mx = __vmaxu2(mx, in[i] & 0x7fff7fffu);  // magnitudes of bf16 numbers order as integers
  }
  mx = max(mx >> 16, mx & 0xffffu);
  if (mx > 0x4770u) {  // beyond 61440, infinite or NaN
    __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = sane_pair(w[i]);
      m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
    }
    mx = __float_as_uint(fmaxf(__low2float(m), __high2float(m))) >> 16;
  }
  const uint32_t b = scale_byte(__uint_as_float(mx << 16));
  const float s = scale_float(b);
  const float r = b ? rcp_approx(s) : 0.0f;
  const uint64_t s2 = pack2(s, s), r2 = pack2(r, r), m2 = pack2(-r, -r);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // corrected_quotient on pairs
    const uint64_t x = pack2(bf16_lo(w[i]), bf16_hi(w[i]));
    const uint64_t n = pack2(__uint_as_float((w[i] << 16) ^ 0x80000000u),
                             __uint_as_float((w[i] & 0xffff0000u) ^ 0x80000000u));
    const uint64_t q = mul2(x, r2);
    const float2 y = unpack2(fma2(fma2(q, s2, n), m2, q));
    c[i] = codes_of(y.x, y.y);
  }
  *sb = b;
  return make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24),
                    c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
}

// The bf16 values (8 words) that a block of codes stands for.
__device__ __forceinline__ void values16(uint2 codes, uint32_t sb, uint32_t (&out)[8]) {
  uint32_t h[2][4];
  codes_to_half2(codes.x, h[0]);
  codes_to_half2(codes.y, h[1]);
  const __half2 s = __half2half2(scale_half(sb));
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // exact in fp16, and in bf16
    const float2 f = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&h[i >> 2][i & 3]), s));
    out[i] = pack_bf16x2(f.x, f.y);
  }
}

}  // namespace rkv
