// Device functions of the FP4 rows: E2M1 codes with one E4M3 scale per block
// of 32 values, both ways (the cache write and the exact dequantisation).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace csa2 {

// Non-negative E4M3 value of byte c (0..126).
__device__ __forceinline__ float e4m3_pos(uint32_t c) {
  const uint32_t e = c >> 3, m = c & 7u;
  return e == 0 ? (float)m * 0.001953125f : __int_as_float((int)(((e + 120u) << 23) | (m << 20)));
}

__device__ __forceinline__ uint32_t e4m3_scale_for(float amax) {
  if (amax >= 6.0f * 448.0f) return 0x7Eu;
  // a first guess from amax / 6 (approximate), then the exact largest c with 6 v(c) <= amax
  const float y = amax * (1.0f / 6.0f);
  int c;
  if (y < 0.015625f) {   // below the smallest normal 2^-6: v = m 2^-9
    c = (int)(y * 512.0f);
  } else {
    const uint32_t bits = __float_as_uint(y);
    c = (int)((((bits >> 23) - 120u) << 3) | ((bits >> 20) & 7u));
  }
  c = c < 0 ? 0 : (c > 126 ? 126 : c);
  while (c < 126 && 6.0f * e4m3_pos((uint32_t)c + 1) <= amax) ++c;
  while (c > 0 && 6.0f * e4m3_pos((uint32_t)c) > amax) --c;
  if (c == 126) return 126u;
  const float mid2 = 3.0f * (e4m3_pos((uint32_t)c) + e4m3_pos((uint32_t)c + 1));   // 6 * midpoint, exact
  if (amax > mid2) return (uint32_t)c + 1;
  if (amax < mid2) return (uint32_t)c;
  return (c & 1) ? (uint32_t)c + 1 : (uint32_t)c;
}

// x / s, correctly rounded except within 2^-24 (relative) of a rounding
// boundary between two floats; exact whenever the quotient is representable.
__device__ __forceinline__ float quot(float x, float s, float r) {
  const float q0 = x * r;
  return fmaf(fmaf(-q0, s, x), r, q0);
}

// fp32 input only: a quotient on an E2M1 midpoint is moved one ulp toward
// the side of the exact value (the residual x - q s is exact there).
__device__ __forceinline__ float off_midpoint(float q, float x, float s) {
  const float a = fabsf(q);
  const bool mid = a == 0.25f || a == 0.75f || a == 1.25f || a == 1.75f || a == 2.5f || a == 3.5f || a == 5.0f;
  if (!mid) return q;
  const float res = fmaf(-q, s, x);
  return res > 0.f ? nextafterf(q, INFINITY) : (res < 0.f ? nextafterf(q, -INFINITY) : q);
}

// Eight E2M1 codes in one word, element k in nibble k (the conversion puts
// its first operand in the high nibble); magnitude-zero codes lose their sign.
__device__ __forceinline__ uint32_t e2m1x8(const float* y) {
  uint32_t w;
  asm("{ .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3}; }"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  const uint32_t m = w & 0x77777777u;
  const uint32_t nz = (m + 0x77777777u) & 0x88888888u;   // bit 3 of a nibble: its magnitude is not 0
  return w & (0x77777777u | nz);
}

// Two E2M1 codes (low nibble = first element) -> f16x2, exactly (every E2M1
// value is an f16 value).
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(byte));
  return r;
}
// One E4M3 byte -> the f16x2 pair (s, s), exactly (E4M3 spans 2^-9..448).
__device__ __forceinline__ uint32_t e4m3_to_f16x2_pair(uint32_t byte) {
  uint32_t r;
  const uint16_t two = (uint16_t)(byte | (byte << 8));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
  return r;
}
// Four packed codes (8 elements) times their block scale -> 4 bf16x2 words.
// The f16 product is exact (at most 6 significant bits, between 2^-10 and
// 2688), and so is its bf16 copy.
__device__ __forceinline__ void dequant8(uint32_t codes, uint32_t scale_byte, uint32_t (&out)[4]) {
  const __half2 s2 = __halves2half2(__ushort_as_half((uint16_t)(e4m3_to_f16x2_pair(scale_byte) & 0xFFFFu)),
                                    __ushort_as_half((uint16_t)(e4m3_to_f16x2_pair(scale_byte) & 0xFFFFu)));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t h = e2m1x2_to_f16x2((codes >> (8 * e)) & 0xFFu);
    __half2 v = *reinterpret_cast<const __half2*>(&h);
    v = __hmul2(v, s2);
    const float2 f = __half22float2(v);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    out[e] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

}  // namespace csa2
