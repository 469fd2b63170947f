// NVFP4 arithmetic shared by the residual quantiser and the 4-bit KV cache:
// E2M1 elements (Blackwell's cvt.rn.satfinite conversions), one E4M3 scale per
// 16 of them, one fp32 tensor scale.
#pragma once

#include <cfloat>

#include "common.cuh"

namespace ps {

// Eight fp32 values -> eight E2M1 codes, element 2j in the low nibble of
// byte j.  cvt ... e2m1x2 d, a, b puts a in the high nibble, b in the low.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t out;
  asm("{\n\t"
      ".reg .b8 q0, q1, q2, q3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q3, %8, %7;\n\t"
      "mov.b32 %0, {q0, q1, q2, q3};\n\t"
      "}"
      : "=r"(out)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]),
        "f"(v[6]), "f"(v[7]));
  return out;
}

// fp32 -> E4M3 code (low byte of the x2 conversion).
__device__ __forceinline__ uint32_t e4m3_code(float x) {
  unsigned short h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(x));
  return h & 0xFFu;
}

// Exact value of a non-negative E4M3 code (bias 7, subnormal step 2^-9).
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  const uint32_t e = (c >> 3) & 15u, m = c & 7u;
  if (e == 0) return (float)m * 0.001953125f;
  return __uint_as_float(((e + 120u) << 23) | (m << 20));
}

// The codes of x[0..7] / den (four bytes, element 2j in the low nibble of
// byte j), with rinv = RN(1 / den) finite: the product path where both
// ends of its error band convert alike, else the IEEE division.
__device__ __forceinline__ uint32_t e2m1_div8(const float* x, float den, float rinv) {
  constexpr float kLo = 1.0f - 0x1p-20f, kHi = 1.0f + 0x1p-20f;
  float lo[8], hi[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = __fmul_rn(x[e], rinv);
    lo[e] = __fmul_rn(q, kLo);
    hi[e] = __fmul_rn(q, kHi);
  }
  const uint32_t a = e2m1x8(lo), b = e2m1x8(hi);
  if (a == b) return a;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __fdiv_rn(x[e], den);
  return e2m1x8(v);
}

// One 16-element block: its E4M3 scale and eight bytes of E2M1 codes.  The
// codes of r / den come from r * RN(1 / den) wherever that cannot change
// them (e2m1_div8), else from the IEEE division.
__device__ __forceinline__ void quant_block(const float* r, float S, float six_s,
                                            uint8_t* __restrict__ codes_at,
                                            uint8_t* __restrict__ scale_at) {
  float bm = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) bm = fmaxf(bm, fabsf(r[e]));
  const uint32_t sc = e4m3_code(__fdiv_rn(bm, six_s));
  const float sb = e4m3_value(sc);
  uint2 q = make_uint2(0u, 0u);
  if (sb != 0.f) {
    const float den = __fmul_rn(sb, S);
    if (den >= FLT_MIN) {
      const float rinv = __frcp_rn(den);
      q.x = e2m1_div8(r, den, rinv);
      q.y = e2m1_div8(r + 8, den, rinv);
    } else {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = __fdiv_rn(r[e], den);
      q.x = e2m1x8(v);
      q.y = e2m1x8(v + 8);
    }
  }
  *reinterpret_cast<uint2*>(codes_at) = q;
  *scale_at = (uint8_t)sc;
}

}  // namespace ps
