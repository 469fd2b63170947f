// NVFP4 conversions shared by the residual quantiser and the 4-bit KV cache: E2M1
// elements (Blackwell's cvt.rn.satfinite), one E4M3 scale per 16 of them.
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

}  // namespace ps
