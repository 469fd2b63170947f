// The 4-bit KV cache: what its kernels share.
//
// A cache holds, for every (sequence, KV head, slot), a K and a V row of dh
// E2M1 codes (dh / 2 bytes, element 2j in the low nibble of byte j) and dh / 16
// E4M3 block scales; an element is code * scale * tensor scale.  code * scale
// has at most 2 + 4 significant bits and lies in [2^-10, 2688], so it is exact
// in f16 (and bf16): the tensor-core kernels dequantise without rounding and
// put the tensor scales into the scores and the output.
#pragma once

#include <cuda_fp16.h>

#include "fp4.cuh"
#include "ops.h"
#include "vec.cuh"

namespace ps {

// Four f16 pairs (elements 0,1 / 2,3 / 4,5 / 6,7) of the eight codes of w.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t* r) {
  asm("{\n\t"
      ".reg .b8 q0, q1, q2, q3;\n\t"
      "mov.b32 {q0, q1, q2, q3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, q0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, q1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, q2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, q3;\n\t"
      "}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// (s, s) in f16 of one E4M3 scale byte.  A NaN byte, which the store never
// writes but a slot that was never stored may hold, becomes 448: such slots
// are masked, and a finite value keeps 0 * v at 0.
__device__ __forceinline__ __half2 e4m3_pair(uint32_t byte) {
  const uint16_t two = static_cast<uint16_t>(byte * 0x0101u);
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return __hmin2(*reinterpret_cast<__half2*>(&h), __float2half2_rn(448.f));
}

__device__ __forceinline__ uint32_t h2_bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 h2_of(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// D += A B, m16n8k16, f16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace ps
