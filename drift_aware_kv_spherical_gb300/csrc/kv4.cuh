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

// Two E4M3 scale bytes (low byte first) in f16.  A NaN byte, which the store
// never writes but a slot that was never stored may hold, becomes 448: such
// slots are masked, and a finite value keeps 0 * v at 0.
__device__ __forceinline__ __half2 e4m3x2_f16(uint32_t bytes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes)));
  return __hmin2(*reinterpret_cast<__half2*>(&h), __float2half2_rn(448.f));
}
// (s, s) of one scale byte.
__device__ __forceinline__ __half2 e4m3_pair(uint32_t byte) { return e4m3x2_f16(byte * 0x0101u); }

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

// Two fp32 operations an instruction: the same rate on the FMA pipe, half the
// issue slots.
__device__ __forceinline__ uint64_t f2_pack(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The smaller one, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Small capped scores: for |y| <= kTanhTop, tanh y = y (1 + z p(z)), z = y^2, p
// interpolated at the Chebyshev nodes of [0, kTanhTop^2]; relative error 4.3e-8.
constexpr float kTanhTop = 0.3f;
constexpr float kTanh0 = -0.33333286f, kTanh1 = 0.13323874f, kTanh2 = -0.051132676f;
__device__ __forceinline__ float tanh_small(float y) {
  const float z = y * y;
  return fmaf(y, z * fmaf(z, fmaf(z, kTanh2, kTanh1), kTanh0), y);
}
// 1 - 2 / (e^2y + 1) of y2 = 2 log2(e) y: absolute error 2.5e-7, of a score that
// times the cap.  Up to kCapAbs that is 1/30 of what P's 11 bits of bf16 queries
// leave; under a larger cap it would be more than a small score itself.
constexpr float kCapAbs = 64.f, kTwoLog2e = 2.f * kLog2e;
__device__ __forceinline__ float tanh_abs(float y2) {
  return fmaf(-2.f, rcp_approx(exp2_approx(y2) + 1.f), 1.f);
}
// Any y to 2^-20 of its tanh.
__device__ __forceinline__ float tanh_any(float y) {
  const float low = tanh_small(y), t = tanh_abs(y * kTwoLog2e);
  return fabsf(y) <= kTanhTop ? low : t;
}

// D += A B, m16n8k16, f16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr float kPShift = 10.f;  // log2 of the factor that P carries (times growth: < 2^16)

// Per-row constants of a tile, in shared memory.
struct alignas(16) RowPar {
  float f;       // score of a raw product: natural units
  float lse;     // k_kv4_weight; +inf past the last row
  float slope;   // distance bias
  int qpos;
  int lo, last;  // visible positions, both ends included; lo > last: none
};

__device__ __forceinline__ int kv4_len(const Kv4AttnArgs& a, int b) {
  return min(max(a.len != nullptr ? a.len[b] : a.Ncache, 0), a.Ncache);
}

// The power of two that a query row is scaled by before it is rounded to f16
// (2^14 <= max |q| * up < 2^15; 1 for a row without a finite non-zero
// maximum), and the factor that takes a product with K back to a score.  A
// negative scale turns the query's sign instead, so the factor is positive
// and row maxima may be taken of raw products.
__device__ __forceinline__ void row_scale(float mx, float scale, float* up, float* f) {
  int ex = 0;  // subnormal maxima count as 2^-127: the scale ends at 2^110 all the same
  if (mx > 0.f && mx < INFINITY) ex = min(141 - (int)(__float_as_uint(mx) >> 23), 110);
  *up = __uint_as_float((uint32_t)(127 + ex) << 23) * (scale < 0.f ? -1.f : 1.f);
  *f = fmaxf(fabsf(scale) * __uint_as_float((uint32_t)(127 - ex) << 23), FLT_MIN);
}

// lse of a row whose sum l is of 2^(x - mx + kPShift), x its log2-unit scores
// (mx = -inf: nothing but NaN was seen, or nothing at all and l == 0).
__device__ __forceinline__ float row_lse(float mx, float l) {
  return l == 0.f ? -INFINITY : ((mx == -INFINITY ? 0.f : mx - kPShift) + log2f(l)) * kLn2;
}

// Row m of a KV head as (token, query head of the group): m = t G + j.
__device__ __forceinline__ int row_token(const Kv4AttnArgs& a, int m) {
  return (int)a.by_g.of((uint32_t)m);
}

// Four elements of a finished row: O = acc / l.
template <bool F32>
__device__ __forceinline__ void kv4_finish(const Kv4AttnArgs& a, int b, int hkv, int m, int dh,
                                           int d, float4 acc, float mx, float l) {
  const int t = row_token(a, m), h = hkv * a.G + (m - t * a.G);
  const long row = ((long)b * a.T + t) * a.Hq + h;
  const float inv = l == 0.f ? 0.f : a.vmul / l;  // l == 0: nothing seen
  const float x = acc.x * inv, y = acc.y * inv, z = acc.z * inv, w = acc.w * inv;
  if constexpr (F32) {
    reinterpret_cast<float4*>(static_cast<float*>(a.O) + row * dh + d)[0] = make_float4(x, y, z, w);
  } else {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x, y), q = __floats2bfloat162_rn(z, w);
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.O) + row * dh + d)[0] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
  }
  if (d == 0 && a.lse != nullptr) a.lse[row] = row_lse(mx, l);
}

}  // namespace ps
