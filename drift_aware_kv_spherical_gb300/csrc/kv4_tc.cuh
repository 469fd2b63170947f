// What the tcgen05 kernels of the 4-bit KV cache share: 128-row operands in the
// 128-byte-swizzled layout, rows of the cache, query rows.
#pragma once

#include "kv4.cuh"
#include "tc.cuh"

namespace ps {

// Byte offset of 16-byte chunk c (of DH / 8) of row r in an operand.
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return (uint32_t)(c >> 3) * 16384u + (uint32_t)r * 128u + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}

// One lane of a converged warp.  The MMAs below are issued under this and not
// under `lane == 0`: the operands of tcgen05.mma live in uniform registers, and
// under a thread-indexed branch each instruction took 120 clocks to issue
// (measured; 64 elected, the rate of the tensor cores at this size).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The positions that token `tok` sees.  Two loads: `span` may start at any i32.
__device__ __forceinline__ int2 row_span(const Kv4AttnArgs& a, long tok) {
  return make_int2(__ldg(a.span + 2 * tok), __ldg(a.span + 2 * tok + 1));
}

// Codes and scales of one slot's row (K or V).
template <int DH>
struct RawRow {
  uint4 c[DH / 32];
  uint2 s;
};
template <int DH>
__device__ __forceinline__ void load_row(const uint8_t* codes, const uint8_t* scales, long slot,
                                         RawRow<DH>& o) {
  const uint4* p = reinterpret_cast<const uint4*>(codes + slot * (DH / 2));
#pragma unroll
  for (int i = 0; i < DH / 32; ++i) o.c[i] = __ldg(p + i);
  if constexpr (DH == 128) {
    o.s = __ldg(reinterpret_cast<const uint2*>(scales + slot * 8));
  } else {
    o.s.x = __ldg(reinterpret_cast<const uint32_t*>(scales + slot * 4));
    o.s.y = 0;
  }
}
// 32 query rows of a warp into their place in an operand, as they are (bf16):
// cp.async in whole rows.  `src` is the lane's own row, null past the last one:
// zeros (never stored, but a vote of the warp must not hang on what was there).
template <int DH>
__device__ __forceinline__ void fetch_q(const void* any, const __nv_bfloat16* src, uint32_t qs,
                                        int r) {
  constexpr int LN = DH / 8, RP = 32 / LN;  // lanes a row, rows a pass
  const int lane = threadIdx.x & 31, sub = lane % LN;
#pragma unroll
  for (int i = 0; i < 32 / RP; ++i) {
    const int rr = i * RP + lane / LN;
    const unsigned long long from =
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), rr);
    const void* at = from != 0 ? reinterpret_cast<const void*>(from + sub * 16) : any;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(qs + sw128(r + rr, sub)),
                 "l"(at), "r"(from != 0 ? 16 : 0)
                 : "memory");
  }
}

// tanh_small of C products, two at a time: s[c] -> tanh(f s[c]).
template <int C>
__device__ __forceinline__ void tanh_series(float* s, float f) {
  const uint64_t ff = f2_pack(f, f), c0 = f2_pack(kTanh0, kTanh0), c1 = f2_pack(kTanh1, kTanh1),
                 c2 = f2_pack(kTanh2, kTanh2);
#pragma unroll
  for (int c = 0; c < C; c += 2) {
    const uint64_t y = f2_mul(f2_pack(s[c], s[c + 1]), ff), z = f2_mul(y, y);
    const uint64_t q = f2_mul(z, f2_fma(z, f2_fma(z, c2, c1), c0));
    f2_unpack(f2_fma(y, q, y), s[c], s[c + 1]);
  }
}

}  // namespace ps
