// floor(n / d) of a row or warp index by a divisor that the host knows, without a
// division: n r >> s with r = ceil(2^s / d), exact while the excess n (r d - 2^s)
// stays below 2^s and the product below 2^64.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PS_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PS_HOST_DEVICE inline
#endif

namespace ps {

// Every n < 2^31: s = 32 + c with 2^(c-1) < d <= 2^c.  r <= 2^33, and the excess is
// below n 2^c.
struct Quotient {
  uint64_t r;
  int c;

  PS_HOST_DEVICE uint32_t of(uint32_t n) const { return (uint32_t)((n * r) >> 32) >> c; }
};
inline Quotient quotient(uint32_t d) {
  int c = 0;
  while ((1ull << c) < d) ++c;
  return {((1ull << (32 + c)) + d - 1) / d, c};
}

// n < 2^26 and d <= 2^12: s = 38, one shift less (a call of k_kv4_weight_tc on 2048
// rows x 32 heads 87 us, 91 by the other).
struct RowQuotient {
  uint64_t r;

  PS_HOST_DEVICE uint32_t of(uint32_t n) const { return (uint32_t)((n * r) >> 38); }
};
inline RowQuotient row_quotient(uint32_t d) { return {((1ull << 38) + d - 1) / d}; }

}  // namespace ps
