// Eviction from a 4-bit KV cache by accumulated attention weight.
//
//   k_kv4_select  one CTA a (sequence, KV head): the slots to keep, ascending
//   k_kv4_gather  their codes and scales into the other cache
//
// Selection: the weights as order-preserving 32-bit keys.  A histogram of the
// top 11 bits (sign, exponent, two bits of mantissa: few lanes of a warp meet in
// a bin) gives the bin of the first dropped key, the threshold; another of the
// next 11 bits follows inside that bin, and of the last 10 inside that, until a
// bin holds few enough keys to be ranked against one another.
// A last ascending pass turns the three kinds of kept slots (protected, above
// the threshold, the first equal ones) into a packed list.  Up to kMaxPer weights
// a thread stay in registers; a longer row is read again by each pass (2048 slots
// 9.5 us an eviction and read-back, 10.8 reading again and 13.6 with room for
// 8192; 8192 slots x 256 rows 189 and 193).
//
// What bounds them: the selection its block-wide steps, 25 us for 256 rows of
// 8192 slots and 7 for 4 of 2048; the gather memory, at scattered addresses:
// 256 rows x 4096 kept slots (302 MB) 52 us, 5.9 TB/s, 87 % of a copy's rate.
#include <type_traits>

#include "kv4.cuh"

namespace ps {
namespace {

constexpr int kST = 512;     // threads of a select CTA: 256 rows are then one round of CTAs
constexpr int kBins = 2048;  // of the histogram
constexpr int kList = 64;    // keys that are ranked against one another

// Larger weight -> larger key; -0 equals 0, NaN is below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kMaxPer = 16;  // weights a thread in registers

// PER: weights a thread (the row has at most PER * kST slots); 0: read every time.
template <int PER>
__global__ void __launch_bounds__(kST, 2)
k_kv4_select(const __grid_constant__ Kv4EvictArgs a, int32_t* __restrict__ idx) {
  constexpr int kRow = PER > 0 ? PER : 1;
  pdl_prologue();
  constexpr int kWarps = kST / 32;
  __shared__ uint32_t cnt[kRow][kWarps], total[kRow];
  __shared__ int hist[kBins];
  __shared__ uint32_t list[kList];
  __shared__ int wsum[kST / 32], s_n, s_need, s_count;
  __shared__ uint32_t s_at;
  const int bh = blockIdx.x, b = bh / a.Hkv, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int n = min(max(a.len != nullptr ? a.len[b] : a.Ncache, 0), a.Ncache);
  const float* w = a.w + (long)bh * a.Ncache;
  const int32_t* kpos = a.kpos != nullptr ? a.kpos + (long)bh * a.Ncache : nullptr;
  if (bh % a.Hkv == 0 && tid == 0) a.len_dst[b] = min(n, a.keep);
  const bool all = n <= a.keep;
  const int lo = a.sink, hi = n - a.recent;  // candidates [lo, hi); the rest is protected
  float wv[kRow];
  if constexpr (PER > 0) {
#pragma unroll
    for (int q = 0; q < kRow; ++q) {
      const int i = q * kST + tid;
      wv[q] = i < n ? w[i] : 0.f;
    }
  }
  auto each = [&](auto&& f) {  // every candidate's key
    if constexpr (PER > 0) {
#pragma unroll
      for (int q = 0; q < kRow; ++q) {
        const int i = q * kST + tid;
        if (i >= lo && i < hi) f(weight_key(wv[q]));
      }
    } else {
      for (int i = lo + tid; i < hi; i += kST) f(weight_key(w[i]));
    }
  };
  // keys above `at` are kept; of the keys equal to it, the first `need`
  int need = a.keep - a.sink - a.recent;  // of the candidates; 0 <= need < hi - lo
  uint32_t at = 0;
  if (!all) {
    for (int shift = 21;; shift = shift == 21 ? 10 : 0) {
      const uint32_t top = shift == 21 ? 0u : ~0u << (shift == 10 ? 21 : 10);  // bits settled
#pragma unroll
      for (int q = 0; q < kBins / kST; ++q) hist[q * kST + tid] = 0;
      if (tid == 0) s_n = 0;
      __syncthreads();
      each([&](uint32_t k) {
        if (((k ^ at) & top) == 0) atomicAdd(&hist[(k >> shift) & (shift == 0 ? 1023u : 2047u)], 1);
      });
      __syncthreads();
      // thread t holds kBins / kST neighbouring bins, from the top down
      constexpr int kEach = kBins / kST;
      const int bin = kBins - 1 - kEach * tid;
      int c[kEach], sum = 0;
#pragma unroll
      for (int q = 0; q < kEach; ++q) {
        c[q] = hist[bin - q];
        sum += c[q];
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) wsum[warp] = incl;
      __syncthreads();
      int before = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0) + incl - sum;
#pragma unroll
      for (int q = 0; q < kEach; ++q) {
        if (before <= need && need < before + c[q]) {  // one thread's one bin
          s_at = at | ((uint32_t)(bin - q) << shift);
          s_need = need - before;
          s_count = c[q];
        }
        before += c[q];
      }
      __syncthreads();
      at = s_at;
      need = s_need;
      const int count = s_count;
      if (count <= kList || shift == 0) {
        if (shift == 0) break;  // all bits settled: `at` is the threshold
        const uint32_t all_top = ~0u << shift;
        each([&](uint32_t k) {
          if (((k ^ at) & all_top) == 0) list[atomicAdd(&s_n, 1)] = k;
        });
        __syncthreads();
        for (int j = tid; j < count; j += kST) {
          const uint32_t k = list[j];
          int more = 0, same = 0;
          for (int i = 0; i < count; ++i) {
            const uint32_t o = list[i];
            more += o > k;
            same += o == k;
          }
          if (more <= need && need < more + same) {  // equal keys write the same
            s_at = k;
            s_need = need - more;
          }
        }
        __syncthreads();
        at = s_at;
        need = s_need;
        break;
      }
    }
  }
  // Kept: protected slots, keys above `at`, and the first `need` equal to it.
  const int kept_n = all ? n : a.keep;
  if (a.shift_dst != nullptr) {  // the slots behind them: the positions that come next
    const int shift = (a.shift != nullptr ? a.shift[b] : 0) + n - kept_n;
    if (bh % a.Hkv == 0 && tid == 0) a.shift_dst[b] = shift;
    for (int j = kept_n + tid; j < a.Ndst; j += kST) {
      a.w_dst[(long)bh * a.Ndst + j] = 0.f;
      a.kpos_dst[(long)bh * a.Ndst + j] = j + shift;
    }
  }
  int32_t* out = idx + (long)bh * a.keep;
  float* w_dst = a.w_dst + (long)bh * a.Ndst;
  int32_t* kpos_dst = a.kpos_dst != nullptr ? a.kpos_dst + (long)bh * a.Ndst : nullptr;
  const uint32_t below = (1u << lane) - 1u;
  auto kind = [&](int i, uint32_t k, bool* gt, bool* eq) {
    *gt = *eq = false;
    if (i >= n) return;
    if (all || i < lo || i >= hi) {
      *gt = true;
    } else {
      *gt = k > at;
      *eq = k == at;
    }
  };
  auto put = [&](int i, float wi, int pi, bool gt, bool eq, int g, int e) {
    if (!(gt || (eq && e < need))) return;
    const int j = g + min(e, need);
    if (j >= kept_n) return;
    out[j] = i;
    w_dst[j] = wi;
    if (kpos_dst != nullptr) kpos_dst[j] = pi;
  };
  // (gt, eq) counts of kST slots' warps, packed in one word (each <= kST), and
  // their exclusive prefixes
  if constexpr (PER > 0) {
    int pv[kRow];
#pragma unroll
    for (int q = 0; q < kRow; ++q) {
      const int i = q * kST + tid;
      pv[q] = kpos != nullptr && i < n ? kpos[i] : i;
    }
#pragma unroll
    for (int q = 0; q < kRow; ++q) {
      bool gt, eq;
      kind(q * kST + tid, weight_key(wv[q]), &gt, &eq);
      const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
      if (lane == 0) cnt[q][warp] = (uint32_t)__popc(bg) | ((uint32_t)__popc(be) << 16);
    }
    __syncthreads();
    static_assert(kRow <= kWarps && kWarps <= 32, "a warp scans a row of counts");
    if (warp < kRow) {
      const uint32_t mine = lane < kWarps ? cnt[warp][lane] : 0u;
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane < kWarps) cnt[warp][lane] = incl - mine;
      if (lane == 31) total[warp] = incl;
    }
    __syncthreads();
    int g0 = 0, e0 = 0;
#pragma unroll
    for (int q = 0; q < kRow; ++q) {
      const uint32_t before = cnt[q][warp];
      bool gt, eq;
      kind(q * kST + tid, weight_key(wv[q]), &gt, &eq);
      const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
      put(q * kST + tid, wv[q], pv[q], gt, eq, g0 + (int)(before & 0xffffu) + __popc(bg & below),
          e0 + (int)(before >> 16) + __popc(be & below));
      g0 += (int)(total[q] & 0xffffu);
      e0 += (int)(total[q] >> 16);
    }
  } else {
    int g0 = 0, e0 = 0;
    for (int i0 = 0; i0 < n; i0 += kST) {
      const int i = i0 + tid;
      bool gt, eq;
      const float wi = i < n ? w[i] : 0.f;
      const int pi = kpos != nullptr && i < n ? kpos[i] : i;
      kind(i, weight_key(wi), &gt, &eq);
      const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
      if (lane == 0) cnt[0][warp] = (uint32_t)__popc(bg) | ((uint32_t)__popc(be) << 16);
      __syncthreads();
      const uint32_t mine = lane < kWarps ? cnt[0][lane] : 0u;
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t before = __shfl_sync(0xffffffffu, incl - mine, warp);
      const uint32_t sum = __shfl_sync(0xffffffffu, incl, 31);
      put(i, wi, pi, gt, eq, g0 + (int)(before & 0xffffu) + __popc(bg & below),
          e0 + (int)(before >> 16) + __popc(be & below));
      g0 += (int)(sum & 0xffffu);
      e0 += (int)(sum >> 16);
      __syncthreads();
    }
  }
}

// A thread takes one 16-byte piece of the codes of kRowsEach kept rows, all
// loads before the first store, so that enough bytes are in flight at scattered
// addresses (one row a thread 197 us where two take 189, four 190); a row's first
// K and first V thread move its scales too.
constexpr int kRowsEach = 2;

template <int DH>
__global__ void __launch_bounds__(256)
k_kv4_gather(const __grid_constant__ Kv4EvictArgs a, const int32_t* __restrict__ idx) {
  constexpr int kHalf = DH / 32, kPieces = 2 * kHalf;  // of K, of K and V
  constexpr int kRows = 256 / kPieces;                 // rows a pass of the CTA
  using Scale = std::conditional_t<DH == 64, uint32_t, std::conditional_t<DH == 128, uint2, uint4>>;
  pdl_prologue();
  const int bh = blockIdx.y, b = bh / a.Hkv;
  const int n = min(max(a.len != nullptr ? a.len[b] : a.Ncache, 0), a.Ncache);
  const int kept = min(n, a.keep);
  const int p = threadIdx.x % kPieces, q = p % kHalf;
  const bool is_v = p >= kHalf;
  const int j0 = blockIdx.x * (kRows * kRowsEach) + threadIdx.x / kPieces;
  const uint4* c = reinterpret_cast<const uint4*>(is_v ? a.vcode : a.kcode);
  uint4* cd = reinterpret_cast<uint4*>(is_v ? a.vcode_dst : a.kcode_dst);
  const Scale* sc = reinterpret_cast<const Scale*>(is_v ? a.vscale : a.kscale);
  Scale* sd = reinterpret_cast<Scale*>(is_v ? a.vscale_dst : a.kscale_dst);
  long src[kRowsEach];
#pragma unroll
  for (int i = 0; i < kRowsEach; ++i) {
    const int j = j0 + i * kRows;
    src[i] = j < kept ? (long)bh * a.Ncache + idx[(long)bh * a.keep + j] : -1;
  }
  uint4 v[kRowsEach];
  Scale s[kRowsEach];
#pragma unroll
  for (int i = 0; i < kRowsEach; ++i) {
    if (src[i] < 0) continue;
    v[i] = __ldcs(c + src[i] * kHalf + q);
    if (q == 0) s[i] = sc[src[i]];
  }
#pragma unroll
  for (int i = 0; i < kRowsEach; ++i) {
    if (src[i] < 0) continue;
    const long dst = (long)bh * a.Ndst + j0 + i * kRows;
    cd[dst * kHalf + q] = v[i];
    if (q == 0) sd[dst] = s[i];
  }
}

template <int DH>
cudaError_t launch_gather(const Kv4EvictArgs& a, const int32_t* idx, cudaStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.keep, 256 / (DH / 16) * kRowsEach), a.B * a.Hkv);
  return launch_pdl(k_kv4_gather<DH>, grid, dim3(256), 0, s, a, idx);
}

}  // namespace

size_t kv4_evict_ws(int B, int Hkv, int keep) {
  Carver c(nullptr);
  c.take<int32_t>((size_t)B * Hkv * keep);
  return c.bytes();
}

cudaError_t kv4_evict_run(const Kv4EvictArgs& a, cudaStream_t s) {
  Carver c(a.ws);
  int32_t* idx = c.take<int32_t>((size_t)a.B * a.Hkv * a.keep);
  const int per = ceil_div(a.Ncache, kST);
  auto select = per <= 4 ? k_kv4_select<4>
                : per <= kMaxPer ? k_kv4_select<kMaxPer> : k_kv4_select<0>;
  cudaError_t e = launch_pdl(select, dim3(a.B * a.Hkv), dim3(kST), 0, s, a, idx);
  if (e != cudaSuccess) return e;
  switch (a.dh) {
    case 64: return launch_gather<64>(a, idx, s);
    case 128: return launch_gather<128>(a, idx, s);
    case 256: return launch_gather<256>(a, idx, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ps
