// Eviction from a 4-bit KV cache by accumulated attention weight.
//
//   k_kv4_select  one CTA a (sequence, KV head): the slots to keep, ascending
//   k_kv4_gather  their codes and scales into the other cache
//
// Selection: the weights as order-preserving 32-bit keys; four passes of a
// 256-bin histogram in shared memory fix, byte by byte, the key of the last
// kept slot (the threshold) and how many slots equal to it are kept, lowest
// slots first.  A last ascending pass turns the three kinds of kept slots
// (protected, above the threshold, the first equal ones) into a packed list
// with one block scan per 1024 slots.
#include <type_traits>

#include "kv4.cuh"

namespace ps {
namespace {

constexpr int kST = 1024;  // threads of a select CTA

// Larger weight -> larger key; -0 equals 0, NaN is below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kST)
k_kv4_select(const Kv4EvictArgs a, int32_t* __restrict__ idx) {
  pdl_prologue();
  __shared__ int hist[256];
  __shared__ uint32_t scan[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int bh = blockIdx.x, b = bh / a.Hkv, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int n = min(max(a.len != nullptr ? a.len[b] : a.Ncache, 0), a.Ncache);
  const float* w = a.w + (long)bh * a.Ncache;
  const int32_t* kpos = a.kpos != nullptr ? a.kpos + (long)bh * a.Ncache : nullptr;
  if (bh % a.Hkv == 0 && tid == 0) a.len_dst[b] = min(n, a.keep);
  const bool all = n <= a.keep;
  const int lo = a.sink, hi = n - a.recent;  // candidates [lo, hi); the rest is protected
  uint32_t prefix = 0;
  int need = a.keep - a.sink - a.recent;     // kept candidates; 0 <= need < hi - lo
  if (!all) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kST) {
        const uint32_t k = weight_key(w[i]);
        if (shift == 24 || ((k ^ prefix) >> (shift + 8)) == 0)
          atomicAdd(&hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // lane l holds bins 255 - 8 l - (0..7), from the top down
        int c[8], sum = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          c[q] = hist[255 - 8 * lane - q];
          sum += c[q];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        int before = incl - sum;
        // the bin where the running count passes `need`
        if (before <= need && need < incl) {
          int q = 0;
          while (before + c[q] <= need) before += c[q++];
          s_prefix = prefix | ((uint32_t)(255 - 8 * lane - q) << shift);
          s_need = need - before;
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }
  // Kept: protected slots, keys above prefix, and the first `need` equal ones.
  const int kept_n = all ? n : a.keep;
  int32_t* out = idx + (long)bh * a.keep;
  float* w_dst = a.w_dst + (long)bh * a.Ndst;
  int32_t* kpos_dst = a.kpos_dst != nullptr ? a.kpos_dst + (long)bh * a.Ndst : nullptr;
  int done_gt = 0, done_eq = 0;
  for (int i0 = 0; i0 < n; i0 += kST) {
    const int i = i0 + tid;
    bool gt = false, eq = false;
    if (i < n) {
      if (all || i < lo || i >= hi) {
        gt = true;
      } else {
        const uint32_t k = weight_key(w[i]);
        gt = k > prefix;
        eq = k == prefix;
      }
    }
    // exclusive prefix of (gt, eq) counts, packed in one word (each <= 1024)
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    const uint32_t below = (1u << lane) - 1u;
    if (lane == 0) scan[warp] = (uint32_t)__popc(bg) | ((uint32_t)__popc(be) << 16);
    __syncthreads();
    const uint32_t mine = scan[lane];
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t before = __shfl_sync(0xffffffffu, incl - mine, warp);
    const uint32_t total = __shfl_sync(0xffffffffu, incl, 31);
    const int g = done_gt + (int)(before & 0xffffu) + __popc(bg & below);
    const int e = done_eq + (int)(before >> 16) + __popc(be & below);
    if (gt || (eq && e < need)) {
      const int j = g + min(e, need);
      if (j < kept_n) {
        out[j] = i;
        w_dst[j] = w[i];
        if (kpos_dst != nullptr) kpos_dst[j] = kpos != nullptr ? kpos[i] : i;
      }
    }
    done_gt += (int)(total & 0xffffu);
    done_eq += (int)(total >> 16);
    __syncthreads();
  }
}

// A thread takes one 16-byte piece of the codes of kRowsEach kept rows, all
// loads before the first store, so that enough bytes are in flight at scattered
// addresses; a row's first K and first V thread move its scales too.
constexpr int kRowsEach = 4;

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
  cudaError_t e = launch_pdl(k_kv4_select, dim3(a.B * a.Hkv), dim3(kST), 0, s, a, idx);
  if (e != cudaSuccess) return e;
  switch (a.dh) {
    case 64: return launch_gather<64>(a, idx, s);
    case 128: return launch_gather<128>(a, idx, s);
    case 256: return launch_gather<256>(a, idx, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ps
