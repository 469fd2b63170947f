// Rows into and out of the 4-bit KV cache.
//
//   k_kv4_store  K and V rows -> E2M1 codes and E4M3 block scales
//   k_kv4_load   the reverse
//
// A lane owns one 16-element block of K and the same block of V: their scale,
// eight code bytes and 64 input bytes (bf16) need no other lane.  A warp takes
// 512 / dh consecutive list entries of one head, so its scale bytes fill whole
// 32-byte sectors where the entries are consecutive slots, and consecutive
// warps take the heads of the same entries, whose input is contiguous.
//
// What bounds them: memory, and for the store instructions close behind (issue
// 58 % busy): eight 4096-row windows of 32 heads of 128 (688 MB each way) stored
// in 130 us, 5.3 TB/s, and read back in 118, 5.8 TB/s, 86 % of a copy's rate; a
// refresh's list of a few hundred rows 5 us each, the launch.
#include "kv4.cuh"

namespace ps {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load_block(const T* p, float* x) {
  constexpr int V = Vec<T>::n;
#pragma unroll
  for (int q = 0; q < 16 / V; ++q) load16(p + q * V, x + q * V);
}

__device__ __forceinline__ void put_block(__nv_bfloat16* p, const float* x) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void put_block(float* p, const float* x) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    reinterpret_cast<float4*>(p)[q] =
        make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
}

// value = fl(fl(code * scale) * mul) of one block (the first product is exact)
__device__ __forceinline__ void dequant_block(uint2 c, uint32_t sc, float mul, float* x) {
  const __half2 s = e4m3_pair(sc);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t r[4];
    e2m1x8_f16(w == 0 ? c.x : c.y, r);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 v = __half22float2(__hmul2(h2_of(r[q]), s));
      x[8 * w + 2 * q] = __fmul_rn(v.x, mul);
      x[8 * w + 2 * q + 1] = __fmul_rn(v.y, mul);
    }
  }
}

// The codes of x[0..15] / den.  fl(x / den) by Markstein's theorem: with y =
// RN(1 / den), q = RN(x y) and the exact remainder r = x - q den, RN(q + r y) is
// the correctly rounded quotient while nothing over- or underflows.  The remainder
// is taken as q den - x, which is +0 and not -0 where it vanishes, and subtracted:
// so a quotient of -0 stays -0.  Three instructions, no branch: bf16 rows hit E2M1's
// ties exactly so often (x and den have few bits) that a fast path which detects
// them took its slow one in every warp.
__device__ __forceinline__ uint2 codes16(const float* x, float den, float y) {
  float q[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float q0 = __fmul_rn(x[e], y);
    q[e] = __fmaf_rn(-__fmaf_rn(q0, den, -x[e]), y, q0);
  }
  return make_uint2(e2m1x8(q), e2m1x8(q + 8));
}

// One block with the tensor scale S: its codes and scale.
__device__ __forceinline__ uint32_t encode_block(const float* x, float S, float six_s,
                                                 uint2* codes) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
  const uint32_t sc = e4m3_code(__fdiv_rn(m, six_s));
  const float den = __fmul_rn(e4m3_value(sc), S);
  *codes = make_uint2(0u, 0u);
  const float y = __frcp_rn(den);
  // (a block scale that saturates leaves quotients far past 6, infinite ones too)
  if (den >= 0x1p-90f && den <= 0x1p90f && m * y < 0x1p90f) {
    *codes = codes16(x, den, y);
  } else if (den > 0.f) {  // out of the theorem's range
    float q[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = __fdiv_rn(x[e], den);
    *codes = make_uint2(e2m1x8(q), e2m1x8(q + 8));
  }
  return sc;
}

// The slot of a head that holds a position, -1 if none does: positions ascend.
// (A binary search by every lane of a row: lists of 400 rows x 4 sequences x 32
// heads on 2048 slots 18 us, 12 by slots.)
__device__ __forceinline__ long slot_of(const int32_t* __restrict__ kpos, int n, long pos) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (__ldg(kpos + mid) < pos) lo = mid + 1;
    else hi = mid;
  }
  return lo < n && __ldg(kpos + lo) == pos ? lo : -1;
}

// The lane's block: list entry j of sequence b, head h, block blk; false past
// the list, for rows outside [0, R) and for slots outside the cache.
// POS: rows are named by position.
struct BlockAt {
  long src, dst;  // elements into K / V; blocks into the cache
};
template <int DH, bool POS>
__device__ __forceinline__ bool block_at(const Kv4RowsArgs& a, BlockAt* o) {
  constexpr int kBlocks = DH / 16, kRows = 32 / kBlocks;  // a row; rows a warp
  const int lane = threadIdx.x & 31;
  const uint32_t warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int b = blockIdx.y;
  const uint32_t group = a.by_hkv.of(warp);
  const int h = (int)(warp - group * a.Hkv);
  const int j = (int)group * kRows + lane / kBlocks;
  const int cnt = a.cnt != nullptr ? min(a.cnt[b], a.R) : a.R;
  if (j >= cnt) return false;
  const int r = a.rows != nullptr ? a.rows[(long)b * a.R + j] : j;
  if (r < 0 || r >= a.R) return false;
  long slot = (long)r + (a.off != nullptr ? a.off[b] : 0);
  if constexpr (POS) slot = slot_of(a.kpos + ((long)b * a.Hkv + h) * a.Ncache, a.Ncache, slot);
  if (slot < 0 || slot >= a.Ncache) return false;
  const int blk = lane % kBlocks;
  o->src = (long)b * a.b_ld + (long)r * a.ld + (long)h * DH + blk * 16;
  o->dst = (((long)b * a.Hkv + h) * a.Ncache + slot) * kBlocks + blk;
  return true;
}

template <typename T, int DH, bool POS>
__global__ void __launch_bounds__(kThreads)
k_kv4_store(const __grid_constant__ Kv4RowsArgs a) {
  pdl_prologue();
  BlockAt at;
  if (!block_at<DH, POS>(a, &at)) return;
  float k[16], v[16];
  load_block(static_cast<const T*>(a.K) + at.src, k);
  load_block(static_cast<const T*>(a.V) + at.src, v);
  uint2 kc, vc;
  const uint32_t ks = encode_block(k, a.kmul, __fmul_rn(6.0f, a.kmul), &kc);
  const uint32_t vs = encode_block(v, a.vmul, __fmul_rn(6.0f, a.vmul), &vc);
  reinterpret_cast<uint2*>(a.kcode)[at.dst] = kc;
  reinterpret_cast<uint2*>(a.vcode)[at.dst] = vc;
  a.kscale[at.dst] = (uint8_t)ks;
  a.vscale[at.dst] = (uint8_t)vs;
}

template <typename T, int DH>
__global__ void __launch_bounds__(kThreads)
k_kv4_load(const __grid_constant__ Kv4RowsArgs a) {
  pdl_prologue();
  BlockAt at;
  if (!block_at<DH, false>(a, &at)) return;
  const uint2 kc = reinterpret_cast<const uint2*>(a.kcode)[at.dst];
  const uint2 vc = reinterpret_cast<const uint2*>(a.vcode)[at.dst];
  const uint32_t ks = a.kscale[at.dst], vs = a.vscale[at.dst];
  float x[16];
  dequant_block(kc, ks, a.kmul, x);
  put_block(static_cast<T*>(const_cast<void*>(a.K)) + at.src, x);
  dequant_block(vc, vs, a.vmul, x);
  put_block(static_cast<T*>(const_cast<void*>(a.V)) + at.src, x);
}

template <typename T, int DH>
cudaError_t launch_rows(const Kv4RowsArgs& a, bool load, cudaStream_t s) {
  const long warps = (long)ceil_div(a.R, 512 / DH) * a.Hkv;
  const dim3 grid((unsigned)ceil_div(warps, kThreads / 32), a.B);
  auto kern = load ? k_kv4_load<T, DH>
              : a.kpos != nullptr ? k_kv4_store<T, DH, true> : k_kv4_store<T, DH, false>;
  return launch_pdl(kern, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t kv4_rows_run(Kv4RowsArgs a, bool load, cudaStream_t s) {
  a.by_hkv = quotient(a.Hkv);
#define PS_KV4_CASE(DH)                                              \
  if (a.dh == DH)                                                    \
    return a.dtype == PS_F32 ? launch_rows<float, DH>(a, load, s)    \
                             : launch_rows<__nv_bfloat16, DH>(a, load, s);
  PS_KV4_CASE(64)
  PS_KV4_CASE(128)
  PS_KV4_CASE(256)
#undef PS_KV4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace ps
