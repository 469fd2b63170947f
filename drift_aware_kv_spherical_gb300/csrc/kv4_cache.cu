// Rows into and out of the 4-bit KV cache.
//
//   k_kv4_store  K and V rows -> E2M1 codes and E4M3 block scales
//   k_kv4_load   the reverse
//
// A lane owns one 16-element block of K and the same block of V: their scale,
// eight code bytes and 64 input bytes (bf16) need no other lane.  A warp takes
// 32 / (dh / 16) consecutive list entries of one head, so its scale bytes fill
// whole 32-byte sectors where the entries are consecutive slots, and
// consecutive warps take the heads of the same entries, whose input is
// contiguous.
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
    reinterpret_cast<float4*>(p)[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
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

// The lane's block: list entry j of sequence b, head h, block blk; false past
// the list, for rows outside [0, R) and for slots outside the cache.
struct BlockAt {
  long src, dst;  // elements into K / V; blocks into the cache
};
__device__ __forceinline__ bool block_at(const Kv4RowsArgs& a, int rpw, BlockAt* o) {
  const int bpr = a.dh / 16, lane = threadIdx.x & 31;
  const long warp = (long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int b = blockIdx.y;
  const int h = (int)(warp % a.Hkv);
  const long j = warp / a.Hkv * rpw + lane / bpr;
  const int cnt = a.cnt != nullptr ? min(a.cnt[b], a.R) : a.R;
  if (j >= cnt) return false;
  const int r = a.rows != nullptr ? a.rows[(long)b * a.R + j] : (int)j;
  if (r < 0 || r >= a.R) return false;
  const long slot = (long)r + (a.off != nullptr ? a.off[b] : 0);
  if (slot < 0 || slot >= a.Ncache) return false;
  const int blk = lane % bpr;
  o->src = ((long)b * a.R + r) * a.ld + (long)h * a.dh + blk * 16;
  o->dst = (((long)b * a.Hkv + h) * a.Ncache + slot) * bpr + blk;
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
k_kv4_store(const Kv4RowsArgs a, int rpw) {
  pdl_prologue();
  BlockAt at;
  if (!block_at(a, rpw, &at)) return;
  float k[16], v[16];
  load_block(static_cast<const T*>(a.K) + at.src, k);
  load_block(static_cast<const T*>(a.V) + at.src, v);
  quant_block(k, a.kmul, __fmul_rn(6.0f, a.kmul), a.kcode + at.dst * 8, a.kscale + at.dst);
  quant_block(v, a.vmul, __fmul_rn(6.0f, a.vmul), a.vcode + at.dst * 8, a.vscale + at.dst);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
k_kv4_load(const Kv4RowsArgs a, int rpw) {
  pdl_prologue();
  BlockAt at;
  if (!block_at(a, rpw, &at)) return;
  const uint2 kc = *reinterpret_cast<const uint2*>(a.kcode + at.dst * 8);
  const uint2 vc = *reinterpret_cast<const uint2*>(a.vcode + at.dst * 8);
  const uint32_t ks = a.kscale[at.dst], vs = a.vscale[at.dst];
  float x[16];
  dequant_block(kc, ks, a.kmul, x);
  put_block(static_cast<T*>(const_cast<void*>(a.K)) + at.src, x);
  dequant_block(vc, vs, a.vmul, x);
  put_block(static_cast<T*>(const_cast<void*>(a.V)) + at.src, x);
}

}  // namespace

cudaError_t kv4_rows_run(const Kv4RowsArgs& a, bool load, cudaStream_t s) {
  const int rpw = 32 / (a.dh / 16);
  const long warps = (long)ceil_div(a.R, rpw) * a.Hkv;
  const dim3 grid((unsigned)ceil_div(warps, kThreads / 32), a.B);
  if (a.dtype == PS_F32)
    return launch_pdl(load ? k_kv4_load<float> : k_kv4_store<float>, grid, kThreads, 0, s, a, rpw);
  return launch_pdl(load ? k_kv4_load<__nv_bfloat16> : k_kv4_store<__nv_bfloat16>, grid, kThreads,
                    0, s, a, rpw);
}

}  // namespace ps
