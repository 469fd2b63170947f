// Attention over packed sequences or cache rows: what its kernels share.
//
// The query rows of a KV head in a sequence of n tokens are its n G (token, query
// head of the group) pairs, m = t G + j.  Kernels take them in tiles; no tile spans two
// sequences.  The tiles of sequence s are numbered from first(s) = floor(q_off[s] mul
// / div) + s on, where a tile holds div / mul tokens: first(s + 1) - first(s) is never
// less than the tiles that s has, so one number names a tile without a prefix sum,
// and S numbers at most are left over.
#pragma once

#include <climits>

#include "ops.h"
#include "tc.cuh"
#include "vec.cuh"

namespace ps {

// A sequence's rows and slots, cut to the tensors.
struct AttnSeq {
  int q0, n;   // first row of Q; tokens
  int k0, m;   // first row of K and V; slots
};
__device__ __forceinline__ int attn_q_off(const AttnArgs& a, int s) {
  return min(max(__ldg(a.q_off + s), 0), a.Tq);
}
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int s) {
  AttnSeq x;
  x.q0 = attn_q_off(a, s);
  x.n = max(attn_q_off(a, s + 1) - x.q0, 0);
  x.k0 = min(max(__ldg(a.k_off + s), 0), a.Tk);
  const long end = a.k_len != nullptr ? (long)x.k0 + __ldg(a.k_len + s) : (long)__ldg(a.k_off + s + 1);
  x.m = (int)(min(max(end, (long)x.k0), (long)a.Tk) - x.k0);
  return x;
}

// The last sequence s with first(s) <= tile, for a whole warp: 32 probes at a time.
template <class First>
__device__ __forceinline__ int attn_find(int S, long tile, First first) {
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lo + (threadIdx.x & 31) * step;
    const bool below = at < lo + n && first(at) <= tile;
    // (first ascends: the probes that pass are the first ones, and one at least)
    const int pass = max(__popc(__ballot_sync(0xffffffffu, below)), 1) - 1;
    const int end = lo + n;
    lo += pass * step;
    n = min(step, end - lo);
  }
  return lo;
}

// The slots that token t (of its sequence) sees: [x, y), empty as (0, 0).
__device__ __forceinline__ int2 attn_seen(const AttnArgs& a, const AttnSeq& q, int t) {
  long lo = 0, hi = q.m;
  if (a.causal) hi = min(hi, (long)q.m - q.n + t + 1);
  if (a.span != nullptr) {
    const long r = 2 * (long)(q.q0 + t);
    lo = max(lo, (long)__ldg(a.span + r));
    hi = min(hi, (long)__ldg(a.span + r + 1));
  }
  return lo < hi ? make_int2((int)lo, (int)hi) : make_int2(0, 0);
}

// ---------------------------------------------------------------- mma.sync kernels
constexpr int kThreads = 128, kW = 4;  // threads and warps of a CTA

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_b16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// A CTA's row tile (of R rows of a KV head) and share of the slots.
struct AttnTile {
  AttnSeq seq;
  long m0;             // first row
  int s, num, hkv, split; // sequence; rows
  int lo, hi, steps;   // slots that some row sees; stages of them

  // false: no work, or another kernel's sequence.  For whole warps.
  template <int R>
  __device__ __forceinline__ bool find(const AttnArgs& a, int slots) {
    // (the heads of a row lie together in memory: CTAs side by side read them together;
    // a cluster is the shares of a tile)
    long tile;
    if (a.cluster) {
      split = blockIdx.x % a.nsplit;
      hkv = blockIdx.x / a.nsplit % a.Hkv;
      tile = blockIdx.x / a.nsplit / a.Hkv;
    } else {
      hkv = blockIdx.x % a.Hkv;
      split = blockIdx.x / a.Hkv % a.nsplit;
      tile = blockIdx.x / a.Hkv / a.nsplit;
    }
    auto first = [&](int s) {
      return a.per_seq > 0 ? (long)s * a.per_seq : (long)attn_q_off(a, s) * a.G / R + s;
    };
    s = a.per_seq > 0 ? (int)(tile / a.per_seq) : attn_find(a.S, tile, first);
    seq = attn_seq(a, s);
    m0 = (tile - first(s)) * R;
    const long rows = (long)seq.n * a.G;
    if (m0 < 0 || m0 >= rows || rows < a.least || rows > a.most) return false;
    num = (int)min(rows - m0, (long)R);
    const int t0 = (int)a.by_g.of((uint32_t)m0), t1 = (int)a.by_g.of((uint32_t)(m0 + num - 1));
    lo = INT_MAX;
    hi = 0;
    for (int t = t0 + (int)(threadIdx.x & 31); t <= t1; t += 32) {
      const int2 x = attn_seen(a, seq, t);
      if (x.x < x.y) {
        lo = min(lo, x.x);
        hi = max(hi, x.y);
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (a.nsplit > 1) {
      lo = (int)max((long)lo, (long)split * a.chunk);
      if (split + 1 < a.nsplit) hi = (int)min((long)hi, (long)(split + 1) * a.chunk);
      if (lo >= hi && !a.cluster) return false;
    }
    steps = lo < hi ? (int)(((long)hi - lo + slots - 1) / slots) : 0;
    return true;
  }
};

// Which partial sums are those of row m of sequence s and KV head hkv, row `row` of Q and head
// h: by row and head; where a kernel takes few rows of every sequence, by their numbers (a
// long prompt beside a token has rows by the thousand that are not among them).
__device__ __forceinline__ long attn_part(const AttnArgs& a, int s, int hkv, int m, int row,
                                          int h) {
  return a.per_seq > 0 ? ((long)s * a.most + m) * a.Hkv + hkv : (long)row * a.Hq + h;
}

constexpr float kAttnLog2e = 1.4426950408889634f;
constexpr float kAttnLn2 = 0.6931471805599453f;

__device__ __forceinline__ float attn_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// lse of a row whose sum l is of 2^(x - m), x its scores in log2 units.
__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kAttnLn2;
}

__device__ __forceinline__ float2 load_pair(const float* p) {
  return *reinterpret_cast<const float2*>(p);
}
__device__ __forceinline__ float2 load_pair(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}

// One row again, for a whole warp, over the slots that it sees only.  The tiles'
// products multiply what a row does not see by zero, which leaves a NaN if that is
// infinite or NaN, and fp32's low terms turn a seen infinity's score into one (0 times
// infinity): a row that did not come out finite is computed like this, its lse too.
//
// 32 slots at a time, a lane a slot for the scores, then a lane a few elements for O: a slot
// at a time it was a chain of loads and exchanges, and 1280 such rows x 32 heads of 128 on
// 16 K slots took 1486 ms, 437 so; and sums of 32 weights lose less than one weight at a time.
template <typename T>
__device__ __forceinline__ void attn_redo(const AttnArgs& a, const AttnSeq& s, int t, int h) {
  constexpr int E = 4, L = Vec<T>::n;  // pairs of elements a lane: dh <= 256; of a 16-byte load
  const int lane = threadIdx.x & 31;
  __syncwarp();  // (what other lanes stored of the row comes first)
  const int2 see = attn_seen(a, s, t);
  const T* q = static_cast<const T*>(a.Q) + (long)(s.q0 + t) * a.q_ld + (long)h * a.dh;
  const long at = (long)(h / a.G) * a.dh;
  const T* k = static_cast<const T*>(a.K) + at;
  const T* v = static_cast<const T*>(a.V) + at;
  float o[2 * E];
#pragma unroll
  for (int e = 0; e < 2 * E; ++e) o[e] = 0.f;
  const float f = a.scale * kAttnLog2e;
  float m = -INFINITY, l = 0.f;
  for (int n = see.x; n < see.y; n += 32) {
    const int num = min(see.y - n, 32);
    const T* row = k + ((long)s.k0 + n + min(lane, num - 1)) * a.k_ld;
    float sum[L];
#pragma unroll
    for (int i = 0; i < L; ++i) sum[i] = 0.f;
#pragma unroll 2
    for (int d = 0; d < a.dh; d += L) {
      float x[L], y[L];
      load16(q + d, x);
      load16(row + d, y);
#pragma unroll
      for (int i = 0; i < L; ++i) sum[i] = fmaf(x[i], y[i], sum[i]);
    }
#pragma unroll
    for (int i = L / 2; i > 0; i >>= 1)
#pragma unroll
      for (int j = 0; j < i; ++j) sum[j] += sum[j + i];
    const float x = lane < num ? sum[0] * f : -INFINITY;
    const float top = fmaxf(m, warp_max(x)), base = top == -INFINITY ? 0.f : top;
    const float c = attn_exp2(m - base), p = attn_exp2(x - base);
    l = fmaf(l, c, warp_sum(p));
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) o[e] *= c;
#pragma unroll 4
    for (int i = 0; i < num; ++i) {
      const float w = __shfl_sync(0xffffffffu, p, i);
      const T* from = v + ((long)s.k0 + n + i) * a.v_ld + 2 * lane;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (2 * lane + 64 * e < a.dh) {
          const float2 y = load_pair(from + 64 * e);
          o[2 * e] = fmaf(w, y.x, o[2 * e]);
          o[2 * e + 1] = fmaf(w, y.y, o[2 * e + 1]);
        }
    }
    m = top;
  }
  T* to = static_cast<T*>(a.O) + (long)(s.q0 + t) * a.o_ld + (long)h * a.dh + 2 * lane;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (l == 0.f) {  // no weight at all: nothing of V, infinite or not
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) o[e] = 0.f;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (2 * lane + 64 * e < a.dh) {
      Store<T>::put(to + 64 * e, o[2 * e] * inv);
      Store<T>::put(to + 64 * e + 1, o[2 * e + 1] * inv);
    }
  if (lane == 0 && a.lse != nullptr) a.lse[(long)(s.q0 + t) * a.Hq + h] = attn_lse(m, l);
}

// The same as a call: in the kernels of attn.cu it costs their loops registers otherwise (2048
// x 2048 fp32 rows x 32 heads 1878 us, 2030 with it inlined; a join of 1024 rows 7.1, 9.3).
template <typename T>
__device__ __noinline__ void attn_redo_call(const AttnArgs& a, const AttnSeq s, int t, int h) {
  attn_redo<T>(a, s, t, h);
}

// Four finished elements of a row from its sums; false where one is infinite or NaN.
template <typename T>
__device__ __forceinline__ bool attn_store4(const AttnArgs& a, int r, int h, int d, float4 x,
                                            float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float y[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
  T* to = static_cast<T*>(a.O) + (long)r * a.o_ld + (long)h * a.dh + d;
  bool fine = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float z = l == 0.f ? 0.f : y[e];
    fine = fine && fabsf(z) < INFINITY;
    Store<T>::put(to + e, z);
  }
  if (d == 0 && a.lse != nullptr) a.lse[(long)r * a.Hq + h] = attn_lse(m, l);
  return fine;
}
__device__ __forceinline__ void attn_add4(float4& x, float& l, float4 y, float ly, float c) {
  l = fmaf(ly, c, l);
  x.x = fmaf(y.x, c, x.x);
  x.y = fmaf(y.y, c, x.y);
  x.z = fmaf(y.z, c, x.z);
  x.w = fmaf(y.w, c, x.w);
}

// The sums of a CTA's warps joined and stored: acc [kW][R][DH], m and l [kW][16] in shared
// memory, written by the threads just before.  Shares of a cluster are joined here too.
// CALL: attn_redo_call.
template <typename T, int DH, int R, bool CALL>
__device__ __forceinline__ void attn_join_warps(const AttnArgs& a, const AttnTile& tile, float* acc,
                                                float* s_m, float* s_l, int* s_bad) {
  const int tid = threadIdx.x, num = tile.num;
  const bool part = a.nsplit > 1 && !a.cluster;
  if (tid == 0) *s_bad = 0;
  __syncthreads();
  const int per = a.dh / 4;
  auto token = [&](int r, int* h) {
    const long m = tile.m0 + r;
    const int t = (int)a.by_g.of((uint32_t)m);
    *h = tile.hkv * a.G + (int)(m - (long)t * a.G);
    return t;
  };
  for (int i = tid; i < num * per; i += kThreads) {
    const int r = i / per, d = 4 * (i - r * per);
    float top = s_m[r];
#pragma unroll
    for (int w = 1; w < kW; ++w) top = fmaxf(top, s_m[16 * w + r]);
    const float base = top == -INFINITY ? 0.f : top;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w)
      attn_add4(x, sum, *reinterpret_cast<const float4*>(acc + (w * R + r) * DH + d),
                s_l[16 * w + r], attn_exp2(s_m[16 * w + r] - base));
    int h;
    const int row = tile.seq.q0 + token(r, &h);
    if (a.cluster) {  // over the first warp's, and m and l behind the rows
      *reinterpret_cast<float4*>(acc + r * DH + d) = x;
      if (d == 0) {
        acc[kW * R * DH + 2 * r] = top;
        acc[kW * R * DH + 2 * r + 1] = sum;
      }
    } else if (part) {
      const long at = attn_part(a, tile.s, tile.hkv, (int)tile.m0 + r, row, h) * a.nsplit +
                      tile.split;
      *reinterpret_cast<float4*>(a.po + at * a.dh + d) = x;
      if (d == 0) {
        a.pml[2 * at] = top;
        a.pml[2 * at + 1] = sum;
      }
    } else if (!attn_store4<T>(a, row, h, d, x, top, sum)) {
      atomicOr(s_bad, 1 << r);
    }
  }
  if (part) return;
  if (a.cluster) {
    __syncwarp();
    tc::cluster_sync_all();
    const uint32_t at = smem_addr(acc);
    // a CTA the elements of its turn
    for (int i = tid + kThreads * tile.split; i < num * per; i += kThreads * a.nsplit) {
      const int r = i / per, d = 4 * (i - r * per);
      float top = -INFINITY, m[8];
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        m[z] = z < a.nsplit ? tc::ld_dsmem_f32(tc::cluster_map(at, z) + 4 * (kW * R * DH + 2 * r))
                            : -INFINITY;
        top = fmaxf(top, m[z]);
      }
      const float base = top == -INFINITY ? 0.f : top;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int z = 0; z < 8; ++z)
        if (z < a.nsplit) {
          const uint32_t from = tc::cluster_map(at, z);
          attn_add4(x, sum, tc::ld_dsmem_v4(from + 4 * (r * DH + d)),
                    tc::ld_dsmem_f32(from + 4 * (kW * R * DH + 2 * r + 1)), attn_exp2(m[z] - base));
        }
      int h;
      const int row = tile.seq.q0 + token(r, &h);
      // (the CTA that finds an element infinite or NaN computes its row again below;
      // the others' elements are stored before that)
      if (!attn_store4<T>(a, row, h, d, x, top, sum)) atomicOr(s_bad, 1 << r);
    }
    __syncwarp();
    tc::cluster_sync_all();
  } else {
    __syncthreads();
  }
  const int bad = *s_bad;
  for (int r = tid >> 5; r < num; r += kW)
    if (bad >> r & 1) {
      int h;
      const int t = token(r, &h);
      if (CALL) attn_redo_call<T>(a, tile.seq, t, h);
      else attn_redo<T>(a, tile.seq, t, h);
    }
}

// Host: a launch of `threads` a CTA, the shares of a tile in a cluster if they are joined so.
template <typename Kernel>
cudaError_t attn_launch(Kernel kern, unsigned grid, int threads, size_t smem, cudaStream_t s,
                        const AttnArgs& a, const CUtensorMap& k, const CUtensorMap& v) {
  if (!a.cluster) return launch_pdl(kern, dim3(grid), dim3(threads), smem, s, a, k, v);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)a.nsplit, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_ex(cfg, kern, a, k, v);
}

// Host: the maps of K and V for tiles of `slots` rows.
inline bool attn_tmaps(const AttnArgs& a, int slots, CUtensorMap* k, CUtensorMap* v) {
  if (a.Tk == 0)  // no slots to read: any row stands for those of K and V
    return make_tmap_bf16_rows(k, a.Q, a.dh, a.Hkv, 1, a.q_ld, 1, slots) &&
           make_tmap_bf16_rows(v, a.Q, a.dh, a.Hkv, 1, a.q_ld, 1, slots);
  return make_tmap_bf16_rows(k, a.K, a.dh, a.Hkv, a.Tk, a.k_ld, 1, slots) &&
         make_tmap_bf16_rows(v, a.V, a.dh, a.Hkv, a.Tk, a.v_ld, 1, slots);
}

}  // namespace ps
