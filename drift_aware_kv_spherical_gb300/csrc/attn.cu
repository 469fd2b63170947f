// Attention over packed sequences or cache rows on mma.sync: few query rows a KV head,
// fp32, and heads of more than 128.  (Many bf16 rows run on tcgen05, attn_tc.cu.)
//
// A CTA of four warps takes a tile of query rows against a share of the slots, which
// stream through a ring of shared-memory stages: bf16 heads of 64 and more by TMA (an
// instruction a tile; by cp.async, as the others still do it, addresses and copies were
// two thirds of all instructions), 128-byte swizzled.
//   narrow  16 rows; the warps take a quarter of every stage's slots each and join
//           their sums at the end (bf16 heads of 64 and more: k_attn_few, attn_few.cu)
//   wide    64 rows or 128, 16 a warp; every warp takes all slots of a stage (fp32: 16 at a
//           time, so that more products do not wait on one another)
// bf16 products are exact (m16n8k16), the weights rounded to bf16 on their way to V (2^-8 of
// one at most; their sum is of the unrounded ones); fp32 operands are split into two tf32 terms,
// three products (m16n8k8): the term left out is 2^-22 of a product, and so is what
// ex2.approx is off by.  The indices
// of a contraction may be permuted freely, so fp32 fragments are loaded as vectors.
// Rows of a stage lie an odd number of 16-byte units apart: no bank conflicts.
// What bounds fp32: three products of mma.sync and the splitting of K and V, which every
// warp repeats; 2048 x 2048 rows of 8 heads of 128 take 513 us, tensor cores 36 % busy,
// issue slots 46 %, two CTAs an SM at 255 registers.  Leading terms are summed by adds that
// round; low terms in accumulators of their own, so that no product waits on another.
//
// Long caches: a share is `chunk` slots, counted from slot 0, so that ragged lengths
// give as many CTAs as they have slots; the shares of a row are joined by k_attn_join or
// k_attn_join_rows.
#include <algorithm>
#include <climits>

#include "attn.cuh"

namespace ps {
namespace {

__device__ __forceinline__ void mma_t32(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// x = hi + lo, hi of 11 bits; lo's own 11 leave 2^-22 of x.  An infinity or NaN is
// all in hi.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  const float r = x - __uint_as_float(hi);
  lo = __float_as_uint(fabsf(x) < INFINITY ? r : 0.f);
}
// What a type's fragments are made of: D += A B over the slots or elements.
template <typename T, int DH, bool WIDE, bool TMA>
struct Tile;

template <int DH, bool WIDE, bool TMA>
struct Tile<__nv_bfloat16, DH, WIDE, TMA> {
  using T = __nv_bfloat16;
  static constexpr int kStep = 16;                 // slots a warp takes at a time
  static constexpr bool kKeep = DH <= 128;         // query fragments stay in registers
  uint32_t q[kKeep ? DH / 16 : 1][4];
  uint32_t qs;                                     // the warp's query rows
  int dh, ld;                                      // elements of a head; bytes of a stage's row

  __device__ __forceinline__ void q_frag(int kk, uint32_t* r) const {
    const int lane = threadIdx.x & 31;
    ldsm4(r, qs + (lane & 15) * ld + kk * 32 + (lane >> 4) * 16);
  }
  __device__ __forceinline__ void init() {
    if constexpr (kKeep) {
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk)
        if (16 * kk < dh) q_frag(kk, q[kk]);
    }
  }
  // 16-byte chunk 2 kk + b of the lane's row: `at` as row_at gave it
  __device__ __forceinline__ uint32_t chunk(uint32_t at, int kk, int b) const {
    if (!TMA) return at + kk * 32;
    return at + (kk >> 2) * (64 * 128) + ((((2 * kk) & 7) ^ ((threadIdx.x & 7) ^ b)) << 4);
  }
  __device__ __forceinline__ uint32_t row_at(uint32_t base, int row, int b) const {
    return TMA ? base + row * 128 : base + row * ld + b * 16;
  }
  // s[2][4]: rows x slots of the step
  __device__ __forceinline__ void scores(uint32_t k, float (*s)[4]) {
    const int lane = threadIdx.x & 31, id = lane >> 3, b1 = id & 1;
    const uint32_t at = row_at(k, (id >> 1) * 8 + (lane & 7), b1);
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
      if (16 * kk < dh) {
        uint32_t b[4], tmp[4];
        ldsm4(b, chunk(at, kk, b1));
        if constexpr (!kKeep) q_frag(kk, tmp);
        const uint32_t* f = kKeep ? q[kKeep ? kk : 0] : tmp;
        mma_b16(s[0], f, b[0], b[1]);
        mma_b16(s[1], f, b[2], b[3]);
      }
    }
  }
  // o[DH / 8][4] += P V; columns 8 j + 2 (lane % 4) + {0, 1}
  __device__ __forceinline__ void values(uint32_t v, const float (*p)[4], float (*o)[4]) {
    const int lane = threadIdx.x & 31, id = lane >> 3;
    const uint32_t f[4] = {pack2(p[0][0], p[0][1]), pack2(p[0][2], p[0][3]),
                           pack2(p[1][0], p[1][1]), pack2(p[1][2], p[1][3])};
    const int b1 = id >> 1;
    const uint32_t at = row_at(v, (id & 1) * 8 + (lane & 7), b1);
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
      if (16 * kk < dh) {
        uint32_t b[4];
        ldsm4_t(b, chunk(at, kk, b1));
        mma_b16(o[2 * kk], f, b[0], b[1]);
        mma_b16(o[2 * kk + 1], f, b[2], b[3]);
      }
    }
  }
  // element of a head that o[j][i] (i of 0, 1) is
  static __device__ __forceinline__ int column(int j, int i) {
    return 8 * j + 2 * (threadIdx.x & 3) + i;
  }
};

template <int DH, bool WIDE, bool TMA>
struct Tile<float, DH, WIDE, TMA> {
  using T = float;
  static constexpr int kStep = WIDE && DH <= 128 ? 16 : 8, NT = kStep / 8;
  static constexpr bool kKeep = DH <= 128;  // the queries' two terms stay in registers
  uint32_t qh[kKeep ? DH / 16 : 1][8], ql[kKeep ? DH / 16 : 1][8];
  uint32_t qs;
  int dh, ld;

  // 16 elements of the lane's rows g and g + 8 from d on: element 4 q + i of either
  __device__ __forceinline__ void q_frag(int d, uint32_t* hi, uint32_t* lo) const {
    const int lane = threadIdx.x & 31;
    const uint32_t at = qs + (lane >> 2) * ld + (d + 4 * (lane & 3)) * 4;
    const float4 x = load4(at), y = load4(at + 8 * ld);
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) split(v[i], hi[i], lo[i]);
  }
  __device__ __forceinline__ void init() {
    if constexpr (kKeep) {
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk)
        if (16 * kk < dh) q_frag(16 * kk, qh[kk], ql[kk]);
    }
  }
  __device__ __forceinline__ static float4 load4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
    return v;
  }
  __device__ __forceinline__ static float2 load2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
    return v;
  }
  // 16 elements at a time: lane q of four holds elements 4 q .. 4 q + 3, which are
  // k = q and q + 4 of two m16n8k8 products
  __device__ __forceinline__ void scores(uint32_t k, float (*s)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    // Products that follow one another go to accumulators of their own: one would wait
    // on itself.  Those of the leading terms are summed by rounding adds every 8 elements
    // (the unit truncates), the others' (2^-11 of them) where they are.
    float low[NT][4][4] = {};
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
      if (16 * kk < dh) {
        uint32_t th[8], tl[8];
        if constexpr (!kKeep) q_frag(16 * kk, th, tl);
        const uint32_t *h = kKeep ? qh[kKeep ? kk : 0] : th, *lo = kKeep ? ql[kKeep ? kk : 0] : tl;
        float top[NT][2][4] = {};
        uint32_t bh[NT][4], bl[NT][4];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          const float4 z = load4(k + (8 * c + g) * ld + (16 * kk + 4 * q) * 4);
          const float zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) split(zs[e], bh[c][e], bl[c][e]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t ah[4] = {h[2 * e], h[2 * e + 4], h[2 * e + 1], h[2 * e + 5]};
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            mma_t32(top[c][e], ah, bh[c] + 2 * e);
            mma_t32(low[c][e], ah, bl[c] + 2 * e);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t al[4] = {lo[2 * e], lo[2 * e + 4], lo[2 * e + 1], lo[2 * e + 5]};
#pragma unroll
          for (int c = 0; c < NT; ++c) mma_t32(low[c][2 + e], al, bh[c] + 2 * e);
        }
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[c][i] += top[c][0][i] + top[c][1][i];
      }
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[c][i] += (low[c][0][i] + low[c][1][i]) + (low[c][2][i] + low[c][3][i]);
  }
  // 8 slots: k = q is slot 2 q, k = q + 4 slot 2 q + 1 -- P's accumulators as they lie;
  // column g of the products i = 0, 1 is element 16 j + 2 g + i
  __device__ __forceinline__ void values(uint32_t v, const float (*p)[4], float (*o)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    uint32_t ah[NT][4], al[NT][4];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      split(p[c][0], ah[c][0], al[c][0]);
      split(p[c][2], ah[c][1], al[c][1]);
      split(p[c][1], ah[c][2], al[c][2]);
      split(p[c][3], ah[c][3], al[c][3]);
    }
#pragma unroll
    for (int k0 = 0; k0 < DH / 16; k0 += 2) {
      if (16 * k0 < dh) {  // (an odd last one: the second's columns are not stored)
        float top[4][4] = {}, low[4][4] = {};
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          uint32_t bh[4][2], bl[4][2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t col = (16 * (16 * (k0 + n) < dh ? k0 + n : k0) + 2 * g) * 4;
            const uint32_t at = v + (8 * c + 2 * q) * ld + col;
            const float2 x = load2(at), y = load2(at + ld);
            split(x.x, bh[2 * n][0], bl[2 * n][0]);
            split(y.x, bh[2 * n][1], bl[2 * n][1]);
            split(x.y, bh[2 * n + 1][0], bl[2 * n + 1][0]);
            split(y.y, bh[2 * n + 1][1], bl[2 * n + 1][1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_t32(low[i], al[c], bh[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_t32(top[i], ah[c], bh[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_t32(low[i], ah[c], bl[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[2 * k0 + i][e] += top[i][e] + low[i][e];
      }
    }
  }
  static __device__ __forceinline__ int column(int j, int i) {
    return 16 * (j >> 1) + 4 * (threadIdx.x & 3) + 2 * i + (j & 1);
  }
};

// Rows of a wide tile, 16 a warp.  bf16 heads of more than 128 leave an SM one CTA by their
// shared memory: 2 x 1024^2 rows x 8 heads of 256 take 91 us in tiles of 128, 114 of 64.
constexpr int wide_rows(bool f32, int dh) { return !f32 && dh > 128 ? 128 : 64; }

template <typename T, int DH, bool WIDE, bool TMA>
struct Shape {
  static constexpr int kStep = Tile<T, DH, WIDE, TMA>::kStep;
  static constexpr int kSlots = sizeof(T) == 4 ? 32 : 64; // of a stage
  static_assert(WIDE || kSlots == kW * kStep, "a step a warp");
  static constexpr int kRow = DH * (int)sizeof(T) + 16;   // bytes of a row, at most
  static constexpr int kHalf = kSlots * (TMA ? DH * (int)sizeof(T) : kRow);  // K, or V
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = DH <= 64 ? 4 : DH <= 128 && sizeof(T) == 2 ? 3 : 2;
  // bytes from one step's rows to the next
  static __device__ __forceinline__ int step(int ld) { return kStep * (TMA ? 128 : ld); }
  static constexpr int kRows = WIDE ? wide_rows(sizeof(T) == 4, DH) : 16;
  static constexpr int kCta = WIDE ? 2 * kRows : kThreads;  // threads
  static constexpr size_t kBytes =
      (TMA ? 1024 : 0) + (size_t)kStages * kStage + kRows * kRow;
};

template <typename T, int DH, bool WIDE, bool TMA>
__global__ void __launch_bounds__((Shape<T, DH, WIDE, TMA>::kCta))
k_attn(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tk,
       const __grid_constant__ CUtensorMap tv) {
  pdl_prologue();
  using SH = Shape<T, DH, WIDE, TMA>;
  using TL = Tile<T, DH, WIDE, TMA>;
  constexpr int kRows = SH::kRows, kStep = TL::kStep, kSlots = SH::kSlots;
  constexpr int NT = kStep / 8;                 // score fragments of a step
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = TMA ? reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                   ~static_cast<uintptr_t>(1023))
                      : smem_raw;
  __shared__ float s_m[kW][16], s_l[kW][16];
  __shared__ int s_bad, s_abort;
  __shared__ uint64_t s_full[SH::kStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int ld = a.dh * (int)sizeof(T) + 16;
  uint8_t* qs = smem + SH::kStages * SH::kStage;

  AttnTile tile{};
  if (!tile.find<kRows>(a, kSlots)) return;
  const AttnSeq& seq = tile.seq;
  const long m0 = tile.m0;
  const int hkv = tile.hkv, num = tile.num, lo = tile.lo, hi = tile.hi, steps = tile.steps;
  const bool part = a.nsplit > 1;

  // ---- queries; rows past the last one are zero
  {
    const int cpr = a.dh * (int)sizeof(T) / 16;
    for (int i = tid; i < kRows * cpr; i += SH::kCta) {
      const int r = i / cpr, c = i - r * cpr;
      const long m = m0 + min(r, num - 1);
      const int t = (int)a.by_g.of((uint32_t)m), h = hkv * a.G + (int)(m - (long)t * a.G);
      const T* src = static_cast<const T*>(a.Q) + (long)(seq.q0 + t) * a.q_ld + (long)h * a.dh;
      cp_async16(smem_addr(qs + r * ld + c * 16), reinterpret_cast<const uint8_t*>(src) + c * 16,
                 r < num);
    }
  }
  const T* K = static_cast<const T*>(a.K) + (long)hkv * a.dh;
  const T* V = static_cast<const T*>(a.V) + (long)hkv * a.dh;
  if (TMA) {
    if (tid == 0) {
#pragma unroll
      for (int i = 0; i < SH::kStages; ++i) tc::mbar_init(s_full + i, 1);
      s_abort = 0;
      tc::fence_mbar_init();
    }
    __syncthreads();
  }
  // a stage: slots from n on; those past hi are zero, or by TMA whatever comes next
  auto load = [&](int j) {
    if (TMA) {
      if (tid == 0 && j < steps) {
        uint64_t* bar = s_full + j % SH::kStages;
        uint8_t* to = smem + (j % SH::kStages) * SH::kStage;
        tc::mbar_expect_tx(bar, SH::kStage);
#pragma unroll
        for (int p = 0; p < DH / 64; ++p) {
          const int row = seq.k0 + lo + j * kSlots;
          tc::tma_load_3d(to + p * kSlots * 128, &tk, bar, 64 * p, hkv, row);
          tc::tma_load_3d(to + SH::kHalf + p * kSlots * 128, &tv, bar, 64 * p, hkv, row);
        }
      }
      if (j >= SH::kStages - 1) return;  // (what is committed below is the queries)
    } else if (j < steps) {
      constexpr int kCpr = DH * (int)sizeof(T) / 16;
      const long n0 = lo + (long)j * kSlots;
      const uint32_t base = smem_addr(smem + (j % SH::kStages) * SH::kStage);
      const int used = a.dh * (int)sizeof(T) / 16;
#pragma unroll 4
      for (int i = tid; i < kSlots * kCpr; i += SH::kCta) {
        const int r = i / kCpr, c = i % kCpr;
        if (c < used) {
          const bool in = n0 + r < hi;
          const long row = seq.k0 + min(n0 + r, (long)hi - 1);
          cp_async16(base + r * ld + c * 16,
                     reinterpret_cast<const uint8_t*>(K + row * a.k_ld) + c * 16, in);
          cp_async16(base + SH::kHalf + r * ld + c * 16,
                     reinterpret_cast<const uint8_t*>(V + row * a.v_ld) + c * 16, in);
        }
      }
    }
    cp_commit();
  };
  for (int j = 0; j < SH::kStages - 1; ++j) load(j);

  // ---- the lane's two rows
  int2 see[2];
  long m_of[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (WIDE ? 16 * warp : 0) + g + 8 * i;
    m_of[i] = m0 + r;
    see[i] = make_int2(lo, hi);  // past the last row: no mask
    if (r < num) {
      const int2 x = attn_seen(a, seq, (int)a.by_g.of((uint32_t)(m0 + r)));
      see[i] = make_int2(max(x.x, lo), min(x.y, hi));  // of the share
    }
  }
  const int all_lo = __reduce_max_sync(0xffffffffu, max(see[0].x, see[1].x));
  const int all_hi = __reduce_min_sync(0xffffffffu, min(see[0].y, see[1].y));
  float o[DH / 8][4];
#pragma unroll
  for (int j = 0; j < DH / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
  float mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float f = a.scale * kAttnLog2e;
  TL tl;
  tl.qs = smem_addr(qs + (WIDE ? 16 * warp : 0) * ld);
  tl.dh = a.dh;
  tl.ld = ld;

  bool ok = true;  // (of the warp)
  for (int j = 0; j < steps; ++j) {
    if (!TMA || j == 0) cp_wait<TMA ? 0 : SH::kStages - 2>();
    __syncthreads();
    if (j == 0) tl.init();
    load(j + SH::kStages - 1);
    uint8_t* stage = smem + (j % SH::kStages) * SH::kStage;
    const uint32_t kb = smem_addr(stage), vb = kb + SH::kHalf;
    if (TMA) {
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(s_full + j % SH::kStages,
                                                       (j / SH::kStages) & 1, a.status, &s_abort));
      if (!ok) continue;  // (its barriers go on; the other waits end soon too)
    }
#pragma unroll 1
    for (int x = WIDE ? 0 : warp; x < (WIDE ? kSlots / kStep : warp + 1); ++x) {
      const int n = lo + j * kSlots + x * kStep;
      if (n >= hi) break;
      float sc[NT][4];
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[c][i] = 0.f;
      tl.scores(kb + x * SH::step(ld), sc);
      const bool whole = n >= all_lo && n + kStep <= all_hi;
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[c][i] *= f;
          const int at = n + 8 * c + 2 * q4 + (i & 1);
          if (!whole && (at < see[i >> 1].x || at >= see[i >> 1].y)) sc[c][i] = -INFINITY;
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float t = fmaxf(sc[0][2 * r], sc[0][2 * r + 1]);
        if (NT == 2) t = fmaxf(t, fmaxf(sc[NT - 1][2 * r], sc[NT - 1][2 * r + 1]));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        const bool grow = t > mx[r];
        if (__any_sync(0xffffffffu, grow)) {
          const float c = grow ? attn_exp2(mx[r] - t) : 1.f;
          mx[r] = grow ? t : mx[r];
          l[r] *= c;
#pragma unroll
          for (int d = 0; d < DH / 8; ++d) {
            o[d][2 * r] *= c;
            o[d][2 * r + 1] *= c;
          }
        }
        const float base = mx[r] == -INFINITY ? 0.f : mx[r];
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p = attn_exp2(sc[c][2 * r + i] - base);
            sc[c][2 * r + i] = p;
            l[r] += p;
          }
      }
      if (TMA && n + kStep > seq.m) {
        // slots that the sequence does not have may hold anything, and P's zeros times
        // NaN are NaN
        for (int c = lane; c < kStep * DH / 8; c += 32) {
          const int r = c / (DH / 8), k = c % (DH / 8);
          if (n + r >= seq.m)
            *reinterpret_cast<uint4*>(stage + SH::kHalf + (k >> 3) * (kSlots * 128) +
                                      (x * kStep + r) * 128 + (k & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      tl.values(vb + x * SH::step(ld), sc, o);
    }
  }
  cp_wait<0>();
  if (TMA && __syncthreads_or(!ok)) {  // a timeout: wait for the copies under way
    if (tid == 0) {
      const uint64_t t0 = tc::globaltimer();
      for (int i = 0; i < SH::kStages; ++i) {
        const int uses = (steps + SH::kStages - 1 - i) / SH::kStages;
        while (uses > 0 && !tc::mbar_try_wait(s_full + i, (uses - 1) & 1) &&
               tc::globaltimer() - t0 < tc::kWaitLimitNs) {
        }
      }
    }
    if (!a.cluster) return;  // (else the others still read this CTA's shared memory)
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }

  // ---- the finished rows.  Narrow: the warps' sums joined through shared memory
  if constexpr (!WIDE) {
    float* acc = reinterpret_cast<float*>(smem);  // [kW][16][DH], and 32 behind
    __syncthreads();  // no warp reads the stages any more
    if (q4 == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        s_m[warp][g + 8 * r] = mx[r];
        s_l[warp][g + 8 * r] = l[r];
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int d = 0; d < DH / 8; ++d)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[(warp * 16 + g + 8 * r) * DH + TL::column(d, i)] = o[d][2 * r + i];
    attn_join_warps<T, DH, 16, true>(a, tile, acc, &s_m[0][0], &s_l[0][0], &s_bad);
  } else {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool in = m_of[r] < m0 + num;
      const long m = in ? m_of[r] : m0;
      const int t = (int)a.by_g.of((uint32_t)m), h = hkv * a.G + (int)(m - (long)t * a.G);
      const long row = (long)(seq.q0 + t) * a.Hq + h;
      bool fine = true;
      if (part) {
        const long at = row * a.nsplit + tile.split;
        if (in) {
#pragma unroll
          for (int d = 0; d < DH / 8; ++d)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (TL::column(d, i) < a.dh) a.po[at * a.dh + TL::column(d, i)] = o[d][2 * r + i];
          if (q4 == 0) {
            a.pml[2 * at] = mx[r];
            a.pml[2 * at + 1] = l[r];
          }
        }
        continue;
      }
      const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
      if (in) {
        T* to = static_cast<T*>(a.O) + (long)(seq.q0 + t) * a.o_ld + (long)h * a.dh;
#pragma unroll
        for (int d = 0; d < DH / 8; ++d)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = TL::column(d, i);
            if (c < a.dh) {
              const float z = l[r] == 0.f ? 0.f : o[d][2 * r + i] * inv;
              fine = fine && fabsf(z) < INFINITY;
              Store<T>::put(to + c, z);
            }
          }
        if (q4 == 0 && a.lse != nullptr) a.lse[row] = attn_lse(mx[r], l[r]);
      }
      uint32_t bad = __ballot_sync(0xffffffffu, !fine);
      for (int k = 0; k < 8; ++k)
        if (bad >> (4 * k) & 15) {
          const int tk = __shfl_sync(0xffffffffu, t, 4 * k), hk = __shfl_sync(0xffffffffu, h, 4 * k);
          attn_redo_call<T>(a, seq, tk, hk);
        }
    }
  }
}

// Row number i of those that are joined (its partial sums' too, attn_part): its sequence,
// token and head; false where there is none.  For whole warps.
__device__ __forceinline__ bool join_row(const AttnArgs& a, int i, AttnSeq* seq, int* t, int* h) {
  if (a.per_seq > 0) {  // numbers for the most rows that a sequence may have
    const int k = i / a.Hkv, hkv = i - k * a.Hkv, s = k / a.most, m = k - s * a.most;
    *seq = attn_seq(a, s);
    *t = m / a.G;
    *h = hkv * a.G + m - *t * a.G;
  } else {
    const int r = i / a.Hq;
    *h = i - r * a.Hq;
    *seq = attn_seq(a, attn_find(a.S, r, [&](int s) { return (long)attn_q_off(a, s); }));
    *t = r - seq->q0;
  }
  const long rows = (long)seq->n * a.G;
  return *t >= 0 && *t < seq->n && rows >= a.least && rows <= a.most;
}
// A row's shares: the first and last that saw a slot of it.
__device__ __forceinline__ int2 join_shares(const AttnArgs& a, const AttnSeq& seq, int t) {
  const int2 see = attn_seen(a, seq, t);
  const int from = min(see.x / a.chunk, a.nsplit - 1);
  return make_int2(from, see.x < see.y ? min((see.y - 1) / a.chunk, a.nsplit - 1) : from - 1);
}

// The shares of a row joined, in order.  Where they are many and the rows few a CTA takes
// a row, dh / 4 lanes an element group, the groups of lanes taking the shares in turn (the
// loads are one round or few: 57 shares of 224 rows 5.5 us, 9.6 by 128 threads) ...
constexpr int kJoin = 512;
template <typename T>
__global__ void __launch_bounds__(kJoin)
k_attn_join(const __grid_constant__ AttnArgs a) {
  pdl_prologue();
  __shared__ float4 s_o[kJoin];
  __shared__ float s_l[kJoin], s_top[kJoin / 32];
  int t, h;
  AttnSeq seq;
  if (!join_row(a, blockIdx.x, &seq, &t, &h)) return;
  const int r = seq.q0 + t, tid = threadIdx.x;
  const long row = blockIdx.x;
  const int2 shares = join_shares(a, seq, t);
  const int from = shares.x, to = shares.y;
  const float* pml = a.pml + 2 * row * a.nsplit;
  const float* po = a.po + row * a.nsplit * a.dh;
  float top = -INFINITY;
  for (int i = from + tid; i <= to; i += kJoin) top = fmaxf(top, pml[2 * i]);
  top = warp_max(top);
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoin / 32; ++w) top = fmaxf(top, s_top[w]);
  const float base = top == -INFINITY ? 0.f : top;
  const int lanes = a.dh / 4, groups = kJoin / lanes;
  const int grp = tid / lanes, d = 4 * (tid - grp * lanes);
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  if (grp < groups) {
#pragma unroll 4
    for (int i = from + grp; i <= to; i += groups)
      attn_add4(x, l, *reinterpret_cast<const float4*>(po + (long)i * a.dh + d), pml[2 * i + 1],
                attn_exp2(pml[2 * i] - base));
  }
  s_o[tid] = x;
  s_l[tid] = l;
  __syncthreads();
  bool fine = true;
  if (grp == 0) {
    for (int k = 1; k < min(groups, to - from + 1); ++k)
      attn_add4(x, l, s_o[tid + k * lanes], s_l[tid + k * lanes], 1.f);
    fine = attn_store4<T>(a, r, h, d, x, top, l);
  }
  if (__syncthreads_or(!fine) && tid < 32) attn_redo_call<T>(a, seq, t, h);
}

// ... else a warp does (18800 rows of two shares 12 us, by a CTA of 128 threads each 38).
template <typename T>
__global__ void __launch_bounds__(128)
k_attn_join_rows(const __grid_constant__ AttnArgs a, int count) {
  pdl_prologue();
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  int t, h;
  AttnSeq seq;
  if (i >= count || !join_row(a, i, &seq, &t, &h)) return;
  const long row = i;
  const int2 shares = join_shares(a, seq, t);
  const float* pml = a.pml + 2 * row * a.nsplit;
  const float* po = a.po + row * a.nsplit * a.dh;
  float top = -INFINITY;
  for (int k = shares.x + lane; k <= shares.y; k += 32) top = fmaxf(top, pml[2 * k]);
  top = warp_max(top);
  const float base = top == -INFINITY ? 0.f : top;
  bool fine = true;
  for (int d = 4 * lane; d < a.dh; d += 128) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int k = shares.x; k <= shares.y; ++k)
      attn_add4(x, l, *reinterpret_cast<const float4*>(po + (long)k * a.dh + d), pml[2 * k + 1],
                attn_exp2(pml[2 * k] - base));
    fine = attn_store4<T>(a, seq.q0 + t, h, d, x, top, l) && fine;
  }
  if (__any_sync(0xffffffffu, !fine)) attn_redo_call<T>(a, seq, t, h);
}

// ---------------------------------------------------------------- host
// Rows of a sequence and KV head up to which the narrow kernel takes it: 4 x 32 rows x
// 32 heads on 768 slots 24 us on tcgen05, 50 here.
constexpr int kFew = 8;

// One kernel's part of a call.
struct Part {
  bool on = false, wide = false;
  int least = 0, most = INT_MAX;  // rows of the sequences that it takes
  int per_seq = 0, rows = 0;      // rows of a tile
  long tiles = 0;
  int nsplit = 1, chunk = INT_MAX;
  bool cluster = false;           // the shares are joined in a cluster
};
// Few rows on mma.sync, many of bf16 on tcgen05; a batch of unequal lengths may hold both.
struct Plan {
  Part few, tc;
  int R = 1;
};

// Rows of a narrow tile: k_attn_few has one of 8.
int few_rows(int dtype, int dh, int G, int max_q) {
  return dtype == PS_BF16 && dh >= 64 && (long)max_q * G <= 8 ? 8 : 16;
}

// Shares of max_k slots for `ctas` CTAs a share: `all` CTAs or so, shares of `least`
// slots at least, a multiple of `unit` each.
void share(Part& p, long ctas, long all, int max_k, int least, int unit) {
  const long want = std::min({all / std::max(ctas, 1L), (long)max_k / least, 512L});
  const long n = std::max(want, 1L);
  const long chunk = (((long)max_k + n - 1) / n + unit - 1) / unit * unit;
  p.nsplit = (int)(((long)max_k + chunk - 1) / chunk);
  p.chunk = (int)std::min(chunk, (long)INT_MAX);
}

Plan plan(int dtype, int S, int max_k, int Hq, int Hkv, int dh, int Tq, int max_q) {
  Plan p;
  const int G = Hq / Hkv;
  const long rows = (long)Tq * G;
  const bool many = (long)max_q * G > kFew;
  const bool tc = many && dtype == PS_BF16 && dh >= 64 && dh <= 128 && G <= kTcRows;
  if (tc) {
    p.R = kTcRows / G;
    p.tc.on = true;
    p.tc.tiles = Tq / (2 * p.R) + S;
    const long items = ((long)Tq + 2 * p.R - 1) / (2 * p.R) * Hkv;
    // Joining costs some 2.5 us and one more for 2000 rows and query heads, which short
    // sequences do not give back: 4700 packed causal tokens of 4 heads 32 us, 40 in two
    // shares; 2048 tokens of 4 heads on 2048 slots 34, 30 in two.
    const bool split = (long)Tq * Hq <= 8L * max_k;
    share(p.tc, split ? items : (long)kSmTarget, kSmTarget, max_k, 512, 128);
  }
  if (!tc || (long)S * max_q != Tq) {
    p.few.on = true;
    const int slots = dtype == PS_F32 ? 32 : 64;   // of a stage
    long ctas;
    if (tc) {  // the sequences of few rows among longer ones
      p.tc.least = kFew + 1;
      p.few.most = kFew;
      p.few.per_seq = 1;
      p.few.tiles = (long)S * p.few.per_seq;
      p.few.rows = kFew;
      ctas = (long)S * Hkv;
    } else {
      // Wide tiles read K and V a quarter or an eighth as often, and leave SMs idle where
      // there are few.  fp32: 2048^2 x 32 heads x 128 2509 -> 1878 us, 1024^2 x 8 x 64 (128
      // tiles) 116 -> 97, but 3 x 77 rows of 4 heads (16 tiles) 17.5 -> 28, and in shares
      // 4 x 32 x 8 (32 tiles) 69 -> 81.  bf16 gains with shares too, heads of 256:
      // 2 x 1024^2 x 8 292 -> 91, 71 x 32 on 16 K slots 583 -> 206, 6 x 100 x 4 on 900
      // (20 tiles in three shares) 91 -> 44.
      const int w = wide_rows(dtype == PS_F32, dh);
      const long tiles = (rows + w - 1) / w * Hkv;
      const long shares = std::max(max_k / (4 * slots), 1);
      p.few.wide = many && (dtype == PS_F32 ? tiles >= kSmTarget / 2
                                            : tiles * shares >= kSmTarget / 4);
      const int r = p.few.wide ? w : few_rows(dtype, dh, G, max_q);
      p.few.tiles = rows / r + S;
      p.few.rows = r;
      ctas = (rows + r - 1) / r * Hkv;
    }
    share(p.few, ctas, (p.few.wide ? 1 : 4) * kSmTarget, max_k, 4 * slots, slots);
    p.few.cluster = !p.few.wide && p.few.nsplit > 1 && p.few.nsplit <= 8;
  }
  return p;
}
// Rows whose shares are joined.
long joined(const Part& p, int S, int Hq, int Hkv, int Tq) {
  return p.per_seq > 0 ? (long)S * p.most * Hkv : (long)Tq * Hq;
}
void parts(Carver& cv, const Part& p, int S, int Hq, int Hkv, int dh, int Tq, float** po,
           float** pml) {
  if (!p.on || p.nsplit == 1 || p.cluster) return;
  const size_t rows = (size_t)joined(p, S, Hq, Hkv, Tq) * p.nsplit;
  *po = cv.take<float>(rows * dh);
  *pml = cv.take<float>(rows * 2);
}

template <typename T, int DH, bool WIDE, bool TMA>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
  auto kern = k_attn<T, DH, WIDE, TMA>;
  using SH = Shape<T, DH, WIDE, TMA>;
  constexpr size_t smem = SH::kBytes;
  static_assert(smem <= 227 * 1024 - 1024, "a CTA's shared memory");
  static_assert((size_t)kW * 16 * DH * 4 + 128 <= (size_t)SH::kStages * SH::kStage, "the warps' sums");
  static DeviceOnce once;
  const cudaError_t e = allow_smem(kern, smem, once);
  if (e != cudaSuccess) return e;
  const long grid = a.tiles * a.Hkv * a.nsplit;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap k{}, v{};
  if (TMA && !attn_tmaps(a, SH::kSlots, &k, &v)) return cudaErrorInvalidValue;
  return attn_launch(kern, (unsigned)grid, SH::kCta, smem, s, a, k, v);
}
template <typename T, int DH>
cudaError_t by_width(const AttnArgs& a, bool wide, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (a.dh >= 64)  // (a tile's 64 elements are no more than a head has)
      return wide ? launch<T, DH, true, true>(a, s) : attn_few_launch(a, s);
    return wide ? launch<T, 64, true, false>(a, s) : launch<T, 64, false, false>(a, s);
  } else {
    return wide ? launch<T, DH, true, false>(a, s) : launch<T, DH, false, false>(a, s);
  }
}
template <typename T>
cudaError_t by_dh(const AttnArgs& a, bool wide, cudaStream_t s) {
  if (a.dh <= 64) return by_width<T, 64>(a, wide, s);
  if (a.dh <= 128) return by_width<T, 128>(a, wide, s);
  return by_width<T, 256>(a, wide, s);
}

template <typename T>
cudaError_t join(const AttnArgs& a, long rows, cudaStream_t s) {
  if (a.nsplit > 16 && rows <= 512)
    return launch_pdl(k_attn_join<T>, dim3((unsigned)rows), dim3(kJoin), 0, s, a);
  return launch_pdl(k_attn_join_rows<T>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, a,
                    (int)rows);
}

size_t ws_of(int dtype, int S, int max_k, int Hq, int Hkv, int dh, int Tq, int max_q) {
  const Plan p = plan(dtype, S, max_k, Hq, Hkv, dh, Tq, max_q);
  Carver cv(nullptr);
  float *po, *pml;
  parts(cv, p.few, S, Hq, Hkv, dh, Tq, &po, &pml);
  parts(cv, p.tc, S, Hq, Hkv, dh, Tq, &po, &pml);
  return cv.bytes();
}

}  // namespace

size_t attn_ws(int S, int max_k, int Hq, int Hkv, int dh, int Tq, int max_q) {
  return std::max(ws_of(PS_F32, S, max_k, Hq, Hkv, dh, Tq, max_q),
                  ws_of(PS_BF16, S, max_k, Hq, Hkv, dh, Tq, max_q));
}

cudaError_t attn_run(AttnArgs a, cudaStream_t s) {
  const Plan p = plan(a.dtype, a.S, a.max_k, a.Hq, a.Hkv, a.dh, a.Tq, a.max_q);
  a.by_g = quotient((uint32_t)a.G);
  a.R = p.R;
  Carver cv(a.ws);
  auto run = [&](const Part& x, bool tc) {
    if (!x.on) return cudaSuccess;
    AttnArgs b = a;
    b.least = x.least;
    b.most = x.most;
    b.per_seq = x.per_seq;
    b.rows = x.rows;
    b.tiles = x.tiles;
    b.nsplit = x.nsplit;
    b.chunk = x.chunk;
    b.cluster = x.cluster;
    parts(cv, x, a.S, a.Hq, a.Hkv, a.dh, a.Tq, &b.po, &b.pml);
    cudaError_t e = tc ? attn_tc_launch(b, s)
                       : a.dtype == PS_F32 ? by_dh<float>(b, x.wide, s)
                                           : by_dh<__nv_bfloat16>(b, x.wide, s);
    if (e != cudaSuccess || x.nsplit == 1 || x.cluster) return e;
    const long rows = joined(x, a.S, a.Hq, a.Hkv, a.Tq);
    return a.dtype == PS_F32 ? join<float>(b, rows, s) : join<__nv_bfloat16>(b, rows, s);
  };
  const cudaError_t e = run(p.few, false);
  return e != cudaSuccess ? e : run(p.tc, true);
}

}  // namespace ps
