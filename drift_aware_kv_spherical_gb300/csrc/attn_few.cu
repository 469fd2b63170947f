// Attention over packed sequences or cache rows for few bf16 query rows a KV head: single
// tokens of grouped heads above all.
//
// A CTA of four warps takes a tile of 8 (or 16) query rows against a share of the slots, 64
// slots a stage by TMA, 128-byte swizzled; a warp takes 16 of them.  The products are
// turned round: slots are the 16 of the m16n8k16 tile and rows its 8, S^T = K Q^T and
// O^T += V^T P^T, so that 7 rows of a group of heads fill a tile that rows on the 16
// would leave half empty: half the products, and half of O's registers.  P^T comes out of
// the accumulators of S^T by a transposing move of 8x8 halves, rounded to bf16 (V's type: half
// a step, 2^-8 at most, of a weight; the row's sum is of the unrounded ones).
// The running maximum of a row is common to the warp and follows the scores only when one
// passes it by 2^kGrow (P carries a factor up to that): most steps vote once and
// exchange nothing.
//
// One token of 28/4 heads for each of 8 sequences of up to 32 K slots: 52 us, 75 % of the
// memory's nominal rate (86 % of a copy's); with rows as the 16 it was 85 us for 8 tokens
// where this takes 75.  What bounds it is the latency of a warp's own steps, 12 warps an SM:
// three CTAs of two stages of two 16 KB tiles each.
#include <algorithm>

#include "attn.cuh"

namespace ps {
namespace {

constexpr int kStep = 16, kSlots = kW * kStep;  // slots of a warp, of a stage
constexpr float kGrow = 8.f;

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int DH, int RT>
struct Few {
  static constexpr int kRows = 8 * RT;
  static constexpr int kHalf = kSlots * DH * 2;         // K, or V, of a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = DH <= 64 ? 4 : 2;      // (three CTAs an SM at 128)
  static constexpr int kQ = kStages * kStage;
  static constexpr int kRow = DH * 2 + 16;              // bytes between the queries' rows
  static constexpr size_t kBytes = 1024 + kQ + kRows * kRow;
};

template <int DH, int RT>
__global__ void __launch_bounds__(kThreads)
k_attn_few(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tk,
           const __grid_constant__ CUtensorMap tv) {
  pdl_prologue();
  using F = Few<DH, RT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ float s_m[kW][16], s_l[kW][16];
  __shared__ int s_bad, s_abort;
  __shared__ uint64_t s_full[F::kStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  AttnTile tile{};
  if (!tile.find<F::kRows>(a, kSlots)) return;
  const int lo = tile.lo, hi = tile.hi, steps = tile.steps;
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < F::kStages; ++i) tc::mbar_init(s_full + i, 1);
    s_abort = 0;
    tc::fence_mbar_init();
  }
  auto load = [&](int j) {  // by one thread
    uint64_t* bar = s_full + j % F::kStages;
    uint8_t* to = smem + (j % F::kStages) * F::kStage;
    const int row = tile.seq.k0 + lo + j * kSlots;
    tc::mbar_expect_tx(bar, F::kStage);
#pragma unroll
    for (int p = 0; p < DH / 64; ++p) {
      tc::tma_load_3d(to + p * kSlots * 128, &tk, bar, 64 * p, tile.hkv, row);
      tc::tma_load_3d(to + F::kHalf + p * kSlots * 128, &tv, bar, 64 * p, tile.hkv, row);
    }
  };
  if (tid == 0)
    for (int j = 0; j < min(F::kStages, steps); ++j) load(j);
  // ---- queries; rows past the last one are zero
  uint8_t* qs = smem + F::kQ;
  {
    const int cpr = a.dh / 8;
    for (int i = tid; i < F::kRows * cpr; i += kThreads) {
      const int r = i / cpr, c = i - r * cpr;
      const long m = tile.m0 + min(r, tile.num - 1);
      const int t = (int)a.by_g.of((uint32_t)m), h = tile.hkv * a.G + (int)(m - (long)t * a.G);
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.Q) +
                                 (long)(tile.seq.q0 + t) * a.q_ld + (long)h * a.dh;
      cp_async16(smem_addr(qs + r * F::kRow + c * 16), src + c * 8, r < tile.num);
    }
    // (a head's elements end inside a pair of products: what lies behind is not read)
    cp_commit();
  }
  // ---- the lane's rows: 8 i + 2 q and the next one
  int2 see[RT][2];
  int all_lo = lo, all_hi = hi;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * i + 2 * q + e;
      see[i][e] = make_int2(lo, hi);  // past the last row: no mask
      if (r < tile.num) {
        const int2 x = attn_seen(a, tile.seq, (int)a.by_g.of((uint32_t)(tile.m0 + r)));
        see[i][e] = make_int2(max(x.x, lo), min(x.y, hi));  // of the share
      }
      all_lo = max(all_lo, see[i][e].x);
      all_hi = min(all_hi, see[i][e].y);
    }
  all_lo = __reduce_max_sync(0xffffffffu, all_lo);
  all_hi = __reduce_min_sync(0xffffffffu, all_hi);
  float o[DH / 16][RT][4];
#pragma unroll
  for (int d = 0; d < DH / 16; ++d)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[d][i][c] = 0.f;
  float mx[RT][2], l[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[i][e] = -INFINITY;
      l[i][e] = 0.f;
    }
  const float f = a.scale * kAttnLog2e;
  cp_wait<0>();
  __syncthreads();
  uint32_t qf[DH / 16][RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int kk = 0; kk < DH / 16; kk += 2) {
      uint32_t r[4] = {0, 0, 0, 0};
      if (16 * kk < a.dh)  // (one chunk past a head's end at most: within the row's padding
                           // or the next row; its products are not formed)
        ldsm4(r, smem_addr(qs + (8 * i + (lane & 7)) * F::kRow + min(2 * kk + (lane >> 3), a.dh / 8) * 16));
      qf[kk][i][0] = r[0];
      qf[kk][i][1] = r[1];
      qf[kk + 1][i][0] = r[2];
      qf[kk + 1][i][1] = r[3];
    }
  const int id = lane >> 3, l7 = lane & 7;
  // the lane's row of K's and V's fragments in the warp's 16, and the chunk of each pair
  const uint32_t k_at = (uint32_t)(warp * kStep + (id & 1) * 8 + l7) * 128u, k_c = l7 ^ (id >> 1);
  const uint32_t v_at = (uint32_t)(warp * kStep + (id >> 1) * 8 + l7) * 128u, v_c = l7 ^ (id & 1);

  bool ok = true;  // (of the warp)
  for (int j = 0; j < steps; ++j) {
    uint8_t* stage = smem + (j % F::kStages) * F::kStage;
    const uint32_t kb = smem_addr(stage), vb = kb + F::kHalf;
    ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(s_full + j % F::kStages,
                                                     (j / F::kStages) & 1, a.status, &s_abort));
    const int n = lo + j * kSlots + warp * kStep;
    if (ok && n < hi) {
      float s[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][c] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk)
        if (16 * kk < a.dh) {
          uint32_t k[4];
          ldsm4(k, kb + k_at + (kk >> 2) * (kSlots * 128) + ((((2 * kk) & 7) ^ k_c) << 4));
#pragma unroll
          for (int i = 0; i < RT; ++i) mma_b16(s[i], k, qf[kk][i][0], qf[kk][i][1]);
        }
      const bool whole = n >= all_lo && n + kStep <= all_hi;
      bool grow = false;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int2 x = see[i][c & 1];
          const int at = n + g + 8 * (c >> 1);
          s[i][c] *= f;
          if (!whole && (at < x.x || at >= x.y)) s[i][c] = -INFINITY;
          grow = grow || s[i][c] > mx[i][c & 1] + kGrow;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = fmaxf(s[i][e], s[i][e + 2]);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            const float m = t > mx[i][e] ? t : mx[i][e];
            const float c = m > mx[i][e] ? attn_exp2(mx[i][e] - m) : 1.f;
            mx[i][e] = m;
            l[i][e] *= c;
#pragma unroll
            for (int d = 0; d < DH / 16; ++d) {
              o[d][i][e] *= c;
              o[d][i][e + 2] *= c;
            }
          }
      }
      uint32_t p[RT][2];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float m = mx[i][c & 1];
          s[i][c] = attn_exp2(s[i][c] - (m == -INFINITY ? 0.f : m));
          l[i][c & 1] += s[i][c];
        }
        p[i][0] = transposed(pack2(s[i][0], s[i][1]));
        p[i][1] = transposed(pack2(s[i][2], s[i][3]));
      }
      if (n + kStep > tile.seq.m) {
        // slots that the sequence does not have may hold anything, and P's zeros times
        // NaN are NaN
        for (int c = lane; c < kStep * DH / 8; c += 32) {
          const int r = c / (DH / 8), k = c % (DH / 8);
          if (n + r >= tile.seq.m)
            *reinterpret_cast<uint4*>(stage + F::kHalf + (k >> 3) * (kSlots * 128) +
                                      (warp * kStep + r) * 128 + (k & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk)
        if (16 * kk < a.dh) {
          uint32_t v[4];
          ldsm4_t(v, vb + v_at + (kk >> 2) * (kSlots * 128) + ((((2 * kk) & 7) ^ v_c) << 4));
#pragma unroll
          for (int i = 0; i < RT; ++i) mma_b16(o[kk][i], v, p[i][0], p[i][1]);
        }
    }
    __syncthreads();  // the stage has been read
    if (tid == 0 && j + F::kStages < steps) load(j + F::kStages);
  }
  if (__syncthreads_or(!ok)) {  // a timeout: wait for the copies under way
    if (tid == 0) {
      const uint64_t t0 = tc::globaltimer();
      for (int i = 0; i < F::kStages; ++i) {
        const int uses = (steps + F::kStages - 1 - i) / F::kStages;
        while (uses > 0 && !tc::mbar_try_wait(s_full + i, (uses - 1) & 1) &&
               tc::globaltimer() - t0 < tc::kWaitLimitNs) {
        }
      }
    }
    if (!a.cluster) return;  // (else the others still read this CTA's shared memory)
  }
  // ---- the warps' sums
  float* acc = reinterpret_cast<float*>(smem);  // [kW][kRows][DH]
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[i][e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int r = 8 * i + 2 * q + e;
      if (g == 0) {
        s_m[warp][r] = mx[i][e];
        s_l[warp][r] = x;
      }
#pragma unroll
      for (int d = 0; d < DH / 16; ++d) {
        acc[(warp * F::kRows + r) * DH + 16 * d + g] = o[d][i][e];
        acc[(warp * F::kRows + r) * DH + 16 * d + g + 8] = o[d][i][e + 2];
      }
    }
  attn_join_warps<__nv_bfloat16, DH, F::kRows, false>(a, tile, acc, &s_m[0][0], &s_l[0][0], &s_bad);
}

template <int DH, int RT>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
  using F = Few<DH, RT>;
  auto kern = k_attn_few<DH, RT>;
  static_assert(F::kBytes <= 227 * 1024 - 1024, "a CTA's shared memory");
  static_assert(kW * F::kRows * DH * 4 + 8 * F::kRows <= F::kQ, "the warps' sums");
  static DeviceOnce once;
  const cudaError_t e = allow_smem(kern, F::kBytes, once);
  if (e != cudaSuccess) return e;
  const long grid = a.tiles * a.Hkv * a.nsplit;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  CUtensorMap k, v;
  if (!attn_tmaps(a, kSlots, &k, &v)) return cudaErrorInvalidValue;
  return attn_launch(kern, (unsigned)grid, kThreads, F::kBytes, s, a, k, v);
}
template <int DH>
cudaError_t by_rows(const AttnArgs& a, cudaStream_t s) {
  return a.rows == 8 ? launch<DH, 1>(a, s) : launch<DH, 2>(a, s);
}

}  // namespace

cudaError_t attn_few_launch(const AttnArgs& a, cudaStream_t s) {
  if (a.dh <= 64) return by_rows<64>(a, s);
  return a.dh <= 128 ? by_rows<128>(a, s) : by_rows<256>(a, s);
}

}  // namespace ps
