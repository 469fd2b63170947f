// Attention over a 4-bit KV cache for many query rows a KV head, on the
// tcgen05 tensor cores.
//
// A CTA takes 256 rows (two tiles of 128) of one KV head against a share of
// its slots, 128 slots at a time.  16 warps:
//   0-3, 4-7  softmax of row tile 0 / 1: a thread a row.  Reads its 128 scores
//             from TMEM, keeps the running maximum and sum in registers, writes
//             P (f16) over the scores, rescales O in TMEM when it must
//   8-11      the slots: 4-bit codes from global memory (the next tile's are in
//             registers while this one is converted), exact f16 into shared
//             memory in the 128-byte-swizzled layout of both operands (K is
//             K-major for S = Q K^T, V is MN-major for O += P V, which is the
//             same placement)
//   12        issues the MMAs: S into 128 TMEM columns a row tile, O into 128
//             more; P is the TMEM-resident A operand of P V
//   13-15     complete the warpgroup for the register split
// Order of the MMAs, per 128 slots j:  P0 V(j), S0(j+1), P1 V(j), S1(j+1): the
// softmax of one row tile runs under the two products of the other.  The
// commit that announces S(j+1) also says that P V(j) is done, so O may be
// rescaled then without another barrier.  O is rescaled only when a row's
// maximum has grown by 2^kGrow or more since the last time: until then P just
// carries a factor up to that.
// Every mbarrier wait is bounded (tc::mbar_wait); after a timeout the CTA waits
// for the MMAs it issued, frees TMEM and returns with the status word set.
#include "kv4.cuh"
#include "tc.cuh"

namespace ps {
namespace {

constexpr int kTcThreads = 512;
// Registers a thread after the split: 256 x 184 + 256 x 72 = 512 x 128, what
// the CTA is launched with.
constexpr int kLaunchRegs = 128;
constexpr int kTile = 128;          // slots a step; rows of a row tile
constexpr float kGrow = 8.f;        // log2 growth of a maximum before O is rescaled
constexpr float kTcShift = 4.f;     // log2 of the factor that P carries: P <= 2^12 in f16

template <int DH>
struct TcSmem {
  static constexpr uint32_t kOp = (DH / 64) * 16384u;  // 128 rows of DH f16
  static constexpr uint32_t kK = 2 * kOp,  // Q at 0
                             kV = 4 * kOp, kPos = 6 * kOp;
  static constexpr uint32_t kPar = kPos + 4 * kTile * 4;
  static constexpr uint32_t kBar = kPar + 256 * sizeof(RowPar);
  static constexpr size_t kBytes = 1024 + kBar + 256;
};

// Byte offset of 16-byte chunk c (of DH / 8) of row r in an operand.
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return (uint32_t)(c >> 3) * 16384u + (uint32_t)r * 128u + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}

// D(tmem) (+)= A . B, f16 operands: A from shared memory, or from TMEM.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  tc::mma_bf16(d, a, b, idesc, acc);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// f16 operands, fp32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn) {
  return tc::idesc_bf16(128, N, b_mn) & ~((1u << 7) | (1u << 10));
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
// The row as f16 into row r of an operand: 16-byte chunks, eight elements each,
// two to a scale.
template <int DH>
__device__ __forceinline__ void put_row(uint8_t* op, int r, const RawRow<DH>& v) {
#pragma unroll
  for (int c = 0; c < DH / 8; ++c) {
    const uint4& q = v.c[c / 4];
    const uint32_t w = c % 4 == 0 ? q.x : c % 4 == 1 ? q.y : c % 4 == 2 ? q.z : q.w;
    const __half2 s = e4m3_pair(((c < 8 ? v.s.x : v.s.y) >> (8 * ((c / 2) & 3))) & 0xffu);
    uint32_t h[4];
    e2m1x8_f16(w, h);
    uint4 o;
    o.x = h2_bits(__hmul2(h2_of(h[0]), s));
    o.y = h2_bits(__hmul2(h2_of(h[1]), s));
    o.z = h2_bits(__hmul2(h2_of(h[2]), s));
    o.w = h2_bits(__hmul2(h2_of(h[3]), s));
    *reinterpret_cast<uint4*>(op + sw128(r, c)) = o;
  }
}

// 256 query rows as f16 operands, with their constants: DH / 8 lanes a row.
template <int DH>
__device__ __forceinline__ void stage_queries(const Kv4AttnArgs& a, int b, int hkv, int m0,
                                              uint8_t* qs, RowPar* par) {
  constexpr int LN = DH / 8;                    // lanes a row
  constexpr int RP = kTcThreads / LN;           // rows a pass
  const int sub = threadIdx.x % LN, tid_lane = threadIdx.x & 31;
#pragma unroll 2
  for (int r = threadIdx.x / LN; r < 2 * kTile; r += RP) {
    const int m = m0 + r;
    float x[8];
    RowPar p{0.f, 0.f, 0, 0, 0, 0.f};
    if (m < a.M) {
      const int t = m / a.G, h = hkv * a.G + m % a.G;
      const long tok = (long)b * a.T + t;
      load16(static_cast<const __nv_bfloat16*>(a.Q) + tok * a.q_ld + (long)h * DH + sub * 8, x);
      p.slope = a.slope != nullptr ? a.slope[h] : 0.f;
      p.lo = a.span != nullptr ? a.span[2 * tok] : 0;
      p.hi = a.span != nullptr ? a.span[2 * tok + 1] : INT32_MAX;
      p.qpos = a.qpos != nullptr ? a.qpos[tok] : 0;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
    const uint32_t mask = (uint32_t)((1ull << LN) - 1) << (tid_lane & ~(LN - 1));
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(mask, mx, o));
    float up;
    row_scale(mx, a.scale, &up, &p.f);
    if (sub == 0) par[r] = p;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = h2_bits(__floats2half2_rn(x[2 * e] * up, x[2 * e + 1] * up));
    *reinterpret_cast<uint4*>(qs + (r / kTile) * TcSmem<DH>::kOp + sw128(r % kTile, sub)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// GEN: capped scores, a distance bias or explicit positions.
template <int DH, bool GEN>
__global__ void __launch_bounds__(kTcThreads, 1)
k_kv4_attn_tc(const __grid_constant__ Kv4AttnArgs a) {
  using SM = TcSmem<DH>;
  pdl_prologue();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  int* pos_ring = reinterpret_cast<int*>(smem + SM::kPos);  // [4][128]
  RowPar* par = reinterpret_cast<RowPar*>(smem + SM::kPar);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + SM::kBar);
  uint64_t *k_empty = k_full + 2, *v_full = k_full + 4, *v_empty = k_full + 6;
  uint64_t *s_full = k_full + 8, *p_full = k_full + 10, *o_full = k_full + 12, *drain = k_full + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(k_full + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_range = reinterpret_cast<int*>(tmem_slot + 2);  // lo, hi; per row tile lo_all, hi_all

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = blockIdx.x % a.nsplit;
  const int tile = blockIdx.x / a.nsplit % a.ntile;
  const int bh = blockIdx.x / a.nsplit / a.ntile;
  const int b = bh / a.Hkv, hkv = bh % a.Hkv, m0 = tile * 2 * kTile;
  const bool two = a.M - m0 > kTile;  // the second row tile holds rows
  const int len = min(max(a.len != nullptr ? a.len[b] : a.Ncache, 0), a.Ncache);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(k_full + i, 4);
      tc::mbar_init(k_empty + i, 1);
      tc::mbar_init(v_full + i, 4);
      tc::mbar_init(v_empty + i, 1);
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(p_full + i, 4);
      tc::mbar_init(o_full + i, 1);
    }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    s_range[0] = INT32_MAX;
    s_range[1] = INT32_MIN;
    s_range[2] = s_range[4] = INT32_MIN;
    s_range[3] = s_range[5] = INT32_MAX;
    tc::fence_mbar_init();
  }
  if (warp == 12) tc::tmem_alloc(tmem_slot, 512);
  stage_queries<DH>(a, b, hkv, m0, smem, par);
  tc::fence_proxy_async_smem();
  __syncthreads();
  if (tid < 2 * kTile && m0 + tid < a.M) {
    // slots some row sees, and slots every row of a row tile sees
    if (par[tid].lo < par[tid].hi) {
      atomicMin(&s_range[0], par[tid].lo);
      atomicMax(&s_range[1], par[tid].hi);
    }
    atomicMax(&s_range[2 + 2 * (tid / kTile)], par[tid].lo);
    atomicMin(&s_range[3 + 2 * (tid / kTile)], par[tid].hi);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const bool by_pos = GEN && a.kpos != nullptr;
  int n_lo = 0, n_hi = len;
  if (!by_pos) {
    n_lo = max(0, s_range[0]);
    n_hi = min(len, s_range[1]);
  }
  if (n_lo >= n_hi) {
    n_lo = n_hi = 0;
  } else {
    const int share = ceil_div(ceil_div(n_hi - n_lo, kTile), a.nsplit) * kTile;
    n_lo = min((long)n_hi, n_lo + (long)split * share);
    n_hi = min((long)n_hi, (long)n_lo + share);
  }
  const int nt = ceil_div(n_hi - n_lo, kTile);

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int g = warp >> 2, r = tid;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + g * 128;
    const uint32_t o_col = tmem + lane_base + 256 + g * 128;
    const RowPar rp = par[r];
    const int all_lo = by_pos ? INT32_MAX : s_range[2 + 2 * g];
    const int all_hi = min(len, s_range[3 + 2 * g]);
    const float f2 = GEN ? 1.f : rp.f * kLog2e;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    if (g == 0 || two) {
      for (int j = 0; j < nt; ++j) {
        const int n0 = n_lo + j * kTile;
        if (!tc::mbar_wait(s_full + g, j & 1, a.status, abort_flag)) { ok = false; break; }
        tc::fence_after_sync();
        float s[128];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tc::tmem_ld32_nowait(s_col + 32 * q, reinterpret_cast<uint32_t*>(s) + 32 * q);
        tc::tmem_wait_ld();
        if constexpr (GEN) {
          const int* ps = pos_ring + (j & 3) * kTile;
#pragma unroll
          for (int c = 0; c < 128; ++c) {
            const int pos = by_pos ? ps[c] : n0 + c;
            s[c] = kv4_score<false>(a, s[c], rp.f, rp.slope, rp.qpos, pos) * kLog2e;
            if (n0 + c >= len || pos < rp.lo || pos >= rp.hi) s[c] = -INFINITY;
          }
        } else if (n0 < all_lo || n0 + kTile > all_hi) {
          // columns [lo, hi) of this tile are seen
          const int lo = min(max((long)rp.lo - n0, 0L), 128L);
          const int hi = (int)min(max((long)min(rp.hi, len) - n0, 0L), 128L);
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c < lo || c >= hi) s[c] = -INFINITY;
        }
        float mx = s[0];
#pragma unroll
        for (int c = 1; c < 128; ++c) mx = fmaxf(mx, s[c]);
        const float m_tile = mx * f2;
        const bool grow = m_tile > m_used + kGrow;
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? m_tile : m_used;
          const float corr = grow ? exp2_approx(m_used - m_new) : 1.f;
          if (j > 0) {
#pragma unroll 1
            for (int q = 0; q < DH / 32; ++q) {
              uint32_t o[32];
              tc::tmem_ld32_nowait(o_col + 32 * q, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * corr);
              tc::tmem_st32(o_col + 32 * q, o);
            }
          }
          l *= corr;
          m_used = m_new;
        }
        const float base = m_used == -INFINITY ? 0.f : m_used - kTcShift;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float p0 = exp2_approx(fmaf(s[64 * q + 2 * c], f2, -base));
            const float p1 = exp2_approx(fmaf(s[64 * q + 2 * c + 1], f2, -base));
            sum[2 * (c & 1)] += p0;
            sum[2 * (c & 1) + 1] += p1;
            pk[c] = h2_bits(__floats2half2_rn(p0, p1));
          }
          tc::tmem_st32(s_col + 32 * q, pk);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + g);
      }
      // the finished row
      const int m = m0 + r;
      if (ok && nt > 0) {
        ok = tc::mbar_wait(o_full + g, 0, a.status, abort_flag);
        tc::fence_after_sync();
      }
      if (ok) {
        const float mx = m_used == -INFINITY ? -INFINITY : m_used - kTcShift + kPShift;
#pragma unroll 1
        for (int q = 0; q < DH / 32; ++q) {
          uint32_t o[32];
          if (nt > 0) {
            tc::tmem_ld32_nowait(o_col + 32 * q, o);  // warp-collective
            tc::tmem_wait_ld();
          }
          if (m < a.M) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              float4 v = make_float4(__uint_as_float(o[c]), __uint_as_float(o[c + 1]),
                                     __uint_as_float(o[c + 2]), __uint_as_float(o[c + 3]));
              if (l == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
              const int d = 32 * q + c;
              if (a.nsplit > 1) {
                const size_t at = ((size_t)bh * a.M + m) * a.nsplit + split;
                *reinterpret_cast<float4*>(a.po + at * DH + d) = v;
                if (d == 0) {
                  a.pml[2 * at] = mx;
                  a.pml[2 * at + 1] = l;
                }
              } else {
                kv4_finish<false>(a, b, hkv, m, DH, d, v, mx, l);
              }
            }
          }
        }
      }
    }
    tc::fence_before_sync();
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int p = tid - 256, last = a.Ncache - 1;
    const uint8_t* kc = a.kcode + (long)bh * a.Ncache * (DH / 2);
    const uint8_t* ks = a.kscale + (long)bh * a.Ncache * (DH / 16);
    const uint8_t* vc = a.vcode + (long)bh * a.Ncache * (DH / 2);
    const uint8_t* vs = a.vscale + (long)bh * a.Ncache * (DH / 16);
    const int32_t* kpos = a.kpos != nullptr ? a.kpos + (long)bh * a.Ncache : nullptr;
    RawRow<DH> rk, rv;
    if (nt > 0) {
      const int slot = min(n_lo + p, last);
      load_row<DH>(kc, ks, slot, rk);
      load_row<DH>(vc, vs, slot, rv);
    }
    for (int j = 0; j < nt; ++j) {
      const int st = j & 1;
      const uint32_t ph = ((j >> 1) & 1) ^ 1;
      const int next = (int)min((long)n_lo + (long)(j + 1) * kTile + p, (long)last);
      if (!tc::mbar_wait(k_empty + st, ph, a.status, abort_flag)) break;
      if (by_pos) pos_ring[(j & 3) * kTile + p] = kpos[min(n_lo + j * kTile + p, last)];
      put_row<DH>(smem + SM::kK + st * SM::kOp, p, rk);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(k_full + st);
      if (j + 1 < nt) load_row<DH>(kc, ks, next, rk);
      if (!tc::mbar_wait(v_empty + st, ph, a.status, abort_flag)) break;
      put_row<DH>(smem + SM::kV + st * SM::kOp, p, rv);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(v_full + st);
      if (j + 1 < nt) load_row<DH>(vc, vs, next, rv);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 12 && lane == 0 && nt > 0) {
      constexpr uint32_t kIdQK = idesc_f16(128, false), kIdPV = idesc_f16(DH, true);
      const uint32_t qs = tc::smem_u32(smem), kb = qs + SM::kK, vb = qs + SM::kV;
      bool ok = true;
      auto qk = [&](int g, int j) {
        const uint32_t q = qs + g * SM::kOp, k = kb + (j & 1) * SM::kOp;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          const uint32_t off = (kk / 4) * 16384u + (kk % 4) * 32u;
          mma_ss(tmem + g * 128, tc::desc_sw128(q + off, 16, 1024),
                 tc::desc_sw128(k + off, 16, 1024), kIdQK, kk > 0);
        }
        tc::mma_commit(s_full + g);
      };
      auto pv = [&](int g, int j) {
        const uint32_t v = vb + (j & 1) * SM::kOp;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_ts(tmem + 256 + g * 128, tmem + g * 128 + kk * 8,
                 tc::desc_sw128(v + kk * 2048u, 16384, 1024), kIdPV, j > 0 || kk > 0);
      };
      const int ng = two ? 2 : 1;
      ok = tc::mbar_wait(k_full, 0, a.status, abort_flag);
      tc::fence_after_sync();
      if (ok) {
        for (int g = 0; g < ng; ++g) qk(g, 0);
        tc::mma_commit(k_empty);
      }
      for (int j = 0; ok && j < nt; ++j) {
        const uint32_t ph = (j >> 1) & 1;
        if (!tc::mbar_wait(v_full + (j & 1), ph, a.status, abort_flag)) { ok = false; break; }
        for (int g = 0; g < ng; ++g) {
          if (!tc::mbar_wait(p_full + g, j & 1, a.status, abort_flag)) { ok = false; break; }
          tc::fence_after_sync();
          pv(g, j);
          if (g == ng - 1) tc::mma_commit(v_empty + (j & 1));
          if (j + 1 < nt) {
            if (g == 0) {
              if (!tc::mbar_wait(k_full + ((j + 1) & 1), ((j + 1) >> 1) & 1, a.status,
                                 abort_flag)) { ok = false; break; }
              tc::fence_after_sync();
            }
            qk(g, j + 1);
            if (g == ng - 1) tc::mma_commit(k_empty + ((j + 1) & 1));
          } else {
            tc::mma_commit(o_full + g);
          }
        }
      }
      if (!ok) {  // wait for the MMAs already issued before TMEM is freed
        tc::mma_commit(drain);
        const uint64_t t0 = tc::globaltimer();
        while (!tc::mbar_try_wait(drain, 0) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 12) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int DH, bool GEN>
cudaError_t launch_tc(const Kv4AttnArgs& a, cudaStream_t s) {
  auto kern = k_kv4_attn_tc<DH, GEN>;
  static bool attr_set = false;
  if (!attr_set) {
    // the register split waits for ever if the CTA is launched with fewer
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kLaunchRegs) return cudaErrorLaunchOutOfResources;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)TcSmem<DH>::kBytes);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  const long grid = (long)a.B * a.Hkv * a.ntile * a.nsplit;
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kTcThreads), TcSmem<DH>::kBytes, s, a);
}

}  // namespace

cudaError_t kv4_attn_tc_launch(const Kv4AttnArgs& a, cudaStream_t s) {
  const bool gen = a.cap > 0.f || a.slope != nullptr || a.kpos != nullptr;
  if (a.dh == 64) return gen ? launch_tc<64, true>(a, s) : launch_tc<64, false>(a, s);
  if (a.dh == 128) return gen ? launch_tc<128, true>(a, s) : launch_tc<128, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace ps
