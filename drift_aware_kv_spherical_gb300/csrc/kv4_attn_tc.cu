// Attention over a 4-bit KV cache for many query rows a KV head, on the
// tcgen05 tensor cores.
//
// A CTA takes 256 rows (two tiles of 128) of one KV head against a share of
// its slots, 128 slots at a time.  13 warps:
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

constexpr int kTcThreads = 416;
constexpr int kTile = 128;          // slots a step; rows of a row tile
constexpr float kGrow = 8.f;        // log2 growth of a maximum before O is rescaled
constexpr float kTcShift = 4.f;     // log2 of the factor that P carries: P <= 2^12 in f16

template <int DH>
struct TcSmem {
  static constexpr uint32_t kOp = (DH / 64) * 16384u;  // 128 rows of DH f16
  static constexpr uint32_t kK = 2 * kOp,  // Q at 0
                             kV = 4 * kOp, kPos = 6 * kOp;
  static constexpr uint32_t kFac = kPos + 4 * kTile * 4;
  static constexpr uint32_t kBar = kFac + 256 * 4;
  static constexpr size_t kBytes = 1024 + kBar + 256;
};

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

// 256 query rows as f16 operands and their score factors, DH / 8 lanes a row;
// all of a thread's rows are loaded before the first is used.
template <int DH>
__device__ __forceinline__ void stage_queries(const Kv4AttnArgs& a, int b, int hkv, int m0,
                                              uint8_t* qs, float* fac) {
  constexpr int LN = DH / 8;                          // lanes a row
  constexpr int RP = kTcThreads / LN;                 // rows a pass
  constexpr int NP = (2 * kTile + RP - 1) / RP;       // passes
  const int sub = threadIdx.x % LN;
  uint4 raw[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = threadIdx.x / LN + i * RP, m = m0 + r;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < 2 * kTile && m < a.M) {
      const int t = m / a.G, h = hkv * a.G + m % a.G;
      raw[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.Q) +
                                                    ((long)b * a.T + t) * a.q_ld + (long)h * DH +
                                                    sub * 8));
    }
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = threadIdx.x / LN + i * RP;
    float x[8];
    unpack16(raw[i], x, __nv_bfloat16{});
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float up, f;
    row_scale(mx, a.scale, &up, &f);
    if (r >= 2 * kTile) continue;
    if (sub == 0) fac[r] = f;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = h2_bits(__floats2half2_rn(x[2 * e] * up, x[2 * e + 1] * up));
    *reinterpret_cast<uint4*>(qs + (r / kTile) * TcSmem<DH>::kOp + sw128(r % kTile, sub)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The constants of a softmax thread's row.
struct TcRow {
  float f;                // score factor of a raw product
  float slope2;           // distance bias in log2 units
  int lo, hi, qpos;
};

// s[0..63]: raw products of 64 slots from n0 on -> log2-unit scores (GEN), and
// -inf where the row does not see the slot.  pos: explicit positions, or null.
template <bool GEN>
__device__ __forceinline__ void tc_scores(const Kv4AttnArgs& a, float* s, const TcRow& row,
                                          int n0, int len, bool masked, const int* pos) {
  if constexpr (GEN) {
    if (a.cap > 0.f) {
      const float fy = row.f * a.inv_cap, cap2 = a.cap * kLog2e;
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < 64; ++c) {
        s[c] *= fy;
        top = fmaxf(top, fabsf(s[c]));
      }
      if (__all_sync(0xffffffffu, top <= 0.4f)) {
        // tanh's series to y^11: the next term is under 2^-23 of y here
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          const float y = s[c], z = y * y;
          float q = fmaf(z, -1382.f / 155925.f, 62.f / 2835.f);
          q = fmaf(z, q, -17.f / 315.f);
          q = fmaf(z, q, 2.f / 15.f);
          q = fmaf(z, q, -1.f / 3.f);
          q = z * q;
          s[c] = cap2 * fmaf(y, q, y);
        }
      } else {
        // tanh y = 1 - 2 / (e^2y + 1): absolute error about 1e-7
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          const float e = exp2_approx(s[c] * (2.f * kLog2e));
          s[c] = cap2 * fmaf(-2.f, rcp_approx(e + 1.f), 1.f);
        }
      }
    } else {
      const float f2 = row.f * kLog2e;
#pragma unroll
      for (int c = 0; c < 64; ++c) s[c] *= f2;
    }
    if (a.slope != nullptr) {
      if (pos == nullptr) {
        const float dq = (float)(row.qpos - n0);
#pragma unroll
        for (int c = 0; c < 64; ++c) s[c] = fmaf(-row.slope2, fabsf(dq - (float)c), s[c]);
      } else {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          s[c] = fmaf(-row.slope2, fabsf((float)(row.qpos - pos[c])), s[c]);
      }
    }
    if (masked && pos != nullptr) {
#pragma unroll
      for (int c = 0; c < 64; ++c)
        if (n0 + c >= len || pos[c] < row.lo || pos[c] >= row.hi) s[c] = -INFINITY;
      return;
    }
  }
  if (masked) {  // columns [lo, hi) are seen
    const int lo = (int)min(max((long)row.lo - n0, 0L), 64L);
    const int hi = (int)min(max((long)min(row.hi, len) - n0, 0L), 64L);
#pragma unroll
    for (int c = 0; c < 64; ++c)
      if (c < lo || c >= hi) s[c] = -INFINITY;
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
  float* fac = reinterpret_cast<float*>(smem + SM::kFac);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + SM::kBar);
  uint64_t *k_empty = k_full + 2, *v_full = k_full + 4, *v_empty = k_full + 6;
  uint64_t *s_full = k_full + 8, *o_full = k_full + 10, *drain = k_full + 12;
  uint64_t* p_full = k_full + 13;  // [row tile][half of the slots]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(k_full + 17);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_range = reinterpret_cast<int*>(tmem_slot + 2);  // lo, hi; per row tile lo_all, hi_all

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler too
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
      tc::mbar_init(p_full + 2 + i, 4);
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
  TcRow row{0.f, 0.f, 0, 0, 0};
  const int m = m0 + tid;  // a softmax thread's row
  if (tid < 2 * kTile && m < a.M) {
    const long tok = (long)b * a.T + m / a.G;
    if (a.slope != nullptr) row.slope2 = a.slope[hkv * a.G + m % a.G] * kLog2e;
    row.hi = INT32_MAX;
    if (a.span != nullptr) {
      row.lo = a.span[2 * tok];
      row.hi = a.span[2 * tok + 1];
    }
    if (a.qpos != nullptr) row.qpos = a.qpos[tok];
  }
  stage_queries<DH>(a, b, hkv, m0, smem, fac);
  tc::fence_proxy_async_smem();
  __syncthreads();
  if (tid < 2 * kTile && m < a.M) {
    // slots some row sees, and slots every row of a row tile sees
    const int g = tid / kTile;
    const bool any = row.lo < row.hi;
    const uint32_t act = __activemask();
    const int lo = __reduce_min_sync(act, any ? row.lo : INT32_MAX);
    const int hi = __reduce_max_sync(act, any ? row.hi : INT32_MIN);
    const int lo_all = __reduce_max_sync(act, row.lo), hi_all = __reduce_min_sync(act, row.hi);
    if (lane == 0) {  // a warp's first row is there if any is
      atomicMin(&s_range[0], lo);
      atomicMax(&s_range[1], hi);
      atomicMax(&s_range[2 + 2 * g], lo_all);
      atomicMin(&s_range[3 + 2 * g], hi_all);
    }
    row.f = fac[tid];
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
    const int g = warp >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + g * 128;
    const uint32_t o_col = tmem + lane_base + 256 + g * 128;
    const int all_lo = by_pos ? INT32_MAX : s_range[2 + 2 * g];
    const int all_hi = min(len, s_range[3 + 2 * g]);
    const float f2 = GEN ? 1.f : row.f * kLog2e;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    if (g == 0 || two) {
      for (int j = 0; j < nt; ++j) {
        const int n0 = n_lo + j * kTile;
        const bool masked = n0 < all_lo || n0 + kTile > all_hi;
        const int* ps = by_pos ? pos_ring + (j & 3) * kTile : nullptr;
        if (!tc::mbar_wait(s_full + g, j & 1, a.status, abort_flag)) { ok = false; break; }
        tc::fence_after_sync();
        // The tile's maximum, 64 slots at a time; scores that are more than
        // raw products go back to TMEM for the second pass.
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // chains
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float s[64];
          tc::tmem_ld32_nowait(s_col + 64 * h, reinterpret_cast<uint32_t*>(s));
          tc::tmem_ld32_nowait(s_col + 64 * h + 32, reinterpret_cast<uint32_t*>(s) + 32);
          tc::tmem_wait_ld();
          if (GEN || masked) {
            tc_scores<GEN>(a, s, row, n0 + 64 * h, len, masked, by_pos ? ps + 64 * h : nullptr);
            tc::tmem_st32(s_col + 64 * h, reinterpret_cast<uint32_t*>(s));
            tc::tmem_st32(s_col + 64 * h + 32, reinterpret_cast<uint32_t*>(s) + 32);
          }
#pragma unroll
          for (int c = 0; c < 64; ++c) m4[c & 3] = fmaxf(m4[c & 3], s[c]);
        }
        if (GEN || masked) tc::tmem_wait_st();
        const float m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * f2;
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
        // P over the scores: the first half lies on scores already read
        const float base = m_used == -INFINITY ? 0.f : m_used - kTcShift;
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float s[64];
          tc::tmem_ld32_nowait(s_col + 64 * h, reinterpret_cast<uint32_t*>(s));
          tc::tmem_ld32_nowait(s_col + 64 * h + 32, reinterpret_cast<uint32_t*>(s) + 32);
          tc::tmem_wait_ld();
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float p0 = exp2_approx(fmaf(s[2 * c], f2, -base));
            const float p1 = exp2_approx(fmaf(s[2 * c + 1], f2, -base));
            s4[2 * (c & 1)] += p0;
            s4[2 * (c & 1) + 1] += p1;
            pk[c] = h2_bits(__floats2half2_rn(p0, p1));
          }
          tc::tmem_st32(s_col + 32 * h, pk);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(p_full + 2 * g + h);  // half of P V may start
        }
        l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
      }
      if (ok && nt > 0) {
        ok = tc::mbar_wait(o_full + g, 0, a.status, abort_flag);
        tc::fence_after_sync();
      }
      // The finished rows: through shared memory (Q's, no longer read), 256
      // bytes a row at a time, so that a warp stores whole rows.
      if (ok) {
        const bool part = a.nsplit > 1;
        const float mx = m_used == -INFINITY ? -INFINITY : m_used - kTcShift + kPShift;
        const long orow = ((long)b * a.T + m / a.G) * a.Hq + hkv * a.G + m % a.G;
        const long prow = ((long)bh * a.M + m) * a.nsplit + split;
        if (m < a.M) {
          if (part) {
            a.pml[2 * prow] = mx;
            a.pml[2 * prow + 1] = l;
          } else if (a.lse != nullptr) {
            a.lse[orow] = row_lse(mx, l);
          }
        }
        const float inv = part ? 1.f : l == 0.f ? 0.f : a.vmul / l;
        uint8_t* buf = smem + warp * 8192;  // 32 rows
        const int per = part ? 64 : DH;     // elements a row at a time
        const int lanes = part ? 16 : DH / 8;
#pragma unroll 1
        for (int d0 = 0; d0 < DH; d0 += per) {
#pragma unroll 1
          for (int q = 0; q < per / 32; ++q) {
            uint32_t o[32];
            if (nt > 0) {
              tc::tmem_ld32_nowait(o_col + d0 + 32 * q, o);
              tc::tmem_wait_ld();
            }
#pragma unroll
            for (int c = 0; c < 32; ++c)  // nothing seen: 0, whatever TMEM holds
              o[c] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[c]) * inv);
            if (part) {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(buf + lane * 256 + (((8 * q + c) ^ (lane & 15)) << 4)) =
                    make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __nv_bfloat162 v =
                      __floats2bfloat162_rn(__uint_as_float(o[8 * c + 2 * e]),
                                            __uint_as_float(o[8 * c + 2 * e + 1]));
                  w[e] = *reinterpret_cast<const uint32_t*>(&v);
                }
                *reinterpret_cast<uint4*>(buf + lane * 256 + (((4 * q + c) ^ (lane & 15)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          __syncwarp();
          for (int i = 0; i < lanes; ++i) {
            const int rr = i * (32 / lanes) + lane / lanes, c = lane % lanes;
            const long at = __shfl_sync(0xffffffffu, part ? prow : orow, rr);
            const bool in = __shfl_sync(0xffffffffu, m < a.M, rr);
            const uint4 v =
                *reinterpret_cast<const uint4*>(buf + rr * 256 + ((c ^ (rr & 15)) << 4));
            if (in) {
              if (part) reinterpret_cast<uint4*>(a.po + at * DH + d0)[c] = v;
              else reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) + at * DH)[c] = v;
            }
          }
          __syncwarp();
        }
      }
    }
    tc::fence_before_sync();
  } else if (warp < 12) {
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
    if (warp == 12 && nt > 0) {
      constexpr uint32_t kIdQK = idesc_f16(128, false), kIdPV = idesc_f16(DH, true);
      const uint32_t qs = tc::smem_u32(smem), kb = qs + SM::kK, vb = qs + SM::kV;
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
      auto pv = [&](int g, int j, int half) {
        const uint32_t v = vb + (j & 1) * SM::kOp;
#pragma unroll
        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
          mma_ts(tmem + 256 + g * 128, tmem + g * 128 + kk * 8,
                 tc::desc_sw128(v + kk * 2048u, 16384, 1024), kIdPV, j > 0 || kk > 0);
      };
      const int ng = two ? 2 : 1;
      bool ok = tc::mbar_wait(k_full, 0, a.status, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      if (ok && elect_one()) {
        for (int g = 0; g < ng; ++g) qk(g, 0);
        tc::mma_commit(k_empty);
      }
      for (int j = 0; ok && j < nt; ++j) {
        const int jn = j + 1, stn = jn & 1;
        ok = tc::mbar_wait(v_full + (j & 1), (j >> 1) & 1, a.status, abort_flag);
        for (int g = 0; ok && g < ng; ++g) {
          ok = tc::mbar_wait(p_full + 2 * g, j & 1, a.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          tc::fence_after_sync();
          if (ok && elect_one()) pv(g, j, 0);
          __syncwarp();
          if (ok) ok = tc::mbar_wait(p_full + 2 * g + 1, j & 1, a.status, abort_flag);
          if (ok && g == 0 && jn < nt)
            ok = tc::mbar_wait(k_full + stn, (jn >> 1) & 1, a.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          tc::fence_after_sync();
          if (ok && elect_one()) {
            pv(g, j, 1);
            if (g == ng - 1) tc::mma_commit(v_empty + (j & 1));
            if (jn < nt) {
              qk(g, jn);
              if (g == ng - 1) tc::mma_commit(k_empty + stn);
            } else {
              tc::mma_commit(o_full + g);
            }
          }
          __syncwarp();
        }
      }
      if (!__all_sync(0xffffffffu, ok)) {  // wait for the MMAs issued before TMEM is freed
        if (elect_one()) tc::mma_commit(drain);
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
