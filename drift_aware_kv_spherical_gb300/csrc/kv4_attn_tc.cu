// Attention over a 4-bit KV cache for many query rows a KV head, on the
// tcgen05 tensor cores.
//
// A CTA an SM takes item after item: 256 rows (two tiles of 128) of one KV head
// against a share of its slots, 128 slots a step.  14 warps:
//   0-3, 4-7  softmax of row tile 0 / 1: a thread a row.  Reads its 128 scores
//             from TMEM, keeps the running maximum and sum in registers, writes
//             P (f16) over the scores, 64 slots at a time, and rescales O in
//             TMEM when it must.  Also stages the item's queries and stores its
//             rows, each row tile for itself, so that one finishes and begins
//             an item while the other still has the tensor cores
//   8-11      the slots: 4-bit codes from global memory (the next step's are in
//             registers while this one is converted, across items too), exact
//             f16 into shared memory in the 128-byte-swizzled layout of both
//             operands (K is K-major for S = Q K^T, V is MN-major for O += P V,
//             which is the same placement)
//   12        issues the MMAs: S into 128 TMEM columns a row tile, O into 128
//             more; P is the TMEM-resident A operand of P V
//   13        claims the next item and works out what it is
// Order of the MMAs, per step j:  P0 V(j), S0(j+1), P1 V(j), S1(j+1): the
// softmax of one row tile runs under the two products of the other, and P V of
// its first 64 slots under its second 64 exponentials.  The commit that
// announces S(j+1) also says that P V(j) is done, so O may be rescaled then
// without another barrier.  O is rescaled only when a row's maximum has grown
// by 2^kGrow or more since the last time: until then P just carries a factor up
// to that.
//
// What bounds it: a step's chain of product, two passes over 64 scores from TMEM
// and P back, of which two row tiles hide only half.  4096 rows x 32 heads x 2 on
// 4096 slots 419 us, 1.31 PFLOP/s, 68 % of a large library product's rate; the
// tensor cores are busy half the time, the exponentials' unit a quarter.  Caps and
// biases lengthen the chain: 2048 rows x 32 heads on 4096 slots 122 us plain, 191
// capped, 241 with a bias too.  Explicit positions are masked slot by slot: causal
// 100 us, 563 with them.
// Every mbarrier wait is bounded (tc::mbar_wait); after a timeout the CTA waits
// for the MMAs it issued, frees TMEM and returns with the status word set.
#include "kv4_tc.cuh"

namespace ps {
namespace {

constexpr int kTcThreads = 448;
constexpr int kRing = 4;            // items known and not yet taken by every warp
constexpr int kTile = 128;          // slots a step; rows of a row tile
constexpr float kGrow = 8.f;        // log2 growth of a maximum before O is rescaled
constexpr float kTcShift = 4.f;     // log2 of the factor that P carries: P <= 2^12 in f16
// A maximum from which on scores are rounded before it is subtracted from them: it
// is rounded itself, and by 2^-24 of it P would leave f16.
constexpr float kHuge = 0x1p22f;

template <int DH>
struct TcSmem {
  static constexpr uint32_t kOp = (DH / 64) * 16384u;  // 128 rows of DH f16
  static constexpr uint32_t kK = 2 * kOp,  // Q at 0
                            kV = 4 * kOp, kPos = 6 * kOp;
  static constexpr uint32_t kRow = kPos + 4 * kTile * 4;           // TcRow [256]
  static constexpr uint32_t kWork = kRow + 2 * kTile * 24;         // TcWork [8 warps]
  static constexpr uint32_t kBar = kWork + 8 * 32;
  static constexpr uint32_t kItems = kBar + 256;  // TcWork [kRing], then a claim's 16 bytes
  static constexpr size_t kBytes = 1024 + kItems + kRing * 32 + 16;
};

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

// ---------------------------------------------------------------- work items
// An item: 256 rows of one KV head against one share of its slots; an item is a
// CTA of the grid.  The CTAs that run claim those not yet begun, one ahead, so
// that items of unequal length (spans, ragged lengths) leave no SM idle: packed
// documents of six random lengths 91 us on average, 103 with every 152nd item in
// turn.  The last rows of all heads come first, which causal spans make the
// longest: 2048 rows x 32 heads on 4096 slots 99 us, 120 head by head.
struct TcWork {
  int item, split, tile, hkv, b;
  int n_lo, nt;  // first slot, steps
  int two;       // the second row tile holds rows
};

// A claim asked for: 16 bytes at `to` and `bar` completed.
__device__ __forceinline__ void claim_ask(uint4* to, uint64_t* bar) {
  tc::mbar_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(tc::smem_u32(to)),
      "r"(tc::smem_u32(bar))
      : "memory");
}
// The claimed item, or -1: none is left.
__device__ __forceinline__ int claim_get(const uint4* from) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(tc::smem_u32(from))
      : "memory");
  return got ? (int)x : -1;
}

// The slots of w, for a whole warp: those within the rows' spans.
__device__ __forceinline__ void tc_slots(const Kv4AttnArgs& a, TcWork& w) {
  const int m0 = w.tile * 2 * kTile;
  w.two = a.M - m0 > kTile;
  int n_lo = 0;
  int n_hi = min(max(a.len != nullptr ? __ldg(a.len + w.b) : a.Ncache, 0), a.Ncache);
  if (a.span != nullptr && a.kpos == nullptr) {
    const int t0 = row_token(a, m0), t1 = row_token(a, min(m0 + 2 * kTile, a.M) - 1);
    int lo = INT32_MAX, hi = INT32_MIN;
    for (int t = t0 + (threadIdx.x & 31); t <= t1; t += 32) {
      const int2 x = row_span(a, (long)w.b * a.T + t);
      if (x.x < x.y) {
        lo = min(lo, x.x);
        hi = max(hi, x.y);
      }
    }
    n_lo = max(0, __reduce_min_sync(0xffffffffu, lo));
    n_hi = min(n_hi, __reduce_max_sync(0xffffffffu, hi));
  }
  if (n_lo >= n_hi) return;
  int n = n_hi - n_lo;
  w.n_lo = n_lo;
  if (a.nsplit > 1) {
    const int share = ceil_div(ceil_div(n, kTile), a.nsplit) * kTile;
    const int from = (int)min((long)n, (long)w.split * share);
    w.n_lo += from;
    n = min(n - from, share);
  }
  w.nt = (n + kTile - 1) / kTile;
}
__device__ __forceinline__ TcWork tc_item(const Kv4AttnArgs& a, int item) {
  TcWork w{item, 0, 0, 0, 0, 0, 0, 0};
  if (item < 0) return w;
  int n = item;
  w.split = n % a.nsplit;
  n /= a.nsplit;
  w.hkv = n % a.Hkv;
  n /= a.Hkv;
  w.b = n % a.B;
  w.tile = a.ntile - 1 - n / a.B;
  tc_slots(a, w);
  return w;
}

// The items of a CTA, for a warp of any role; warp 13 claims them and works out
// what they are.
struct TcItems {
  uint64_t *full, *empty;  // an item: known, taken by every warp
  const TcWork* ring;
  int n = 0;  // taken
  // the next item (.item -1: the end); false after a timeout
  __device__ __forceinline__ bool take(const Kv4AttnArgs& a, volatile int* abort_flag, TcWork* w) {
    const int k = n % kRing;
    const bool ok = tc::mbar_wait(full + k, (n / kRing) & 1, a.status, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return false;
    *w = ring[k];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(empty + k);
    ++n;
    return true;
  }
  __device__ __forceinline__ bool ready() const {
    return __all_sync(0xffffffffu, tc::mbar_test(full + n % kRing, (n / kRing) & 1));
  }
};

// ---------------------------------------------------------------- slots
__device__ __forceinline__ void l2_prefetch(const void* p, int bytes) {
  for (int o = 0; o < bytes; o += 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + o));
}

// The row as f16 into row r of an operand: 16-byte chunks, eight elements each,
// two to a scale, two scales to a conversion.
template <int DH>
__device__ __forceinline__ void put_row(uint8_t* op, int r, const RawRow<DH>& v) {
#pragma unroll
  for (int p = 0; p < DH / 32; ++p) {
    const uint32_t two = ((p < 2 ? v.s.x : v.s.y) >> (16 * (p & 1))) & 0xffffu;
    const uint32_t sc = h2_bits(e4m3x2_f16(two));
    const uint32_t w[4] = {v.c[p].x, v.c[p].y, v.c[p].z, v.c[p].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 s = h2_of(__byte_perm(sc, sc, i < 2 ? 0x1010u : 0x3232u));
      uint32_t h[4];
      e2m1x8_f16(w[i], h);
      uint4 o;
      o.x = h2_bits(__hmul2(h2_of(h[0]), s));
      o.y = h2_bits(__hmul2(h2_of(h[1]), s));
      o.z = h2_bits(__hmul2(h2_of(h[2]), s));
      o.w = h2_bits(__hmul2(h2_of(h[3]), s));
      *reinterpret_cast<uint4*>(op + sw128(r, 4 * p + i)) = o;
    }
  }
}

// ---------------------------------------------------------------- queries
// The lane's row (row r of the operand at qs) from bf16 to f16 in place; returns
// its score factor.  (Read from global memory by the lanes themselves, 32 rows a
// load, the same took three times as long.)
template <int DH>
__device__ __forceinline__ float stage_q(float scale, uint8_t* qs, int r) {
  uint4 v[DH / 8];
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int c = 0; c < DH / 8; ++c) v[c] = *reinterpret_cast<const uint4*>(qs + sw128(r, c));
  __nv_bfloat162 m2 = __floats2bfloat162_rn(0.f, 0.f);  // NaN elements do not count
#pragma unroll
  for (int c = 0; c < DH / 8; ++c) {
    const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
  }
  float up, f;
  row_scale(fmaxf(__low2float(m2), __high2float(m2)), scale, &up, &f);
#pragma unroll
  for (int c = 0; c < DH / 8; ++c) {
    float x[8];
    unpack16(v[c], x, __nv_bfloat16{});
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = h2_bits(__floats2half2_rn(x[2 * e] * up, x[2 * e + 1] * up));
    *reinterpret_cast<uint4*>(qs + sw128(r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return f;
}

// ---------------------------------------------------------------- scores
// The constants of a softmax thread's row.  They wait in shared memory, like the
// item: what is not read in every step would push the scores out of registers.
struct TcRow {
  float f;                // score factor of a raw product
  float slope2;           // distance bias, in units of the cap or log2 units
  int lo, hi, qpos, len;  // positions seen; the row's own; the sequence's slots
};
template <class T>
__device__ __forceinline__ void sm_put(volatile int* p, const T& x) {
  static_assert(sizeof(T) % 4 == 0, "words");
  const int* w = reinterpret_cast<const int*>(&x);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 4; ++i) p[i] = w[i];
}
template <class T>
__device__ __forceinline__ T sm_get(volatile int* p) {
  T x;
  int* w = reinterpret_cast<int*>(&x);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 4; ++i) w[i] = p[i];
  return x;
}
// Row m, token t of its sequence, query head h; nothing past the last row.
__device__ __forceinline__ TcRow tc_row(const Kv4AttnArgs& a, bool in, int b, int t, int h) {
  TcRow row{0.f, 0.f, 0, 0, 0, 0};
  row.len = min(max(a.len != nullptr ? __ldg(a.len + b) : a.Ncache, 0), a.Ncache);
  if (in) {
    const long tok = (long)b * a.T + t;
    if (a.slope != nullptr) row.slope2 = a.slope[h] * (a.cap > 0.f ? a.inv_cap : kLog2e);
    row.hi = INT32_MAX;
    if (a.span != nullptr) {
      row.lo = a.span[2 * tok];
      row.hi = a.span[2 * tok + 1];
    }
    if (a.qpos != nullptr) row.qpos = a.qpos[tok];
  }
  return row;
}

// What the rows of a softmax warp see of 64 slots.  A row that sees nothing at
// all has no say (its sum is dropped at the end).  Taken once an item, so that
// a step compares two numbers and does not vote.
enum TcScore { kPlain, kCap, kAny };
enum TcSeen { kNone, kSome, kAll };
struct TcRange {
  int any_lo, any_hi, all_lo, all_hi;  // slots that some, that every row sees
};
__device__ __forceinline__ TcRange tc_range(const TcRow& row) {
  const bool live = row.lo < row.hi;
  const int lo = max(row.lo, 0), hi = max(min(row.hi, row.len), 0);  // of slots: 64 less is one too
  TcRange r;
  r.any_lo = __reduce_min_sync(0xffffffffu, live ? lo : INT32_MAX);
  r.any_hi = __reduce_max_sync(0xffffffffu, live ? hi : INT32_MIN);
  r.all_lo = __reduce_max_sync(0xffffffffu, live ? lo : INT32_MIN);
  r.all_hi = __reduce_min_sync(0xffffffffu, live ? hi : INT32_MAX) - 64;  // of the first of 64
  return r;
}
__device__ __forceinline__ TcSeen tc_seen(const TcRange& r, int n0) {
  if (n0 >= r.any_hi || n0 <= r.any_lo - 64) return kNone;
  return n0 >= r.all_lo && n0 <= r.all_hi ? kAll : kSome;
}

// Capped scores: cap tanh(score / cap).
template <int C>
__device__ __forceinline__ float abs_max(const float* s) {
  float t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < C; c += 2)
    t4[(c >> 1) & 3] = max3(t4[(c >> 1) & 3], fabsf(s[c]), fabsf(s[c + 1]));
  return fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
}
// Score / cap of a raw product, from the row's score factor.
__device__ __forceinline__ float cap_factor(const Kv4AttnArgs& a, float f) {
  return fminf(f * a.inv_cap, FLT_MAX);
}
// s[0..C): raw products, f their factor -> tanh(score / cap), none above `top` (NaN
// stays).  `small`: the series does for all of the warp's.  Caps past kCapAbs pay for
// both formulas where it does not: 2048 rows x 32 heads on 4096 slots under a cap of
// 30 with scores past it 248 us, 461 with both.
template <int C>
__device__ __forceinline__ void cap_tanh(const Kv4AttnArgs& a, float* s, float f, bool small,
                                         float top) {
  if (small) {
    tanh_series<C>(s, f);
  } else if (a.cap <= kCapAbs) {
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = tanh_abs(s[c] * (f * kTwoLog2e));
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = min_nan(tanh_any(s[c] * f), top);
  }
}
// The same of one product, by the same formula.
__device__ __forceinline__ float cap_tanh1(const Kv4AttnArgs& a, float x, float f, bool small) {
  const float y = x * f, low = tanh_small(y), t = tanh_abs(y * kTwoLog2e);
  return small || (a.cap > kCapAbs && fabsf(y) <= kTanhTop) ? low : t;
}

// s[0..C): raw products of C slots from n0 on -> scores (GEN: in units of the cap if
// there is one, else log2 units), and -inf where the row does not see the slot.
// pos: explicit positions, or null.
template <bool GEN, int C>
__device__ __forceinline__ void tc_scores(const Kv4AttnArgs& a, float* s, volatile int* rowp,
                                          int n0, TcSeen seen, const int* pos) {
  const TcRow row = sm_get<TcRow>(rowp);
  if constexpr (GEN) {
    const float f2 = row.f * kLog2e;
    const uint64_t ff = f2_pack(f2, f2);
    if (a.cap > 0.f) {
      const float fy = cap_factor(a, row.f);
      cap_tanh<C>(a, s, fy, __all_sync(0xffffffffu, abs_max<C>(s) * fy <= kTanhTop), 1.f);
    } else {
#pragma unroll
      for (int c = 0; c < C; c += 2)
        f2_unpack(f2_mul(f2_pack(s[c], s[c + 1]), ff), s[c], s[c + 1]);
    }
    if (a.slope != nullptr) {
      if (pos == nullptr) {
        const float dq = (float)(row.qpos - n0);
#pragma unroll
        for (int c = 0; c < C; ++c) s[c] = fmaf(-row.slope2, fabsf(dq - (float)c), s[c]);
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
          s[c] = fmaf(-row.slope2, fabsf((float)(row.qpos - pos[c])), s[c]);
      }
    }
    if (pos != nullptr && a.span != nullptr) {  // (without a span any position is seen)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (n0 + c >= row.len || pos[c] < row.lo || pos[c] >= row.hi) s[c] = -INFINITY;
      return;
    }
  }
  if (seen != kAll) {  // columns [lo, lo + num) are seen
    const int lo = (int)min(max((long)row.lo - n0, 0L), (long)C);
    const int hi = (int)min(max((long)min(row.hi, row.len) - n0, 0L), (long)C);
    const uint32_t num = (uint32_t)max(hi - lo, 0);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if ((uint32_t)(c - lo) >= num) s[c] = -INFINITY;
  }
}

// One step of a softmax warp: its 32 rows' scores of 128 slots at s_col, P over
// them (64 slots at a time: p_full[0], p_full[1]), the rows' maximum and sum,
// and O at o_col rescaled where the maximum has outgrown it.  FAST: every row
// sees every slot (its own copy of the code: tests inside the passes cost a
// fifth of the step).  Scores that are only capped rise with the product: the
// maximum is taken of products and the cap applied on the way to P (LATE), not
// stored back between the passes.
template <int DH, int GEN, bool FAST>
__device__ __forceinline__ void softmax_step(const Kv4AttnArgs& a, volatile int* row, float f2,
                                             int n0, TcSeen seen0, TcSeen seen1, const int* ps,
                                             uint32_t s_col, uint32_t o_col, bool has_o,
                                             uint64_t* p_full, float& m_used, float& l,
                                             bool& huge) {
  // The maximum; scores that are more than raw products go back to TMEM for the
  // second pass (32 at a time then: their arithmetic needs registers too).
  constexpr bool LATE = FAST && GEN == kCap;
  constexpr int C = GEN && !LATE ? 32 : 64;
  const float fy = LATE ? cap_factor(a, __int_as_float(row[0])) : 0.f;
  float top = 0.f;
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // chains: one would wait on itself
#pragma unroll 1
  for (int k = 0; k < 128; k += C) {
    const TcSeen seen = FAST ? kAll : k < 64 ? seen0 : seen1;
    if (seen == kNone) continue;
    float s[C];
#pragma unroll
    for (int q = 0; q < C; q += 32)
      tc::tmem_ld32_nowait(s_col + k + q, reinterpret_cast<uint32_t*>(s) + q);
    tc::tmem_wait_ld();
    if (LATE) top = fmaxf(top, abs_max<C>(s));
    if ((GEN || !FAST) && !LATE) {
      tc_scores<GEN != 0, C>(a, s, row, n0 + k, seen, ps != nullptr ? ps + k : nullptr);
#pragma unroll
      for (int q = 0; q < C; q += 32)
        tc::tmem_st32(s_col + k + q, reinterpret_cast<uint32_t*>(s) + q);
    }
#pragma unroll
    for (int c = 0; c < C; c += 2) m4[(c >> 1) & 3] = max3(m4[(c >> 1) & 3], s[c], s[c + 1]);
  }
  if ((GEN || !FAST) && !LATE) tc::tmem_wait_st();
  const float m_raw = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
  const bool small = LATE && __all_sync(0xffffffffu, top * fy <= kTanhTop);
  const float m_unit = LATE ? cap_tanh1(a, m_raw, fy, small) : m_raw, m_tile = m_unit * f2;
  const bool grow = m_tile > __fadd_rd(m_used, kGrow);
  if (__any_sync(0xffffffffu, grow)) {
    const float m_new = grow ? m_tile : m_used;
    const float corr = grow ? exp2_approx(m_used - m_new) : 1.f;
    if (has_o) {
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
    huge = __any_sync(0xffffffffu, fabsf(m_used) >= kHuge && fabsf(m_used) < INFINITY);
  }
  // P over the scores: the first half lies on scores already read
  const float base = m_used == -INFINITY ? 0.f : __fsub_ru(m_used, kTcShift);
  float fx = f2;
  if (!LATE && huge) {
    fx = 1.f;
#pragma unroll 1
    for (int k = 0; k < 128; k += 32) {
      uint32_t s[32];
      tc::tmem_ld32_nowait(s_col + k, s);
      tc::tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 32; ++c) s[c] = __float_as_uint(__uint_as_float(s[c]) * f2);
      tc::tmem_st32(s_col + k, s);
    }
    tc::tmem_wait_st();
  }
  const uint64_t ff = f2_pack(fx, fx), nb = f2_pack(-base, -base);
  uint64_t sum[2] = {0, 0};
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
    if (!FAST && (h == 0 ? seen0 : seen1) == kNone) {
#pragma unroll
      for (int c = 0; c < 32; ++c) pk[c] = 0u;
    } else {
      float s[64];
      tc::tmem_ld32_nowait(s_col + 64 * h, reinterpret_cast<uint32_t*>(s));
      tc::tmem_ld32_nowait(s_col + 64 * h + 32, reinterpret_cast<uint32_t*>(s) + 32);
      tc::tmem_wait_ld();
      // (the two formulas meet within 2^-20 only: none may pass the maximum)
      if constexpr (LATE) cap_tanh<64>(a, s, fy, small, m_unit);
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(s[2 * c], s[2 * c + 1]), ff, nb), x0, x1);
        const float p0 = exp2_approx(x0), p1 = exp2_approx(x1);
        sum[c & 1] = f2_add(sum[c & 1], f2_pack(p0, p1));
        pk[c] = h2_bits(__floats2half2_rn(p0, p1));
      }
    }
    tc::tmem_st32(s_col + 32 * h, pk);
    tc::tmem_wait_st();
    tc::fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(p_full + h);  // half of P V may start
  }
  float s0, s1;
  f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
  l += s0 + s1;
}

// GEN: kCap, capped scores; kAny, a distance bias or explicit positions too.
template <int DH, int GEN>
__global__ void __launch_bounds__(kTcThreads, 1)
k_kv4_attn_tc(const __grid_constant__ Kv4AttnArgs a) {
  using SM = TcSmem<DH>;
  pdl_prologue();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  int* pos_ring = reinterpret_cast<int*>(smem + SM::kPos);  // [4][128]
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + SM::kBar);
  uint64_t *k_empty = k_full + 2, *v_full = k_full + 4, *v_empty = k_full + 6;
  uint64_t *s_full = k_full + 8, *o_full = k_full + 10, *q_full = k_full + 12;
  uint64_t* p_full = k_full + 14;  // [row tile][half of the slots]
  uint64_t* drain = k_full + 18;
  uint64_t *c_full = k_full + 19, *c_empty = c_full + kRing, *c_ask = c_empty + kRing;
  uint64_t* c_done = c_ask + 1;
  TcWork* ring = reinterpret_cast<TcWork*>(smem + SM::kItems);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(c_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler too
  const bool by_pos = GEN == kAny && a.kpos != nullptr;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(k_full + i, 4);
      tc::mbar_init(k_empty + i, 1);
      tc::mbar_init(v_full + i, 4);
      tc::mbar_init(v_empty + i, 1);
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(o_full + i, 1);
      tc::mbar_init(q_full + i, 4);
      tc::mbar_init(p_full + i, 4);
      tc::mbar_init(p_full + 2 + i, 4);
    }
    tc::mbar_init(drain, 1);
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(c_full + i, 1);
      tc::mbar_init(c_empty + i, 13);
    }
    tc::mbar_init(c_ask, 4);
    tc::mbar_init(c_done, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 12) tc::tmem_alloc(tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  TcItems next{c_full, c_empty, ring};

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int g = warp >> 2, r0 = warp * 32;  // row tile; first row of the warp
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + g * 128;
    const uint32_t o_col = tmem + lane_base + 256 + g * 128;
    uint8_t* qs = smem + g * SM::kOp;         // the row tile's operand
    const int qr = (warp & 3) * 32;           // the warp's first row in it
    volatile int* rowp = reinterpret_cast<volatile int*>(smem + SM::kRow) + 6 * tid;
    volatile int* keep = reinterpret_cast<volatile int*>(smem + SM::kWork) + warp * 8;
    bool ok = true;
    int it = 0, rounds = 0, all = 0;  // the row tile's steps and items, both row tiles' steps
    int nt;
    {
      TcWork w{-1, 0, 0, 0, 0, 0, 0, 0};
      ok = next.take(a, abort_flag, &w);
      if (lane == 0) sm_put(keep, w);
      __syncwarp();
    }
    while (ok && keep[0] >= 0) {
      TcRange range;
      float f2;
      bool act;
      int n_lo;
      {  // an item begins: the row's constants, its query
        const TcWork w = sm_get<TcWork>(keep);
        const int m = w.tile * 2 * kTile + r0 + lane;
        const bool in = m < a.M;
        const int t = row_token(a, m), h = w.hkv * a.G + (m - t * a.G);
        nt = w.nt;
        n_lo = w.n_lo;
        act = nt > 0 && (g == 0 || w.two);
        TcRow row = tc_row(a, in, w.b, t, h);
        range = tc_range(row);
        if (act) {
          fetch_q<DH>(a.Q, in ? static_cast<const __nv_bfloat16*>(a.Q) + (long)w.b * a.q_bld +
                               (long)t * a.q_ld + (long)h * DH
                         : nullptr,
                      tc::smem_u32(qs), qr);
          row.f = stage_q<DH>(a.scale, qs, qr + lane);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(q_full + g);
        }
        sm_put(rowp, row);
        f2 = !GEN ? row.f * kLog2e : a.cap > 0.f ? a.cap * kLog2e : 1.f;  // to log2 units
      }
      float m_used = -INFINITY, l = 0.f;
      bool huge = false;
      for (int j = 0; act && j < nt; ++j, ++it) {
        const int n0 = n_lo + j * kTile;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(s_full + g, it & 1, a.status, abort_flag));
        if (!ok) break;
        tc::fence_after_sync();
        const TcSeen seen0 = by_pos ? kSome : tc_seen(range, n0);
        const TcSeen seen1 = by_pos ? kSome : tc_seen(range, n0 + 64);
        if (seen0 == kAll && seen1 == kAll)
          softmax_step<DH, GEN, true>(a, rowp, f2, n0, kAll, kAll, nullptr, s_col, o_col, j > 0,
                                      p_full + 2 * g, m_used, l, huge);
        else
          // a step's positions: written before its K, and not again until the
          // V of the third step after it has been asked for
          softmax_step<DH, GEN, false>(a, rowp, f2, n0, seen0, seen1,
                                       by_pos ? pos_ring + ((all + j) & 3) * kTile : nullptr,
                                       s_col, o_col, j > 0, p_full + 2 * g, m_used, l, huge);
      }
      all += nt;
      const TcWork w = sm_get<TcWork>(keep);
      const int m = w.tile * 2 * kTile + r0 + lane;
      const bool in = m < a.M;
      const int t = row_token(a, m), h = w.hkv * a.G + (m - t * a.G);
      if (rowp[2] >= rowp[3]) {  // sees nothing anywhere
        l = 0.f;
        m_used = -INFINITY;
      }
      {
        TcWork wn{-1, 0, 0, 0, 0, 0, 0, 0};
        if (ok) ok = next.take(a, abort_flag, &wn);
        __syncwarp();
        if (lane == 0) sm_put(keep, wn);
        __syncwarp();
        if (wn.item >= 0) {  // the next item's queries into L2 while this one is finished
          const int mn = wn.tile * 2 * kTile + r0 + lane, tn = row_token(a, mn);
          if (mn < a.M)
            l2_prefetch(static_cast<const __nv_bfloat16*>(a.Q) +
                            (long)wn.b * a.q_bld + (long)tn * a.q_ld +
                            (long)(wn.hkv * a.G + (mn - tn * a.G)) * DH,
                        DH * 2);
        }
      }
      if (act && ok) {
        ok = __all_sync(0xffffffffu,
                        tc::mbar_wait(o_full + g, rounds & 1, a.status, abort_flag));
        tc::fence_after_sync();
        ++rounds;
      }
      // The finished rows: through the row's own place in the query operand
      // (no longer read), 256 bytes at a time, so that a warp stores whole rows.
      if (ok && (g == 0 || w.two)) {
        const bool part = a.nsplit > 1;
        const float mx = m_used == -INFINITY ? -INFINITY : m_used - kTcShift + kPShift;
        const int orow = (w.b * a.T + t) * a.Hq + h;  // < 2^25
        const uint32_t prow = ((uint32_t)(w.b * a.Hkv + w.hkv) * a.M + m) * a.nsplit + w.split;
        if (in) {
          if (part) {
            a.pml[2 * (size_t)prow] = mx;
            a.pml[2 * (size_t)prow + 1] = l;
          } else if (a.lse != nullptr) {
            a.lse[orow] = row_lse(mx, l);
          }
        }
        const bool zero = __any_sync(0xffffffffu, l == 0.f);  // rows that saw nothing
        const float inv = part ? 1.f : l == 0.f ? 0.f : a.vmul / l;
        const int per = part ? DH / 2 : DH;  // elements a row at a time
        constexpr int kLanes = DH / 8;       // 16-byte pieces of them
#pragma unroll 1
        for (int d0 = 0; d0 < DH; d0 += per) {
#pragma unroll 1
          for (int q = 0; q < per / 32; ++q) {
            uint32_t o[32];
            if (act) {
              tc::tmem_ld32_nowait(o_col + d0 + 32 * q, o);
              tc::tmem_wait_ld();
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv);
            if (zero) {  // 0, whatever TMEM holds
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = l == 0.f ? 0u : o[c];
            }
            if (part) {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(qs + sw128(qr + lane, 8 * q + c)) =
                    make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __nv_bfloat162 p2 =
                      __floats2bfloat162_rn(__uint_as_float(o[8 * c + 2 * e]),
                                            __uint_as_float(o[8 * c + 2 * e + 1]));
                  v[e] = *reinterpret_cast<const uint32_t*>(&p2);
                }
                *reinterpret_cast<uint4*>(qs + sw128(qr + lane, 4 * q + c)) =
                    make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
          }
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < kLanes; ++i) {
            const int rr = i * (32 / kLanes) + lane / kLanes, c = lane % kLanes;
            const size_t at = __shfl_sync(0xffffffffu, part ? prow : (uint32_t)orow, rr);
            const uint4 v = *reinterpret_cast<const uint4*>(qs + sw128(qr + rr, c));
            if (m - lane + rr < a.M) {
              if (part) reinterpret_cast<uint4*>(a.po + at * DH + d0)[c] = v;
              else reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.O) + at * DH)[c] = v;
            }
          }
          __syncwarp();
        }
      }
      tc::fence_before_sync();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ slots
    const int p = tid - 256, last = a.Ncache - 1;
    RawRow<DH> rk, rv;
    bool ok = true;
    auto ask = [&] {  // for the next item
      if (lane == 0) tc::mbar_arrive(c_ask);
    };
    // the next item with slots to read (-1: the end)
    auto take = [&](TcWork* x) {
      do {
        ok = next.take(a, abort_flag, x);
        if (!ok) x->item = -1;
        if (ok && x->item >= 0 && x->nt <= 2) ask();
      } while (x->item >= 0 && x->nt == 0);
    };
    auto load = [&](const TcWork& x, int j, const uint8_t* c, const uint8_t* s, RawRow<DH>& o) {
      const long base = (long)(x.b * a.Hkv + x.hkv) * a.Ncache;
      load_row<DH>(c, s, base + min((long)x.n_lo + (long)j * kTile + p, (long)last), o);
    };
    TcWork w;
    take(&w);
    int j = 0;
    if (w.item >= 0) {
      load(w, 0, a.kcode, a.kscale, rk);
      load(w, 0, a.vcode, a.vscale, rv);
    }
    for (int it = 0; w.item >= 0; ++it) {
      const int st = it & 1;
      const uint32_t ph = ((it >> 1) & 1) ^ 1;
      TcWork wn = w;
      int jn = j + 1;
      // the next item is asked for two steps before this one's end, and its first
      // slots loaded under the last step if the answer is there
      if (w.nt > 2 && jn == w.nt - 2) ask();
      bool known = true;
      if (jn == w.nt) {
        known = next.ready();
        jn = 0;
        if (known) {
          ok = next.take(a, abort_flag, &wn);
          if (ok && wn.item >= 0 && wn.nt <= 2) ask();
          known = ok && (wn.item < 0 || wn.nt > 0);
        }
      }
      const bool more = known && wn.item >= 0;
      if (ok) ok = tc::mbar_wait(k_empty + st, ph, a.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (by_pos)
        pos_ring[(it & 3) * kTile + p] =
            a.kpos[(long)(w.b * a.Hkv + w.hkv) * a.Ncache + min(w.n_lo + j * kTile + p, last)];
      put_row<DH>(smem + SM::kK + st * SM::kOp, p, rk);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(k_full + st);
      if (more) load(wn, jn, a.kcode, a.kscale, rk);
      ok = tc::mbar_wait(v_empty + st, ph, a.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      put_row<DH>(smem + SM::kV + st * SM::kOp, p, rv);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(v_full + st);
      if (more) load(wn, jn, a.vcode, a.vscale, rv);
      if (!known) {
        take(&wn);
        if (wn.item >= 0) {
          load(wn, 0, a.kcode, a.kscale, rk);
          load(wn, 0, a.vcode, a.vscale, rv);
        }
      }
      w = wn;
      j = jn;
    }
  } else if (warp == 13) {
    // ------------------------------------------------------------ claims
    uint4* claim = reinterpret_cast<uint4*>(ring + kRing);
    int item = blockIdx.x;
    for (int k = 0;; ++k) {
      const int at = k % kRing;
      const TcWork w = tc_item(a, item);
      bool ok = tc::mbar_wait(c_empty + at, ((k / kRing) & 1) ^ 1, a.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        ring[at] = w;
        tc::mbar_arrive(c_full + at);
      }
      if (item < 0) break;
      ok = tc::mbar_wait(c_ask, k & 1, a.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        tc::fence_proxy_async_smem();  // the last claim has been read
        claim_ask(claim, c_done);
      }
      __syncwarp();
      // waits for the answer whatever else happens: it is written to this CTA
      const uint64_t t0 = tc::globaltimer();
      while (!(ok = tc::mbar_try_wait(c_done, k & 1)) &&
             tc::globaltimer() - t0 < tc::kWaitLimitNs) {
      }
      if (!__all_sync(0xffffffffu, ok)) {
        set_status(a.status, PS_ERR_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      item = claim_get(claim);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ MMAs
    constexpr uint32_t kIdQK = idesc_f16(128, false), kIdPV = idesc_f16(DH, true);
    const uint32_t qb = tc::smem_u32(smem), kb = qb + SM::kK, vb = qb + SM::kV;
    auto qk = [&](int g, int st) {
      const uint32_t q = qb + g * SM::kOp, k = kb + st * SM::kOp;
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk) {
        const uint32_t off = (kk / 4) * 16384u + (kk % 4) * 32u;
        mma_ss(tmem + g * 128, tc::desc_sw128(q + off, 16, 1024),
               tc::desc_sw128(k + off, 16, 1024), kIdQK, kk > 0);
      }
      tc::mma_commit(s_full + g);
    };
    auto pv = [&](int g, int st, int half, bool first) {
      const uint32_t v = vb + st * SM::kOp;
#pragma unroll
      for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
        mma_ts(tmem + 256 + g * 128, tmem + g * 128 + kk * 8,
               tc::desc_sw128(v + kk * 2048u, 16384, 1024), kIdPV, !first || kk > 0);
    };
    bool ok = true;
    int it = 0, c0 = 0, c1 = 0, i0 = 0, i1 = 0;  // steps; each row tile's steps and items
    auto wait = [&](uint64_t* bar, int n) {
      if (ok) ok = tc::mbar_wait(bar, n & 1, a.status, abort_flag);
    };
    // P V of row tile g's step n, then S of its next step from stage stn
    auto row_tile = [&](int g, int n, bool last_tile, bool first, bool more) {
      const int st = it & 1, stn = st ^ 1;
      wait(p_full + 2 * g, n);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      if (ok && elect_one()) pv(g, st, 0, first);
      __syncwarp();
      wait(p_full + 2 * g + 1, n);
      if (g == 0 && more) wait(k_full + stn, (it + 1) >> 1);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      if (ok && elect_one()) {
        pv(g, st, 1, first);
        if (last_tile) tc::mma_commit(v_empty + st);
        if (more) {
          qk(g, stn);
          if (last_tile) tc::mma_commit(k_empty + stn);
        } else {
          tc::mma_commit(o_full + g);
        }
      }
      __syncwarp();
    };
    auto first_s = [&](int g, int n, bool last_tile) {
      wait(q_full + g, n);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      if (ok && elect_one()) {
        qk(g, it & 1);
        if (last_tile) tc::mma_commit(k_empty + (it & 1));
      }
      __syncwarp();
    };
    TcWork w, wn;
    ok = next.take(a, abort_flag, &w);
    while (ok && w.item >= 0) {
      if (w.nt > 0) {
        wait(k_full + (it & 1), it >> 1);
        first_s(0, i0++, !w.two);
        if (w.two) first_s(1, i1++, true);
      }
      bool known = false;
      for (int j = 0; ok && j < w.nt; ++j, ++it) {
        if (j + 1 == w.nt && next.ready()) known = ok = next.take(a, abort_flag, &wn);
        wait(v_full + (it & 1), it >> 1);
        row_tile(0, c0++, !w.two, j == 0, j + 1 < w.nt);
        if (w.two) row_tile(1, c1++, true, j == 0, j + 1 < w.nt);
      }
      if (ok && !known) ok = next.take(a, abort_flag, &wn);
      w = wn;
    }
    if (!__all_sync(0xffffffffu, ok)) {  // wait for the MMAs issued before TMEM is freed
      if (elect_one()) tc::mma_commit(drain);
      const uint64_t t0 = tc::globaltimer();
      while (!tc::mbar_try_wait(drain, 0) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {
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

template <int DH, int GEN>
cudaError_t launch_tc(const Kv4AttnArgs& a, cudaStream_t s) {
  auto kern = k_kv4_attn_tc<DH, GEN>;
  static DeviceOnce once;
  const cudaError_t e = allow_smem(kern, TcSmem<DH>::kBytes, once);
  if (e != cudaSuccess) return e;
  const unsigned items = (unsigned)(a.B * a.Hkv * a.ntile * a.nsplit);
  return launch_pdl(kern, dim3(items), dim3(kTcThreads), TcSmem<DH>::kBytes, s, a);
}

}  // namespace

cudaError_t kv4_attn_tc_launch(const Kv4AttnArgs& a, cudaStream_t s) {
  // (kCap takes caps that keep scores below kHuge)
  const int gen = a.slope != nullptr || a.kpos != nullptr || a.cap > kHuge / 4 ? kAny
                  : a.cap > 0.f ? kCap : kPlain;
#define PS_KV4_TC(DH, GEN) \
  if (a.dh == DH && gen == GEN) return launch_tc<DH, GEN>(a, s);
  PS_KV4_TC(64, kPlain)
  PS_KV4_TC(64, kCap)
  PS_KV4_TC(64, kAny)
  PS_KV4_TC(128, kPlain)
  PS_KV4_TC(128, kCap)
  PS_KV4_TC(128, kAny)
#undef PS_KV4_TC
  return cudaErrorInvalidValue;
}

}  // namespace ps
