// Attention over packed sequences or cache rows for bf16 rows on the tcgen05 tensor
// cores.
//
// A CTA an SM takes item after item: two tiles of up to 128 query rows (whole tokens:
// R = 128 / G of them) of one KV head against a share of its slots, 128 slots a step.
// 12 warps:
//   0-3, 4-7  softmax of row tile 0 / 1, a thread a row: its 128 scores from TMEM to
//             registers in one trip, the running maximum and sum, P (bf16) over the
//             scores, O in TMEM rescaled when it must be; the finished rows.  Before an
//             item's last P the rows of V that lie behind the sequence's slots are
//             cleared: they may hold anything, and zero times NaN is NaN
//   8         issues the MMAs: S = Q K^T into 128 TMEM columns a row tile, O += P V
//             into 128 more, P the TMEM-resident A operand
//   9         loads by TMA: an item's queries, K and V tiles through one ring
//   10        claims the next item (cluster launch control) and works out what it is
// Order of the MMAs, per step j:  P0 V(j), S0(j+1), P1 V(j), S1(j+1): the softmax of one
// row tile runs under the products of the other.  In an item's last step S(j+1) is the
// first one of the next item, whose queries are loaded as soon as the last S of this
// one has read its own.  The commit that announces S(j+1) also says that P V(j) is
// done, so O may be rescaled then.  It is rescaled only when a row's maximum has grown
// by 2^kGrow or more: until then P just carries a factor up to that.  P is rounded to bf16,
// the type that V is multiplied in: half a step, 2^-8 at most, of a weight, the row's sum being
// of the unrounded ones in fp32.  Of O that makes an error of 0.0023 of its norm where its own
// rounding makes 0.0016; a second term of P would be half as many products again.
//
// What bounds it: the chain of a step, product, softmax, product; the other row tile hides
// half of it.  2 x 4096 rows of 32 heads on 4096 slots: 338 us, 1.63 PFLOP/s, tensor
// cores 66 % busy.  The scores through TMEM in trips of 64 columns took 351 us, of 32 388;
// all the MMA loop by one elected lane 343 where a warp in step took 450; items of 4, 8
// and 32 KV heads' neighbours (kHeads) 343, 339, 351; the next item claimed as early as
// it can be 230 us for causal rows where two steps ahead take 204.
//
// Every mbarrier wait is bounded (tc::mbar_wait); after a timeout the CTA waits for the
// copies and MMAs it issued, frees TMEM and returns with the status word set.
#include <cfloat>
#include <climits>

#include "attn.cuh"
#include "tc.cuh"

namespace ps {
namespace {

constexpr int kTcThreads = 384;
constexpr int kSoftRegs = 208, kOtherRegs = 88;  // 256 x 208 + 128 x 88 = 384 x 168
constexpr int kItems = 4;           // items known and not yet taken by every warp
// Items of a softmax warp with rows to be computed again.  The first is the last one that
// its CTA asks for: kItems more may be known by then, and one claimed.
constexpr int kAgain = 8;
static_assert(kAgain >= kItems + 2, "the items that still come");
constexpr int kTile = 128;          // slots a step
static_assert(kTcRows == 128, "a thread a row");
constexpr float kGrow = 8.f;        // log2 growth of a maximum before O is rescaled
// A maximum from which on scores are rounded before it is subtracted from them: it is
// rounded itself, and by 2^-24 of it P would leave its range.
constexpr float kHuge = 0x1p22f;

struct TcItem {
  int item, split, hkv, s;
  int t0;            // first token of the item in its sequence
  int n_lo;          // first slot
  int nt0, nt1;      // steps of the row tiles (0: none, or no rows)
  AttnSeq seq;
  __device__ __forceinline__ AttnSeq get_seq() const volatile {
    return {seq.q0, seq.n, seq.k0, seq.m};
  }
};

struct TcAgain {
  uint32_t rows;  // of the warp
  int r0, h0;     // first row of Q of the row tile, first head of the group
};
struct TcAgains {
  int num;
  TcAgain item[kAgain];
};

template <int DH>
struct TcSmem {
  static constexpr uint32_t kOp = (DH / 64) * 16384u;      // 128 rows of DH bf16
  static constexpr int kRing = DH == 128 ? 5 : 8;          // K and V tiles
  static constexpr uint32_t kKv = 2 * kOp;                 // Q at 0
  static constexpr uint32_t kBar = kKv + kRing * kOp;
  static constexpr uint32_t kWork = kBar + 512;            // TcItem [kItems], then a claim
  static constexpr uint32_t kRedo = kWork + kItems * sizeof(TcItem) + 16;  // TcAgains [8]
  static constexpr size_t kBytes = 1024 + kRedo + 8 * sizeof(TcAgains);
};
static_assert(sizeof(TcItem) % 16 == 0, "the claim behind the items is 16-byte aligned");
static_assert(TcSmem<128>::kBytes <= 227 * 1024, "a CTA's shared memory");

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
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
__device__ __forceinline__ uint64_t f2_pack(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 bytes of a thread, at once where the rows are aligned to that: rows lie far
// apart, and a store pays for each that it touches.
__device__ __forceinline__ void st32(bool whole, void* p, const uint32_t* v) {
  if (!whole) {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// ---------------------------------------------------------------- work items
__device__ __forceinline__ void claim_ask(uint4* to, uint64_t* bar) {
  tc::mbar_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(tc::smem_u32(to)),
      "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ int claim_get(const uint4* from) {  // -1: none is left
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

// What item number `item` is, for a whole warp.  kHeads KV heads at a time, so that
// the CTAs read the same K and V together; of them the last row tiles first: causal
// masks make them the longest.
constexpr int kHeads = 8;
__device__ __forceinline__ TcItem tc_item(const AttnArgs& a, int item) {
  TcItem w{item, 0, 0, 0, 0, 0, 0, 0, {0, 0, 0, 0}};
  if (item < 0) return w;
  const int lane = threadIdx.x & 31;
  const long block = a.tiles * kHeads * a.nsplit;  // items of kHeads heads
  const int h0 = (int)(item / block) * kHeads, heads = min(kHeads, a.Hkv - h0);
  int k = (int)(item % block);
  w.split = k % a.nsplit;
  k /= a.nsplit;
  w.hkv = h0 + k % heads;
  const long tile = a.tiles - 1 - k / heads;
  auto first = [&](int s) { return (long)attn_q_off(a, s) / (2 * a.R) + s; };
  w.s = attn_find(a.S, tile, first);
  w.seq = attn_seq(a, w.s);
  const long t0 = (tile - first(w.s)) * 2 * a.R;
  const long rows = (long)w.seq.n * a.G;
  if (t0 < 0 || t0 >= w.seq.n || rows < a.least || rows > a.most) {
    w.seq.n = 0;  // a number left over, or another kernel's sequence
    return w;
  }
  w.t0 = (int)t0;
  int lo = INT_MAX, hi[2] = {0, 0};
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int from = w.t0 + g * a.R, to = min(from + a.R, w.seq.n);
    if (a.span == nullptr) {  // the last token sees the most
      if (from < to) {
        const int2 x = attn_seen(a, w.seq, to - 1);
        if (x.x < x.y) {
          lo = 0;
          hi[g] = x.y;
        }
      }
    } else {
      int h = 0;
      for (int t = from + lane; t < to; t += 32) {
        const int2 x = attn_seen(a, w.seq, t);
        if (x.x < x.y) {
          lo = min(lo, x.x);
          h = max(h, x.y);
        }
      }
      hi[g] = __reduce_max_sync(0xffffffffu, h);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (a.nsplit > 1) {
    lo = (int)max((long)lo, (long)w.split * a.chunk);
    if (w.split + 1 < a.nsplit) {
      const long end = (long)(w.split + 1) * a.chunk;
      hi[0] = (int)min((long)hi[0], end);
      hi[1] = (int)min((long)hi[1], end);
    }
  }
  w.n_lo = lo == INT_MAX ? 0 : lo;
  if (hi[0] > w.n_lo) w.nt0 = (int)(((long)hi[0] - w.n_lo + kTile - 1) / kTile);
  if (hi[1] > w.n_lo) w.nt1 = (int)(((long)hi[1] - w.n_lo + kTile - 1) / kTile);
  return w;
}

// The items of a CTA, for a warp of any role.
struct TcItems {
  uint64_t *full, *empty;  // an item: known, taken by every warp
  const TcItem* ring;
  int n = 0;  // taken
  // the next item, which stays where it is until it is put back (null: a timeout)
  __device__ __forceinline__ const TcItem* hold(const AttnArgs& a, volatile int* abort_flag) {
    const int k = n % kItems;
    const bool ok = tc::mbar_wait(full + k, (n / kItems) & 1, a.status, abort_flag);
    return __all_sync(0xffffffffu, ok) ? ring + k : nullptr;
  }
  __device__ __forceinline__ void put_back() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(empty + n % kItems);
    ++n;
  }
  __device__ __forceinline__ bool take(const AttnArgs& a, volatile int* abort_flag, TcItem* w) {
    const TcItem* x = hold(a, abort_flag);
    if (x == nullptr) return false;
    *w = *x;
    put_back();
    return true;
  }
};

// ---------------------------------------------------------------- softmax
struct TcSoft {
  float f2;            // log2 units of a raw product, positive
  bool neg;            // the scale is negative
  float m, l;          // maximum that P is relative to, sum
  bool huge;
};

// One step of a softmax warp: P over the scores at s_col (64 slots at a time: p_full[0],
// p_full[1]), the rows' maximum and sum, O at o_col rescaled where the maximum has
// outgrown it.  GEN: the row sees columns [lo, hi) only, or the scale is negative (tests
// inside the plain pass would take a third of its issue slots).
template <int DH, bool GEN>
__device__ __forceinline__ void softmax_step(TcSoft& r, int lo, int hi, uint32_t s_col,
                                             uint32_t o_col, bool has_o, uint64_t* p_full) {
  float s[kTile];
#pragma unroll
  for (int q = 0; q < kTile; q += 32)
    tc::tmem_ld32_nowait(s_col + q, reinterpret_cast<uint32_t*>(s) + q);
  tc::tmem_wait_ld();
  if (GEN) {
    if (r.neg) {
#pragma unroll
      for (int c = 0; c < kTile; ++c) s[c] = -s[c];
    }
    if (__any_sync(0xffffffffu, lo > 0)) {
#pragma unroll
      for (int c = 0; c < kTile; ++c)
        if (c < lo) s[c] = -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < kTile; ++c)
      if (c >= hi) s[c] = -INFINITY;
  }
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < kTile; c += 2) m4[(c >> 1) & 3] = max3(m4[(c >> 1) & 3], s[c], s[c + 1]);
  const float m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * r.f2;
  const bool grow = m_tile > __fadd_rd(r.m, kGrow);
  if (__any_sync(0xffffffffu, grow)) {
    const float m_new = grow ? m_tile : r.m;
    const float corr = grow ? attn_exp2(r.m - m_new) : 1.f;
    if (has_o) {
#pragma unroll 1
      for (int q = 0; q < DH / 16; ++q) {
        uint32_t o[16];
        tc::tmem_ld16_nowait(o_col + 16 * q, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * corr);
        tc::tmem_st16(o_col + 16 * q, o);
      }
    }
    r.l *= corr;
    r.m = m_new;
    r.huge = __any_sync(0xffffffffu, fabsf(r.m) >= kHuge && fabsf(r.m) < INFINITY);
  }
  float fx = r.f2;
  if (r.huge) {
    fx = 1.f;
#pragma unroll
    for (int c = 0; c < kTile; ++c) s[c] *= r.f2;
  }
  const float base = r.m == -INFINITY ? 0.f : r.m;
  const uint64_t ff = f2_pack(fx, fx), nb = f2_pack(-base, -base);
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(s[64 * h + 2 * c], s[64 * h + 2 * c + 1]), ff, nb), x0, x1);
      const float p0 = attn_exp2(x0), p1 = attn_exp2(x1);
      sum[c & 1] = f2_add(sum[c & 1], f2_pack(p0, p1));
      pk[c] = pack_bf16(p0, p1);
    }
    tc::tmem_st32(s_col + 32 * h, pk);
    tc::tmem_wait_st();
    tc::fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(p_full + h);  // half of P V may start
  }
  float s0, s1;
  f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
  r.l += s0 + s1;
}

template <int DH>
__global__ void __launch_bounds__(kTcThreads, 1)
k_attn_tc(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tq,
          const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using SM = TcSmem<DH>;
  pdl_prologue();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + SM::kBar);  // [kRing]
  uint64_t* kv_empty = kv_full + 8;
  uint64_t *s_full = kv_full + 16, *o_full = s_full + 2, *q_full = s_full + 4,
           *q_empty = s_full + 6;
  uint64_t* p_full = s_full + 8;  // [row tile][half of the slots]
  uint64_t* drain = s_full + 12;
  uint64_t *c_full = drain + 1, *c_empty = c_full + kItems, *c_ask = c_empty + kItems;
  uint64_t* c_done = c_ask + 1;   // the 39th of 64
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(c_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* stop = abort_flag + 1;  // no more items: rows are to be computed again
  TcItem* ring = reinterpret_cast<TcItem*>(smem + SM::kWork);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler too
  if (tid == 0) {
    for (int i = 0; i < SM::kRing; ++i) {
      tc::mbar_init(kv_full + i, 1);
      tc::mbar_init(kv_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(o_full + i, 1);
      tc::mbar_init(q_full + i, 1);
      tc::mbar_init(q_empty + i, 1);
      tc::mbar_init(p_full + i, 4);
      tc::mbar_init(p_full + 2 + i, 4);
    }
    tc::mbar_init(drain, 1);
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(c_full + i, 1);
      tc::mbar_init(c_empty + i, 10);
    }
    tc::mbar_init(c_ask, 1);
    tc::mbar_init(c_done, 1);
    *abort_flag = 0;
    *stop = 0;
    tc::fence_mbar_init();
  }
  if (tid < 8) reinterpret_cast<TcAgains*>(smem + SM::kRedo)[tid].num = 0;
  if (warp == 8) tc::tmem_alloc(tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  TcItems next{c_full, c_empty, ring};

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------------------ softmax
    const int g = warp >> 2;                          // row tile
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + g * 128;
    const uint32_t o_col = tmem + lane_base + 256 + g * 128;
    const int rr = (warp & 3) * 32 + lane;            // the thread's row of the tile
    const int tt = (int)a.by_g.of((uint32_t)rr);      // token and head of it
    const int hh = rr - tt * a.G;
    int it = 0, rounds = 0, places = 0;  // (places: of the ring, up to this item)
    // (an item's numbers are read again when it ends: in registers they would push the
    // scores out)
    const volatile TcItem* w;
    while ((w = next.hold(a, abort_flag)) != nullptr && w->item >= 0) {
      TcSoft r;
      r.f2 = fmaxf(fabsf(a.scale) * kAttnLog2e, FLT_MIN);
      r.neg = a.scale < 0.f;
      r.m = -INFINITY;
      r.l = 0.f;
      r.huge = false;
      const int nt = g == 0 ? w->nt0 : w->nt1;
      // columns of the step that the row sees, and that every row of the warp sees
      int lo, hi, all_lo, all_hi;
      {
        const AttnSeq seq = w->get_seq();
        const int t = w->t0 + g * a.R + tt, n_lo = w->n_lo;
        const int2 see = tt < a.R && t < seq.n ? attn_seen(a, seq, t) : make_int2(0, INT_MAX);
        long end = (long)n_lo + (long)nt * kTile;  // a share ends where the next one begins
        if (a.nsplit > 1 && w->split + 1 < a.nsplit) end = min(end, (long)(w->split + 1) * a.chunk);
        lo = see.x - n_lo;
        hi = (int)(min((long)see.y, end) - n_lo);
        all_lo = __reduce_max_sync(0xffffffffu, lo);
        all_hi = r.neg ? INT_MIN : __reduce_min_sync(0xffffffffu, hi) - kTile;
      }
      bool ok = true;
      // the last V, if this row tile's products are the first that read it
      const int steps = max(w->nt0, w->nt1);
      const bool mend = nt == steps && (g == 0 || w->nt0 < steps) &&
                        w->seq.m - w->n_lo < steps * kTile;
      places += 2 * steps;
      for (int j = 0; j < nt; ++j, ++it) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(s_full + g, it & 1, a.status, abort_flag));
        if (!ok) break;
        if (mend && j + 1 == nt) {
          const int at = (places - 1) % SM::kRing;
          ok = __all_sync(0xffffffffu, tc::mbar_wait(kv_full + at, ((places - 1) / SM::kRing) & 1,
                                                     a.status, abort_flag));
          if (!ok) break;
          uint8_t* v = smem + SM::kKv + at * SM::kOp;
          const int have = w->seq.m - w->n_lo - j * kTile;
          for (int x = have * 8 + (tid & 127); x < kTile * 8; x += 128)
#pragma unroll
            for (int p = 0; p < DH / 64; ++p)
              *reinterpret_cast<uint4*>(v + p * 16384 + x * 16) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async_smem();
        }
        tc::fence_after_sync();
        const int n = j * kTile;
        if (n >= all_lo && n <= all_hi)
          softmax_step<DH, false>(r, 0, 0, s_col, o_col, j > 0, p_full + 2 * g);
        else
          softmax_step<DH, true>(r, lo - n, hi - n, s_col, o_col, j > 0, p_full + 2 * g);
      }
      if (ok && nt > 0) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(o_full + g, rounds & 1, a.status, abort_flag));
        tc::fence_after_sync();
        ++rounds;
      }
      if (!ok) break;
      // the finished rows, a thread a row
      const bool part = a.nsplit > 1;
      const AttnSeq seq = w->get_seq();
      const int t = w->t0 + g * a.R + tt, h = w->hkv * a.G + hh, split = w->split;
      next.put_back();
      if (part && nt == 0) continue;  // (the other row tile's share)
      const bool in = tt < a.R && t < seq.n;
      const long row = (long)(seq.q0 + t) * a.Hq + h;
      const bool none = r.l == 0.f;
      const float inv = part ? 1.f : none ? 0.f : 1.f / r.l;
      // a NaN once an element is infinite or NaN: two chains of products with zero
      const __nv_bfloat162 nil = __floats2bfloat162_rn(0.f, 0.f);
      __nv_bfloat162 zero[2] = {nil, nil};
      float* po = a.po + (row * a.nsplit + split) * a.dh;
      __nv_bfloat16* O = static_cast<__nv_bfloat16*>(a.O) + (long)(seq.q0 + t) * a.o_ld +
                         (long)h * a.dh;
      // (a loop: code that runs once an item is not in the instruction cache, and
      // unrolled it took longer to fetch than to run)
#pragma unroll 1
      for (int d = 0; d < a.dh; d += 16) {
        uint32_t x[16];
        if (nt > 0) {
          tc::tmem_ld16_nowait(o_col + d, x);
          tc::tmem_wait_ld();
        }
        if (none) {
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = 0;
        }
        if (part) {
          if (in) {
            st32(a.whole, po + d, x);
            st32(a.whole, po + d + 8, x + 8);
          }
        } else {
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = pack_bf16(__uint_as_float(x[2 * e]) * inv, __uint_as_float(x[2 * e + 1]) * inv);
            const __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162*>(&v[e]);
            zero[e & 1] = __hfma2(y, nil, zero[e & 1]);
          }
          if (in) st32(a.whole, O + d, v);
        }
      }
      tc::fence_before_sync();
      if (in) {
        if (part) {
          float* ml = a.pml + 2 * (row * a.nsplit + split);
          ml[0] = r.m;
          ml[1] = r.l;
        } else if (a.lse != nullptr) {
          a.lse[row] = attn_lse(r.m, r.l);
        }
      }
      if (!part) {
        const __nv_bfloat162 z = __hadd2(zero[0], zero[1]);
        const bool fine = __low2float(z) == 0.f && __high2float(z) == 0.f;
        const uint32_t bad = __ballot_sync(0xffffffffu, in && !fine);
        if (bad != 0) {
          if (lane == 0) {
            TcAgains* const x = reinterpret_cast<TcAgains*>(smem + SM::kRedo) + warp;
            x->item[x->num++] = TcAgain{bad, seq.q0 + t - tt, h - hh};
            *stop = 1;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---------------------------------------------------------- MMAs
      // One elected lane does it all: what lies between the MMAs is on the step's
      // critical path, and votes and barriers of the warp made up a third of it.
      if (elect_one()) {
        constexpr uint32_t kIdQK = tc::idesc_bf16(128, 128, false);
        constexpr uint32_t kIdPV = tc::idesc_bf16(128, DH, true);
        constexpr uint32_t kOp4 = SM::kOp >> 4;
        const uint64_t k_desc = tc::desc_sw128(0, 16, 1024), v_desc = tc::desc_sw128(0, 16384, 1024);
        const uint32_t q_lo = tc::smem_u32(smem) >> 4, r_lo = q_lo + 2 * kOp4;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (ok) ok = tc::mbar_wait(bar, parity, a.status, abort_flag);
        };
        // a place in the ring: the step's K; its V and the next K lie one and two on
        struct Place {
          int i;
          uint32_t ph;
        };
        auto on = [](Place p, int by) {
          p.i += by;
          if (p.i >= SM::kRing) {
            p.i -= SM::kRing;
            p.ph ^= 1;
          }
          return p;
        };
        auto qk = [&](int g, Place k, bool last_q, bool last_k) {
          const uint32_t ql = q_lo + g * kOp4, kl = r_lo + k.i * kOp4;
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            const uint32_t off = ((kk / 4) * 16384u + (kk % 4) * 32u) >> 4;
            tc::mma_bf16(tmem + g * 128, k_desc + (ql + off), k_desc + (kl + off), kIdQK, kk > 0);
          }
          tc::mma_commit(s_full + g);
          if (last_q) tc::mma_commit(q_empty + g);
          if (last_k) tc::mma_commit(kv_empty + k.i);
        };
        auto pv = [&](int g, Place v, int half, bool fresh) {
          const uint32_t vl = r_lo + v.i * kOp4;
#pragma unroll
          for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
            mma_ts(tmem + 256 + g * 128, tmem + g * 128 + kk * 8, v_desc + (vl + kk * 128u),
                   kIdPV, !fresh || kk > 0);
        };
        uint32_t cp[2] = {0, 0}, cq[2] = {0, 0};  // parities: P, Q
        // the first S of row tile g of an item of nt steps
        auto first_s = [&](int g, int nt, Place k, bool last_k) {
          if (nt == 0) return;
          wait(kv_full + k.i, k.ph);
          wait(q_full + g, cq[g]);
          cq[g] ^= 1;
          tc::fence_after_sync();
          if (ok) qk(g, k, nt == 1, last_k);
        };
        struct Work {
          int item, nt0, nt1;
        };
        auto take = [&]() {
          Work x{-1, 0, 0};
          const int at = next.n % kItems;
          wait(c_full + at, (next.n / kItems) & 1);
          if (ok) {
            const volatile TcItem* w = ring + at;
            x.item = w->item;
            x.nt0 = w->nt0;
            x.nt1 = w->nt1;
            tc::mbar_arrive(c_empty + at);
            ++next.n;
          }
          return x;
        };
        auto idle = [](const Work& x) { return x.item >= 0 && max(x.nt0, x.nt1) == 0; };
        Place k{0, 0};
        Work wn = take();
        bool begun = false;  // the first S of wn are under way
        while (ok) {
          // (items without steps are passed over here, with nothing held back: in a last
          // step the softmax warps could not go on and make room for what comes next)
          while (ok && idle(wn)) wn = take();
          if (!ok || wn.item < 0) break;
          const Work w = wn;
          if (!begun) {
            first_s(0, w.nt0, k, w.nt1 == 0);
            first_s(1, w.nt1, k, true);
          }
          const int steps = max(w.nt0, w.nt1);
          for (int j = 0; ok && j < steps; ++j) {
            const bool end = j + 1 == steps;
            const Place v = on(k, 1), kn = on(k, 2);
            if (end) {
              wn = take();
              begun = wn.item >= 0 && !idle(wn);
            }
            wait(kv_full + v.i, v.ph);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int nt = g == 0 ? w.nt0 : w.nt1;
              if (j < nt) {
                const bool more = j + 1 < nt;
                wait(p_full + 2 * g, cp[g]);
                tc::fence_after_sync();
                if (ok) pv(g, v, 0, j == 0);
                if (more) wait(kv_full + kn.i, kn.ph);
                wait(p_full + 2 * g + 1, cp[g]);
                cp[g] ^= 1;
                tc::fence_after_sync();
                if (ok) {
                  pv(g, v, 1, j == 0);
                  if (g == 1 || j >= w.nt1) tc::mma_commit(kv_empty + v.i);
                  if (more) qk(g, kn, j + 2 == nt, g == 1 || j + 1 >= w.nt1);
                  else tc::mma_commit(o_full + g);
                }
              }
              if (end && ok && begun)
                first_s(g, g == 0 ? wn.nt0 : wn.nt1, kn, g == 1 || wn.nt1 == 0);
            }
            k = kn;
          }
        }
        if (!ok) {  // wait for the MMAs issued before TMEM is freed
          tc::mma_commit(drain);
          const uint64_t t0 = tc::globaltimer();
          while (!tc::mbar_try_wait(drain, 0) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {
          }
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---------------------------------------------------------- loads
      bool ok = true;
      int k = 0, q[2] = {0, 0};  // tiles, queries of each row tile loaded
      const uint32_t rows = (uint32_t)(a.R * a.G) * 128u;
      auto tile = [&](const CUtensorMap* m, int hkv, long row) {
        if (ok) ok = tc::mbar_wait(kv_empty + k % SM::kRing, ((k / SM::kRing) & 1) ^ 1, a.status,
                                   abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && elect_one()) {
          uint64_t* bar = kv_full + k % SM::kRing;
          uint8_t* to = smem + SM::kKv + (k % SM::kRing) * SM::kOp;
          tc::mbar_expect_tx(bar, SM::kOp);
#pragma unroll
          for (int p = 0; p < DH / 64; ++p)
            tc::tma_load_3d(to + p * 16384, m, bar, 64 * p, hkv, (int)row);
        }
        __syncwarp();
        if (ok) ++k;
      };
      TcItem w;
      while (ok && (ok = next.take(a, abort_flag, &w)) && w.item >= 0) {
        const int steps = max(w.nt0, w.nt1);
        bool asked = false;
        for (int j = 0; ok && j < steps; ++j) {
          if (j == 0) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if ((g == 0 ? w.nt0 : w.nt1) == 0) continue;
              if (ok) ok = tc::mbar_wait(q_empty + g, (q[g] & 1) ^ 1, a.status, abort_flag);
              ok = __all_sync(0xffffffffu, ok);
              if (ok && elect_one()) {
                tc::mbar_expect_tx(q_full + g, rows * (DH / 64));
#pragma unroll
                for (int p = 0; p < DH / 64; ++p)
                  tc::tma_load_3d(smem + g * SM::kOp + p * 16384, &tq, q_full + g, 64 * p,
                                  w.hkv * a.G, w.seq.q0 + w.t0 + g * a.R);
              }
              __syncwarp();
              if (ok) ++q[g];
            }
          }
          const long row = (long)w.seq.k0 + w.n_lo + (long)j * kTile;
          tile(&tk, w.hkv, row);
          if (j + 2 >= steps && !asked) {
            asked = true;
            if (ok && lane == 0) tc::mbar_arrive(c_ask);
            __syncwarp();
          }
          tile(&tv, w.hkv, row);
        }
        if (!asked && ok) {
          if (lane == 0) tc::mbar_arrive(c_ask);
          __syncwarp();
        }
      }
      if (!__all_sync(0xffffffffu, ok)) {  // wait for the copies under way
        const uint64_t t0 = tc::globaltimer();
        auto over = [&](uint64_t* bar, int n) {  // the n-th use (from 1) of a barrier
          while (n > 0 && !tc::mbar_try_wait(bar, (n - 1) & 1) &&
                 tc::globaltimer() - t0 < tc::kWaitLimitNs) {
          }
        };
        for (int x = 0; x < SM::kRing; ++x) over(kv_full + x, (k + SM::kRing - 1 - x) / SM::kRing);
        over(q_full, q[0]);
        over(q_full + 1, q[1]);
      }
      __syncwarp();
    } else if (warp == 10) {
      // ---------------------------------------------------------- claims
      uint4* claim = reinterpret_cast<uint4*>(ring + kItems);
      int item = blockIdx.x;
      int k = 0;  // items passed on
      for (int asks = 0;; ++asks) {
        const TcItem w = tc_item(a, item);
        bool ok = true;
        // a number left over, or a share behind the slots: nobody has work
        if (item < 0 || !(w.seq.n == 0 || (a.nsplit > 1 && max(w.nt0, w.nt1) == 0))) {
          const int at = k % kItems;
          ok = tc::mbar_wait(c_empty + at, ((k / kItems) & 1) ^ 1, a.status, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) break;
          if (lane == 0) {
            ring[at] = w;
            tc::mbar_arrive(c_full + at);
          }
          __syncwarp();
          if (item < 0) break;
          ok = tc::mbar_wait(c_ask, k & 1, a.status, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) break;
          ++k;
        }
        if (__any_sync(0xffffffffu, *stop != 0)) {
          item = -1;
          continue;
        }
        if (lane == 0) {
          tc::fence_proxy_async_smem();  // the last claim has been read
          claim_ask(claim, c_done);
        }
        __syncwarp();
        // waits for the answer whatever else happens: it is written to this CTA
        const uint64_t t0 = tc::globaltimer();
        while (!(ok = tc::mbar_try_wait(c_done, asks & 1)) &&
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
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  } else if (warp < 8 && *stop != 0 && *abort_flag == 0) {
    // Rows that are computed again, when no other warp waits any more: 32 over 100 thousand
    // slots take longer than a wait may.  (The items that are left run in CTAs of their own.)
    const TcAgains* const again = reinterpret_cast<const TcAgains*>(smem + SM::kRedo) + warp;
    for (int i = 0; i < again->num; ++i) {
      const TcAgain x = again->item[i];
      const AttnSeq seq =
          attn_seq(a, attn_find(a.S, x.r0, [&](int s) { return (long)attn_q_off(a, s); }));
      for (uint32_t rows = x.rows; rows != 0; rows &= rows - 1) {
        const int m = (warp & 3) * 32 + __ffs(rows) - 1, t = (int)a.by_g.of((uint32_t)m);
        attn_redo<__nv_bfloat16>(a, seq, x.r0 - seq.q0 + t, x.h0 + m - t * a.G);
      }
    }
  }
}

template <int DH>
cudaError_t launch_tc(AttnArgs a, cudaStream_t s) {
  auto kern = k_attn_tc<DH>;
  static DeviceOnce once;
  const cudaError_t e = allow_smem(kern, TcSmem<DH>::kBytes, once);
  if (e != cudaSuccess) return e;
  const uintptr_t to = a.nsplit > 1 ? reinterpret_cast<uintptr_t>(a.po)
                                    : reinterpret_cast<uintptr_t>(a.O) | (uintptr_t)a.o_ld * 2;
  a.whole = to % 32 == 0;
  CUtensorMap q, k, v;
  if (!make_tmap_bf16_rows(&q, a.Q, a.dh, a.Hq, a.Tq, a.q_ld, a.G, a.R) ||
      !attn_tmaps(a, kTile, &k, &v))
    return cudaErrorInvalidValue;
  const long items = (long)a.tiles * a.Hkv * a.nsplit;
  if (items > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_pdl(kern, dim3((unsigned)items), dim3(kTcThreads), TcSmem<DH>::kBytes, s, a, q, k,
                    v);
}

}  // namespace

cudaError_t attn_tc_launch(const AttnArgs& a, cudaStream_t s) {
  return a.dh <= 64 ? launch_tc<64>(a, s) : launch_tc<128>(a, s);
}

}  // namespace ps
