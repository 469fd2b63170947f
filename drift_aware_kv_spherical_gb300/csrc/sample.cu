// Tokens drawn from rows of logits: temperature, top-k, top-p, min-p.
//
// All three filters leave a prefix of the row in descending order (ties by index),
// so a row comes down to the last element that is left: a cut (key, index).  A
// cluster of Z CTAs takes a row and keeps it in shared memory, a slice a CTA: the
// logits are read from memory once.
//   1  the maximum
//   2  top-k and top-p.  Short rows: all elements in one list (by_list).  bf16: a
//      histogram of counts by value (by_value); fp32 top-p: a fine one of counts, which
//      bounds the sums (narrow).  Where these cannot tell, and for fp32 top-k (select):
//      a histogram over 2048 bins of equal width below the maximum, of counts or of w,
//      summed over the cluster, gives the bin that holds the cut and what lies above it;
//      the bin's elements (a few hundred) go to CTA 0, which finds the cut among them.
//      A bin of more than kList elements is split again by its keys; a bin of nothing
//      but ties is counted off by index
//   3  the sum of the w that are left, then the element that u falls on
// w is fixed point with 43 bits behind the point: integer sums do not depend on
// their order, so histograms by atomics are exact and every call gives the same
// bits.  Its 2^-30 keep a draw where fp64 puts it but for one in millions.
//
// What bounds it: instructions, some 30 a logit of w alone, and the barriers between the
// passes (a warp waits five issues at one for every one of its own: CTA 0 finishes alone, and
// two CTAs an SM do not cover that).  256 rows of 152064: fp32 with top-p 237 us, 23 to read
// them; bf16 with a temperature 120, with top-k 200.  Clusters of 16 and CTAs of 256
// threads were slower.
#include <cfloat>
#include <climits>

#include "ops.h"
#include "tc.cuh"
#include "vec.cuh"

namespace ps {
namespace {

constexpr int kST = 512, kWarps = kST / 32;
constexpr int kPer = 4;          // bins a thread sums up, at most
constexpr int kBins = 2048, kList = 1024;
static_assert(kList * 8 <= kBins * 12 && kBins / kST <= 4 && kBins / 8 <= kST, "bins of a CTA");
constexpr int kWords = 3 * kBins, kFine = 2 * kWords;  // two bins of 16 bits a word
constexpr int kOne = 43;         // w of the maximum: 2^43; a million of them fit 63 bits
constexpr int kLimb = 15;        // bits of a histogram's limbs: 2^17 of them fit 32
constexpr int kMaxZ = 8;
constexpr int kRounds = 12;      // of both selections together
constexpr int kStage = 180 * 1024;  // bytes of a slice that stay in shared memory

// 2^(-j/256), in units of 2^-31.
struct Exp2Table {
  uint32_t v[256];
};
constexpr double pow2_256(int j) {  // the exponential series of j ln 2 / 256
  const double x = j * (0.6931471805599453094172321 / 256);
  double t = 1, s = 1;
  for (int i = 1; i < 24; ++i) {
    t *= x / i;
    s += t;
  }
  return s;
}
constexpr Exp2Table make_table() {
  Exp2Table t{};
  for (int j = 0; j < 256; ++j) t.v[j] = static_cast<uint32_t>(pow2_256(-j) * 0x1p31 + 0.5);
  return t;
}
__device__ constexpr Exp2Table kExp2 = make_table();

// A logit as an unsigned number of the same order.  (-0 and NaN do not come here.)
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((int32_t)k < 0 ? k & 0x7fffffffu : ~k);
}
// A logit as it counts: NaN is -inf, -0 is 0.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : x + 0.f; }

struct Weight {
  float top;     // the maximum
  float ah, al;  // log2(e) / T
};
// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 of_f2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// w of two logits (0 of NaN and -inf).  Its exponent (top - l) log2(e) / T is t + q in two
// floats, without error but for al's and q's own; k / 256 is the nearest to t, and
// 2^-(t + q) = 2^-(k / 256) 2^r with |r| <= 2^-9: the table's 32 bits times 1 + r ln 2 +
// (r ln 2)^2 / 2 in 32 bits.  2^-31 of table and series, 4e-10 of the term left out.
__device__ __forceinline__ void weight2(const Weight& p, const uint32_t* table, float l0, float l1,
                                        unsigned long long* w) {
  constexpr float kMagic = 0x1.8p23f;  // sums with it have an integer in their low bits
  constexpr float c1 = 0.69314718f * 0x1p31f, c2 = 0.24022651f * 0x1p31f;  // ln 2, ln^2 2 / 2
  const uint64_t top = f2(p.top, p.top), ah = f2(p.ah, p.ah), magic = f2(kMagic, kMagic);
  const uint64_t l = f2(l0, l1), d = sub2(top, l), v = sub2(d, top);
  const uint64_t e = sub2(sub2(top, sub2(d, v)), add2(l, v));
  float2 t = of_f2(mul2(d, f2(-p.ah, -p.ah)));    // -t
  t.x = fmaxf(t.x, -(kOne + 1.f));                // (NaN too: w is 0 from there on)
  t.y = fmaxf(t.y, -(kOne + 1.f));
  const uint64_t nt = f2(t.x, t.y);
  const uint64_t q = fma2(e, ah, fma2(d, f2(p.al, p.al), fma2(d, ah, nt)));
  const uint64_t kf = fma2(nt, f2(-256.f, -256.f), magic);
  const uint64_t r = sub2(fma2(sub2(kf, magic), f2(1.f / 256, 1.f / 256), nt), q);
  const float2 c = of_f2(fma2(r, fma2(r, f2(c2, c2), f2(c1, c1)), magic));
  const float2 k2 = of_f2(kf);
  const float ks[2] = {k2.x, k2.y}, cs[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t k = __float_as_uint(ks[i]);
    // (r of a clamped t may be anything: the shift leaves nothing of it)
    const uint32_t m = __float_as_uint(cs[i]) + (0x80000000u - 0x4b400000u);
    const unsigned long long x = (unsigned long long)table[k & 255] * m;  // 2^62 at t = 0
    w[i] = x >> (62 - kOne + ((k >> 8) & 63));
  }
}

// Fractions of 2^64: of a number in [0, 1), or the nearest to it.
__device__ __forceinline__ unsigned long long fraction(double x) {
  return !(x > 0.0) ? 0ull : x < 1.0 ? (unsigned long long)(x * 0x1p64) : ~0ull;
}

// The cluster's barrier, from code that need not have converged.
__device__ __forceinline__ void sync_cluster() {
  __syncwarp();
  tc::cluster_sync_all();
}

// A row's filters, worked out by one thread (fp64 is slow here).
struct Filters {
  Weight w;
  unsigned long long p, u;      // fractions of 2^64
  float least;                  // logit that min_p leaves (-inf: any)
  float range_k, range_p;       // what the first histograms span
  double gap;                   // T ln(min_p)
  int k;                        // 0: none
  bool some_p, some_m, greedy;
};

// What the CTAs of a cluster tell each other.
struct Shared {
  uint32_t table[256];
  alignas(16) uint32_t hist[3][kBins];  // read four at a time
  unsigned long long list[kList];        // CTA 0: the cut bin's (key, ~index)
  unsigned long long scratch[32];        // (block_exclusive_scan's size; two sums a warp)
  float best[kMaxZ];                     // of every CTA: its maximum
  float least[kMaxZ];                    // its least finite logit
  unsigned long long sum[4][kMaxZ];      // sums over its slice: two ties, the draw, the first
  int count[kMaxZ];
  uint32_t listed[kRounds], low[kRounds], high[kRounds];  // CTA 0: a round's cut bin
  unsigned long long cut[2];             // (key, ~index) of the last element left
  unsigned long long seg[kMaxZ];         // of every CTA: its part of a histogram, summed
  unsigned long long seg2[kMaxZ];
  unsigned long long kept[kWarps];       // of every warp's part: w of what top-p leaves
  unsigned long long above;
  int bin, left;
  int first, last;                       // narrow's bins
  unsigned long long mixed[2][kMaxZ];    // by_value: sums of its bins of more than a value
  int vbin[2], vties[2];                 // its cuts of top-k and top-p
  unsigned long long vmass;              // what top-k leaves
  uint32_t mine, base;                   // the CTA's elements of the cut bin, their place
  Filters f;
};

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t add_dsmem(uint32_t addr, uint32_t x) {
  uint32_t v;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(addr), "r"(x)
               : "memory");
  return v;
}
__device__ __forceinline__ void min_dsmem(uint32_t addr, uint32_t x) {
  asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void max_dsmem(uint32_t addr, uint32_t x) {
  asm volatile("red.shared::cluster.max.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

// What does not depend on the row's logits, and what does.
__device__ Filters filters(const SampleArgs& a, int r) {
  Filters f;
  const float temp = a.temperature != nullptr ? a.temperature[r] : 1.f;
  f.greedy = !(temp > 0.f);
  const float t = f.greedy ? 1.f : fmaxf(temp, 1e-30f);
  // log2(e) / T in two floats, from log2(e) in two
  constexpr float hi = 1.4426950408889634f, lo = (float)(1.4426950408889634074 - (double)hi);
  f.w.ah = hi / t;
  f.w.al = (fmaf(-f.w.ah, t, hi) + lo) / t;
  if (!(fabsf(f.w.al) < INFINITY)) f.w.al = 0.f;  // (T past 2^126, or infinite)
  f.k = a.top_k != nullptr ? a.top_k[r] : 0;
  if (f.k < 0 || f.k >= a.V) f.k = 0;
  const float p = a.top_p != nullptr ? a.top_p[r] : 1.f;
  f.some_p = p < 1.f;
  f.p = fraction(p);
  f.u = fraction(a.u[r]);
  f.range_p = (kOne + 1) * 0.6931472f * t;
  const float m = a.min_p != nullptr ? a.min_p[r] : 0.f;
  f.some_m = m > 0.f;
  f.gap = m >= 1.f || !f.some_m ? 0.0 : (double)t * log((double)m);
  return f;
}
__device__ void place_filters(Filters& f, float top, float least) {
  f.w.top = top;
  const float span = fmaxf(top - least, FLT_MIN);
  f.range_k = fminf(span, 64.f);
  f.range_p = fminf(span, f.range_p);
  f.least = -INFINITY;
  if (f.some_m) {
    // the least logit l with l - top >= T ln(min_p): rounded, then stepped
    float l = (float)((double)top + f.gap);
    for (int i = 0; i < 2 && (double)l - (double)top < f.gap; ++i) l = of_key(key_of(l) + 1);
    for (int i = 0; i < 2; ++i) {
      const float b = of_key(key_of(l) - 1);
      if (b > -INFINITY && (double)b - (double)top >= f.gap) l = b;
    }
    f.least = clean(l);
  }
}

static_assert(sizeof(Shared) + kStage + 1024 <= 227 * 1024, "a CTA's shared memory");

// Logits at a time.  (Eight doubled the loops' code, which each CTA runs for a handful of
// rounds: fetching it took longer than the loads saved.  32 rows of 126464 with every
// filter 55 us at four, 61 at eight.)
constexpr int kW = 4;

__device__ __forceinline__ void load4(const float* p, float* l) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  l[0] = v.x; l[1] = v.y; l[2] = v.z; l[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* l) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  bf16x2_to_f32(v.x, l[0], l[1]);
  bf16x2_to_f32(v.y, l[2], l[3]);
}

// Elements [from, from + num) of a row: in shared memory, or the row itself.
template <typename T, bool STAGED>
struct Row {
  static constexpr int W = kW;
  const T* x;
  int from, num;
  bool inf_top;  // (not staged: the maximum is infinite)

  __device__ __forceinline__ float one(int i) const {
    const float l = to_f32(x[i]);
    return STAGED || !inf_top ? l : l == INFINITY ? 0.f : -INFINITY;
  }
  // elements i .. i + W - 1 (i a multiple of W); -inf past the end
  __device__ __forceinline__ void load(int i, float* l) const {
    if (STAGED && i + W <= num) {
      load4(x + i, l);
    } else {
#pragma unroll
      for (int q = 0; q < W; ++q) l[q] = i + q < num ? one(i + q) : -INFINITY;
    }
  }
};

// The last element left: those of larger logits, and of equal ones up to it.
struct Cut {
  float l;
  int i;
  __device__ __forceinline__ bool has(float x, int at) const { return x > l || (x == l && at <= i); }
};
__device__ __forceinline__ Cut cut_of(unsigned long long c) {
  // (0: all but -inf)
  return c == 0 ? Cut{-INFINITY, -1} : Cut{of_key((uint32_t)(c >> 32)), (int)~(uint32_t)c};
}

template <typename T, bool STAGED>
struct Sampler {
  static constexpr int W = kW;
  Shared& sh;
  Row<T, STAGED> row;
  Weight wp;
  int rank, Z;

  __device__ __forceinline__ uint32_t remote(const void* p, int z) const {
    return tc::cluster_map(tc::smem_u32(p), z);
  }
  __device__ __forceinline__ unsigned long long w_of(float l) const {
    unsigned long long w[2];
    weight2(wp, sh.table, l, l, w);
    return w[0];
  }
  __device__ __forceinline__ void w_of_all(const float* l, unsigned long long* w) const {
#pragma unroll
    for (int q = 0; q < W; q += 2) weight2(wp, sh.table, l[q], l[q + 1], w + q);
  }
  static __device__ __forceinline__ unsigned long long pack(float l, int i) {
    return (unsigned long long)key_of(clean(l)) << 32 | (uint32_t)~i;
  }
  // f(i, l): i of the slice, W logits from it on, for all of the slice's; a warp takes
  // a contiguous part of it, 32 W at a time.
  __device__ __forceinline__ int part() const {
    return (row.num + kWarps * 32 * W - 1) / (kWarps * 32 * W) * (32 * W);
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    const int per = part(), i0 = (threadIdx.x >> 5) * per;
    for (int i = i0; i < min(i0 + per, row.num); i += 32 * W) {
      float l[W];
      const int at = i + (int)(threadIdx.x & 31) * W;
      row.load(at, l);
      f(at, l);
    }
  }

  // The first element in index order at which the running sum of f over the row exceeds
  // target(sum); f(l, index, W sums) adds up W elements from index on.  The thread that
  // has it calls found(index, its part, sum).  (Past the end f is asked of -inf.)
  template <class F, class G, class H>
  __device__ __forceinline__ void find(int slot, F f, G target, H found) {
    add_up(f);
    locate(slot, f, target, found);
  }
  // The sums of the warps' parts, into sh.scratch.
  template <class F>
  __device__ __forceinline__ void add_up(F f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long s = 0;
    each([&](int i, const float* l) {
      unsigned long long w[W];
      f(l, row.from + i, w);
#pragma unroll
      for (int q = 0; q < W; ++q) s += w[q];
    });
    s = warp_sum_u64(s);
    __syncwarp();
    __syncthreads();
    if (lane == 0) sh.scratch[warp] = s;
    __syncthreads();
  }
  template <class F, class G, class H>
  __device__ void locate(int slot, F f, G target, H found) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (threadIdx.x < Z) {
      unsigned long long t = 0;
      for (int w = 0; w < kWarps; ++w) t += sh.scratch[w];
      tc::st_dsmem_u64(remote(&sh.sum[slot][rank], threadIdx.x), t);
    }
    sync_cluster();
    unsigned long long all = 0, before = 0;
    for (int z = 0; z < Z; ++z) {
      if (z == rank) before = all;
      all += sh.sum[slot][z];
    }
    const unsigned long long want = target(all);
    // the CTA and of it the warp's part that holds it; that part again, by all warps
    int at_warp = -1;
    for (int w = 0; w < kWarps; ++w) {
      if (at_warp < 0 && want >= before && want - before < sh.scratch[w]) at_warp = w;
      if (at_warp < 0) before += sh.scratch[w];
    }
    if (at_warp < 0) return;
    const int per = part(), i0 = at_warp * per, i1 = min(i0 + per, row.num);
    unsigned long long* sums = sh.scratch + kWarps;
    for (int b = i0; b < i1; b += kWarps * 32 * W) {
      float l[W];
      unsigned long long w[W], run = 0;
      const int at = b + tid * W;
      row.load(at, l);
#pragma unroll
      for (int q = 0; q < W; ++q)
        if (at + q >= i1) l[q] = -INFINITY;  // (the next part's)
      f(l, row.from + at, w);
#pragma unroll
      for (int q = 0; q < W; ++q) run += w[q];
      const unsigned long long mine = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      if (lane == 31) sums[warp] = run;
      __syncthreads();
      unsigned long long e = before + run - mine;
      for (int v = 0; v < kWarps; ++v) {
        if (v < warp) e += sums[v];
        before += sums[v];
      }
      if (want >= e && want - e < mine) {
#pragma unroll
        for (int q = 0; q < W; ++q) {
          if (want >= e && want - e < w[q]) found(row.from + at + q, w[q], all);
          e += w[q];
        }
      }
      if (want < before) return;
      __syncthreads();
    }
  }

  // The cut that leaves `part` elements (MASS: those whose w sum up to at least part
  // 2^-64 of all that `in` leaves) of the ones that the cut `in` leaves, into
  // sh.cut[slot].
  template <bool MASS>
  __device__ void select(int slot, Cut in, unsigned long long part, float range, int& round) {
    const int tid = threadIdx.x, lane = tid & 31;
    // the first round's bins: (top - l) scale, of logits below INFINITY; then the keys
    // from khi down
    uint32_t klo = 0, khi = 0;
    int shift = -1;
    const float scale = kBins / range;
    unsigned long long above = 0, target = 0;
    auto bin_of = [&](float l) {  // < 0: not in this round
      if (shift < 0) {
        const float b = fminf((wp.top - l) * scale, (float)(kBins - 1));  // (NaN: the last)
        return (int)b;
      }
      const uint32_t key = key_of(clean(l));
      return key >= klo && key <= khi ? (int)((khi - key) >> shift) : -1;
    };
    for (;; ++round) {
      for (int i = tid; i < 3 * kBins; i += kST) (&sh.hist[0][0])[i] = 0;
      __syncthreads();
      each([&](int i, const float* l) {
        int b[W];
        bool any = false;
#pragma unroll
        for (int q = 0; q < W; ++q) {
          b[q] = in.has(l[q], row.from + i + q) ? bin_of(l[q]) : -1;
          any = any || b[q] >= 0;
        }
        if (!__any_sync(0xffffffffu, any)) return;
        if constexpr (MASS) {
          unsigned long long w[W];
          w_of_all(l, w);
#pragma unroll
          for (int q = 0; q < W; ++q) {
            constexpr uint32_t m = (1u << kLimb) - 1;
            const uint32_t x0 = (uint32_t)w[q] & m, x1 = (uint32_t)(w[q] >> kLimb) & m;
            const uint32_t x2 = (uint32_t)(w[q] >> (2 * kLimb));
            if (b[q] >= 0 && w[q] != 0) {
              atomicAdd(&sh.hist[0][b[q]], x0);
              if (w[q] >> kLimb) atomicAdd(&sh.hist[1][b[q]], x1);
              if (x2) atomicAdd(&sh.hist[2][b[q]], x2);
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < W; ++q)
            if (b[q] >= 0) atomicAdd(&sh.hist[0][b[q]], 1u);
        }
      });
      sync_cluster();
      // a CTA sums up its part of the bins over the cluster, and they tell each other
      const int nb = kBins / Z, per = max(nb / kST, 1);  // bins of a CTA, of a thread
      unsigned long long h[kPer], sum = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        h[q] = 0;
        if (q < per && tid * per + q < nb) {
          const uint32_t* at = &sh.hist[0][rank * nb + tid * per + q];
          for (int z = 0; z < Z; ++z)
#pragma unroll
            for (int m = 0; m < (MASS ? 3 : 1); ++m)
              h[q] += (unsigned long long)ld_dsmem_u32(remote(at + m * kBins, z)) << (m * kLimb);
        }
        sum += h[q];
      }
      unsigned long long all, e = block_exclusive_scan(sum, sh.scratch, &all);
      if (tid < Z) tc::st_dsmem_u64(remote(&sh.seg[rank], tid), all);
      if (tid == 0) sh.mine = 0;
      sync_cluster();
      all = 0;
      e += above;
      for (int z = 0; z < Z; ++z) {
        if (z < rank) e += sh.seg[z];
        all += sh.seg[z];
      }
      if (shift < 0) {  // (the first round)
        if constexpr (MASS) {
          target = max(__umul64hi(part, all) + (part * all != 0), 1ull);
        } else {
          target = part;
          if (all <= target) {  // no more than that are there
            if (tid == 0) sh.cut[slot] = 0;
            sync_cluster();
            ++round;
            return;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (e < target && e + h[q] >= target)
          for (int z = 0; z < Z; ++z) {
            tc::st_dsmem_u32(remote(&sh.bin, z), rank * nb + tid * per + q);
            tc::st_dsmem_u64(remote(&sh.above, z), e);
          }
        e += h[q];
      }
      sync_cluster();
      const int bin = sh.bin;
      above = sh.above;
      // its elements, into a list (where the histogram was) and from there to CTA 0's
      unsigned long long* list = reinterpret_cast<unsigned long long*>(sh.hist);
      uint32_t lo = 0xffffffffu, hi = 0;
      each([&](int i, const float* l) {
        uint32_t mine = 0;
#pragma unroll
        for (int q = 0; q < W; ++q)
          if (in.has(l[q], row.from + i + q) && bin_of(l[q]) == bin) mine |= 1u << q;
        if (mine == 0) return;
        uint32_t at = atomicAdd(&sh.mine, (uint32_t)__popc(mine));
#pragma unroll
        for (int q = 0; q < W; ++q)
          if (mine >> q & 1) {
            const unsigned long long x = pack(l[q], row.from + i + q);
            lo = min(lo, (uint32_t)(x >> 32));
            hi = max(hi, (uint32_t)(x >> 32));
            if (at < kList) list[at] = x;
            ++at;
          }
      });
      __syncthreads();
      if (tid == 0) sh.base = add_dsmem(remote(&sh.listed[round], 0), sh.mine);
      __syncthreads();
      for (uint32_t i = tid; i < min(sh.mine, (uint32_t)kList); i += kST)
        if (sh.base + i < kList) tc::st_dsmem_u64(remote(&sh.list[sh.base + i], 0), list[i]);
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (lane == 0 && lo <= hi) {
        min_dsmem(remote(&sh.low[round], 0), lo);
        max_dsmem(remote(&sh.high[round], 0), hi);
      }
      sync_cluster();
      const int m = (int)ld_dsmem_u32(remote(&sh.listed[round], 0));
      klo = ld_dsmem_u32(remote(&sh.low[round], 0));
      khi = ld_dsmem_u32(remote(&sh.high[round], 0));
      if (klo == khi) {  // nothing but ties: count them off
        const float tie = of_key(klo);
        unsigned long long c = target - above;
        if constexpr (MASS) {
          const unsigned long long w = w_of(tie);
          c = (c + w - 1) / w;
        }
        find(slot,
             [&](const float* l, int i, unsigned long long* w) {
#pragma unroll
               for (int q = 0; q < W; ++q) w[q] = l[q] == tie && in.has(l[q], i + q);
             },
             [&](unsigned long long) { return c - 1; },
             [&](int i, unsigned long long, unsigned long long) {
               for (int z = 0; z < Z; ++z) tc::st_dsmem_u64(remote(&sh.cut[slot], z), pack(tie, i));
             });
        break;
      }
      if (m <= kList) {
        if (rank == 0) finish<MASS>(slot, m, klo, khi, 0.f, above, target);
        break;
      }
      shift = max(0, 32 - __clz(khi - klo) - 11);
    }
    sync_cluster();
    ++round;
  }

  // select<true> by counts: how many elements lie in each of 12288 bins (one atomic an
  // element in place of three, and no w) says to a few 10^-4 what the sums of w above
  // every bin are, and so which few bins can hold the cut.  The pass that adds up the
  // exact w of all lists their elements, CTA 0 looks for the cut among them, and the sums
  // of what it leaves are there for the draw.  False: the elements are more than kList,
  // or the cut is not among them; the row is select's.  (256 rows of 152064, top-p:
  // 288 us by select alone, 237 so.  bf16 logits are ties by the thousand, which the
  // list does not hold.)
  __device__ bool narrow(int slot, Cut in, unsigned long long part, float range, int& round,
                         int& left) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // (a row of one CTA: half as many bins as elements; 1000 rows of 4000 99 us, 64 so)
    const int words = Z > 1 ? kWords : min(kWords, (row.num / 4 + kST - 1) / kST * kST);
    const int bins = 2 * words;
    const float scale = bins / range;
    uint32_t* hist = &sh.hist[0][0];
    auto place = [&](float l) { return fminf((wp.top - l) * scale, (float)(bins - 1)); };
    for (int i = tid; i < words; i += kST) hist[i] = 0;
    if (tid == 0) {
      sh.mine = 0;
      sh.cut[slot] = 0;
      sh.first = 0;
      sh.last = bins - 1;
    }
    __syncthreads();
    each([&](int i, const float* l) {
#pragma unroll
      for (int q = 0; q < W; ++q)
        if (in.has(l[q], row.from + i + q)) {
          const int b = (int)place(l[q]);
          atomicAdd(&hist[b >> 1], (b & 1) ? 0x10000u : 1u);
        }
    });
    sync_cluster();
    // The sums, from w of a bin's middle: off by a sixteenth of its width (by half of it
    // where all elements crowd at its edge, but over many bins that levels out).
    const int nw = words / Z, per = (nw + kST - 1) / kST, w0 = tid * per, w1 = min(w0 + per, nw);
    const float step = -range * wp.ah / bins;
    auto counts = [&](int i, uint32_t& c0, uint32_t& c1) {
      c0 = c1 = 0;
      if (Z == 1) {
        c0 = hist[i] & 0xffff;
        c1 = hist[i] >> 16;
        return;
      }
#pragma unroll
      for (int z = 0; z < kMaxZ; ++z) {
        const uint32_t v = z < Z ? ld_dsmem_u32(remote(hist + rank * nw + i, z)) : 0u;
        c0 += v & 0xffff;
        c1 += v >> 16;
      }
    };
    const float off = -step * (0.6931472f / 16) + 0x1p-14f;
    const float up = (1.f + off) * 0x1p43f, down = (1.f - off) * 0x1p43f;
    auto mid = [&](int b) { return exp2f(((float)b + 0.5f) * step); };
    auto high = [&](float w, uint32_t c) { return c * ((unsigned long long)(w * up) + 1); };
    auto low = [&](float w, uint32_t c) { return c * (unsigned long long)(w * down); };
    unsigned long long hi = 0, lo = 0, all_hi, all_lo;
    for (int i = w0; i < w1; ++i) {
      const int b = 2 * (rank * nw + i);
      uint32_t c0, c1;
      counts(i, c0, c1);
      const float m0 = mid(b), m1 = mid(b + 1);
      hi += high(m0, c0) + high(m1, c1);
      lo += low(m0, c0) + low(m1, c1);
    }
    unsigned long long eh = block_exclusive_scan(hi, sh.scratch, &all_hi);
    unsigned long long el = block_exclusive_scan(lo, sh.scratch, &all_lo);
    if (tid < Z) {
      tc::st_dsmem_u64(remote(&sh.seg[rank], tid), all_hi);
      tc::st_dsmem_u64(remote(&sh.seg2[rank], tid), all_lo);
    }
    sync_cluster();
    all_hi = all_lo = 0;
    for (int z = 0; z < Z; ++z) {
      if (z < rank) {
        eh += sh.seg[z];
        el += sh.seg2[z];
      }
      all_hi += sh.seg[z];
      all_lo += sh.seg2[z];
    }
    const unsigned long long least = max(__umul64hi(part, all_lo), 1ull);
    const unsigned long long most = __umul64hi(part, all_hi) + 1;
    const bool from = eh < least && eh + hi >= least, to = el < most && el + lo >= most;
    if (from || to) {
      for (int i = w0; i < w1; ++i) {
        uint32_t c[2];
        counts(i, c[0], c[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int b = 2 * (rank * nw + i) + q;
          const unsigned long long h = high(mid(b), c[q]), o = low(mid(b), c[q]);
          if (eh < least && eh + h >= least)
            for (int z = 0; z < Z; ++z) tc::st_dsmem_u32(remote(&sh.first, z), b);
          if (el < most && el + o >= most)
            for (int z = 0; z < Z; ++z) tc::st_dsmem_u32(remote(&sh.last, z), b);
          eh += h;
          el += o;
        }
      }
    }
    sync_cluster();
    // the exact sums, and the list (where the histogram was)
    const float b0 = (float)sh.first, b1 = (float)(sh.last + 1);
    unsigned long long* list = reinterpret_cast<unsigned long long*>(sh.hist);
    unsigned long long all = 0, above = 0;
    uint32_t klo = 0xffffffffu, khi = 0;
    each([&](int i, const float* l) {
      bool live[W], any = false;
#pragma unroll
      for (int q = 0; q < W; ++q) {
        live[q] = in.has(l[q], row.from + i + q);
        any = any || live[q];
      }
      if (!__any_sync(0xffffffffu, any)) return;
      unsigned long long w[W];
      w_of_all(l, w);
      uint32_t mine = 0;
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const float t = place(l[q]);
        if (live[q]) {
          all += w[q];
          if (t < b0) {
            above += w[q];
            ++left;
          } else if (t < b1) {
            mine |= 1u << q;
          }
        }
      }
      if (mine == 0) return;
      uint32_t at = atomicAdd(&sh.mine, (uint32_t)__popc(mine));
#pragma unroll
      for (int q = 0; q < W; ++q)
        if (mine >> q & 1) {
          const unsigned long long x = pack(l[q], row.from + i + q);
          klo = min(klo, (uint32_t)(x >> 32));
          khi = max(khi, (uint32_t)(x >> 32));
          if (at < kList) list[at] = x;
          ++at;
        }
    });
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
    if (lane == 0 && klo <= khi) {
      min_dsmem(remote(&sh.low[round], 0), klo);
      max_dsmem(remote(&sh.high[round], 0), khi);
    }
    all = warp_sum_u64(all);
    above = warp_sum_u64(above);
    __syncwarp();
    if (lane == 0) {
      sh.scratch[warp] = all;
      sh.kept[warp] = above;
    }
    __syncthreads();
    if (tid < Z) {
      all = above = 0;
      for (int w = 0; w < kWarps; ++w) {
        all += sh.scratch[w];
        above += sh.kept[w];
      }
      tc::st_dsmem_u64(remote(&sh.seg[rank], tid), all);
      tc::st_dsmem_u64(remote(&sh.seg2[rank], tid), above);
    }
    if (tid == 0) sh.base = add_dsmem(remote(&sh.listed[round], 0), sh.mine);
    __syncthreads();
    const int mine = min(sh.mine, (uint32_t)kList);
    for (uint32_t i = tid; i < mine; i += kST)
      if (sh.base + i < kList) tc::st_dsmem_u64(remote(&sh.list[sh.base + i], 0), list[i]);
    sync_cluster();
    const int m = (int)ld_dsmem_u32(remote(&sh.listed[round], 0));
    klo = ld_dsmem_u32(remote(&sh.low[round], 0));
    khi = ld_dsmem_u32(remote(&sh.high[round], 0));
    ++round;
    if (m == 0 || m > kList) {
      left = 0;
      return false;
    }
    all = above = 0;
    for (int z = 0; z < Z; ++z) {
      all += sh.seg[z];
      above += sh.seg2[z];
    }
    if (rank == 0)
      finish<true>(slot, m, klo, khi, 0.f, above,
                   max(__umul64hi(part, all) + (part * all != 0), 1ull));
    sync_cluster();
    if (sh.cut[slot] == 0) {
      left = 0;
      return false;
    }
    const Cut cut = cut_of(sh.cut[slot]);
    for (int i = tid; i < mine; i += kST) {
      const Cut x = cut_of(list[i]);
      if (!cut.has(x.l, x.i)) continue;
      atomicAdd(&sh.kept[(x.i - row.from) / this->part()], w_of(x.l));
      ++left;
    }
    __syncthreads();
    return true;
  }

  // top-k and top-p of bf16 rows by counts: a bin of the histogram is one value, so w of a
  // bin's elements is its count times w of the value, exactly, and one pass that works out
  // no w gives both cuts.  12288 values from the maximum down, but for those below
  // 2^-12 in size, which are one bin, and what lies further down, which is the last: w of
  // these two's elements is summed up one by one.  False: a cut falls on one of the two, and the
  // row is select's.  (32 rows of 126464 with every filter: 58 us by select, 46 so; 256
  // rows of 152064 with top-k 212 and 200.)
  __device__ __forceinline__ int code(float l) const {  // of the same order as l
    const int size = (int)(__float_as_uint(l) >> 16 & 0x7fff) - 0x397f;  // (2^-12: 1)
    return size <= 0 ? 0 : l < 0.f ? -size : size;
  }
  __device__ bool by_value(int k, bool some_p, unsigned long long part, Cut& cut) {
    const int tid = threadIdx.x;
    uint32_t* hist = &sh.hist[0][0];
    const int top = code(wp.top);
    for (int i = tid; i < kWords; i += kST) hist[i] = 0;
    if (tid < 2) {
      sh.vbin[tid] = -1;
      sh.kept[tid] = 0;
    }
    __syncthreads();
    each([&](int, const float* l) {
#pragma unroll
      for (int q = 0; q < W; ++q)
        if (l[q] > -INFINITY) {
          const int c = code(l[q]), b = min(top - c, kFine - 1);
          atomicAdd(&hist[b >> 1], (b & 1) ? 0x10000u : 1u);
          if (c == 0 || b == kFine - 1) atomicAdd(&sh.kept[b == kFine - 1], w_of(l[q]));
        }
    });
    __syncwarp();
    __syncthreads();
    if (tid < 2 * Z) tc::st_dsmem_u64(remote(&sh.mixed[tid & 1][rank], tid >> 1), sh.kept[tid & 1]);
    sync_cluster();
    const int nw = kWords / Z, per = (nw + kST - 1) / kST, w0 = tid * per, w1 = min(w0 + per, nw);
    auto counts = [&](int i, uint32_t* c) {
      c[0] = c[1] = 0;
      if (Z == 1) {
        c[0] = hist[i] & 0xffff;
        c[1] = hist[i] >> 16;
        return;
      }
#pragma unroll
      for (int z = 0; z < kMaxZ; ++z) {
        const uint32_t v = z < Z ? ld_dsmem_u32(remote(hist + rank * nw + i, z)) : 0u;
        c[0] += v & 0xffff;
        c[1] += v >> 16;
      }
    };
    auto value = [&](int b) {  // of a bin but the two
      const int c = top - b, size = c < 0 ? -c : c;
      return __uint_as_float((uint32_t)(size + 0x397f) << 16 | (c < 0 ? 0x80000000u : 0u));
    };
    auto mixed = [&](int b) { return b == top || b == kFine - 1; };
    auto mass = [&](int b, uint32_t c) {
      if (c == 0) return 0ull;
      if (!mixed(b)) return c * w_of(value(b));
      unsigned long long t = 0;
      for (int z = 0; z < Z; ++z) t += sh.mixed[b == kFine - 1][z];
      return t;
    };
    unsigned long long n = 0, m = 0, all_n, all_m;
    for (int i = w0; i < w1; ++i) {
      const int b = 2 * (rank * nw + i);
      uint32_t c[2];
      counts(i, c);
      n += c[0] + c[1];
      m += mass(b, c[0]) + mass(b + 1, c[1]);
    }
    const unsigned long long en0 = block_exclusive_scan(n, sh.scratch, &all_n);
    const unsigned long long em0 = block_exclusive_scan(m, sh.scratch, &all_m);
    if (tid < Z) {
      tc::st_dsmem_u64(remote(&sh.seg[rank], tid), all_n);
      tc::st_dsmem_u64(remote(&sh.seg2[rank], tid), all_m);
    }
    sync_cluster();
    unsigned long long before_n = en0, before_m = em0;
    all_m = 0;
    for (int z = 0; z < Z; ++z) {
      if (z < rank) {
        before_n += sh.seg[z];
        before_m += sh.seg2[z];
      }
      all_m += sh.seg2[z];
    }
    // the cut on which a thread's bins come to `target`, by count or by mass
    auto look = [&](int which, unsigned long long target) {
      unsigned long long en = before_n, em = before_m;
      const unsigned long long e = which ? em : en;
      if (e < target && e + (which ? m : n) >= target) {
        for (int i = w0; i < w1; ++i) {
          uint32_t c[2];
          counts(i, c);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int b = 2 * (rank * nw + i) + q;
            const unsigned long long x = mass(b, c[q]);
            const unsigned long long f = which ? em : en, add = which ? x : c[q];
            if (f < target && f + add >= target) {
              const unsigned long long w = mixed(b) ? 1 : w_of(value(b));
              const unsigned long long ties = which ? (target - f + w - 1) / w : target - f;
              for (int z = 0; z < Z; ++z) {
                tc::st_dsmem_u32(remote(&sh.vbin[which], z), b);
                tc::st_dsmem_u32(remote(&sh.vties[which], z), ties >= c[q] ? INT_MAX : (int)ties);
                if (!which)
                  tc::st_dsmem_u64(remote(&sh.vmass, z),
                                   em + min(ties, (unsigned long long)c[q]) * w);
              }
            }
            en += c[q];
            em += x;
          }
        }
      }
      sync_cluster();
    };
    if (k > 0) {
      look(0, k);
      if (sh.vbin[0] >= 0) {
        if (mixed(sh.vbin[0])) return false;
        all_m = sh.vmass;
      }
    }
    if (some_p) look(1, max(__umul64hi(part, all_m) + (part * all_m != 0), 1ull));
    const int b = some_p ? sh.vbin[1] : sh.vbin[0], ties = some_p ? sh.vties[1] : sh.vties[0];
    if (b < 0) return true;
    if (mixed(b)) return false;
    cut = Cut{value(b), INT_MAX};
    if (ties < INT_MAX) {  // so many of them, in order of their index
      find(0,
           [&](const float* l, int, unsigned long long* w) {
#pragma unroll
             for (int q = 0; q < W; ++q) w[q] = l[q] == cut.l;
           },
           [&](unsigned long long) { return (unsigned long long)ties - 1; },
           [&](int i, unsigned long long, unsigned long long) {
             for (int z = 0; z < Z; ++z) tc::st_dsmem_u64(remote(&sh.cut[0], z), pack(cut.l, i));
           });
      sync_cluster();
      cut = cut_of(sh.cut[0]);
    }
    return true;
  }

  // top-k and top-p of a row that the list holds.
  __device__ void by_list(int k, bool some_p, unsigned long long part, float range_k, float range_p,
                          Cut& cut) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
      sh.mine = 0;
      sh.cut[0] = 0;
    }
    __syncthreads();
    for (int i = tid; i < row.num; i += kST) {
      const float l = row.one(i);
      if (l > -INFINITY) sh.list[atomicAdd(&sh.mine, 1u)] = pack(l, i);
    }
    __syncthreads();
    const int m = (int)sh.mine;
    if (k > 0) {
      if (k < m) finish<false>(0, m, 0, 0, kST / range_k, 0, k);
      sync_cluster();
      cut = cut_of(sh.cut[0]);
    }
    if (!some_p) return;
    unsigned long long all = 0;
    for (int i = tid; i < m; i += kST) {
      const Cut x = cut_of(sh.list[i]);
      if (cut.has(x.l, x.i)) all += w_of(x.l);
    }
    all = warp_sum_u64(all);
    if (lane == 0) sh.scratch[warp] = all;
    __syncthreads();
    all = 0;
    for (int w = 0; w < kWarps; ++w) all += sh.scratch[w];
    __syncthreads();
    // (what the first cut leaves comes first: the sums up to the second are those of the list)
    finish<true>(1, m, 0, 0, kST / range_p, 0,
                 max(__umul64hi(part, all) + (part * all != 0), 1ull));
    sync_cluster();
    cut = cut_of(sh.cut[1]);
  }

  // CTA 0: of the list's m elements, with keys from klo to khi, the one whose sum reaches
  // target: sums of kST bins by key (scale > 0: by distance from the maximum), then the
  // elements of the bin (a few), each with those before it.  Where the bin holds more than a
  // warp, the list is sorted.  (Sorting it always took 16 K cycles: 45 steps of all warps,
  // next to another CTA's work.)
  template <bool MASS>
  __device__ void finish(int slot, int m, uint32_t klo, uint32_t khi, float scale,
                         unsigned long long above, unsigned long long target) {
    const int tid = threadIdx.x;
    // (behind the CTA's own list in the histogram's place)
    unsigned long long* bins = reinterpret_cast<unsigned long long*>(sh.hist) + kList;
    unsigned long long* few = bins + kST;
    static_assert((kList + kST + 32) * 8 <= kBins * 12 && kList == 2 * kST, "the list and bins");
    const int shift = max(0, 32 - __clz(khi - klo) - 9);
    auto w_in = [&](unsigned long long x) { return MASS ? w_of(of_key((uint32_t)(x >> 32))) : 1ull; };
    auto bin_of = [&](unsigned long long x) {
      const uint32_t key = (uint32_t)(x >> 32);
      return scale > 0.f ? (int)fminf((wp.top - of_key(key)) * scale, kST - 1.f)
                         : (int)((khi - key) >> shift);
    };
    bins[tid] = 0;
    if (tid == 0) sh.base = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kST) {
      const unsigned long long x = sh.list[i];
      atomicAdd(&bins[bin_of(x)], w_in(x));
    }
    __syncthreads();
    unsigned long long all;
    const unsigned long long b = bins[tid];
    const unsigned long long e = above + block_exclusive_scan(b, sh.scratch, &all);
    if (tid == 0) sh.bin = -1;
    __syncthreads();
    if (e < target && e + b >= target) {
      sh.bin = tid;
      sh.above = e;
    }
    __syncthreads();
    if (sh.bin < 0) return;  // (the cut is not in the list)
    for (int i = tid; i < m; i += kST) {
      const unsigned long long x = sh.list[i];
      if (bin_of(x) == sh.bin) {
        const uint32_t at = atomicAdd(&sh.base, 1u);
        if (at < 32) few[at] = x;
      }
    }
    __syncthreads();
    const int num = (int)sh.base;
    if (num <= 32) {
      if (tid < 32) {
        const unsigned long long x = tid < num ? few[tid] : 0, w = tid < num ? w_in(x) : 0;
        unsigned long long before = sh.above;
        for (int i = 0; i < num; ++i) {
          const unsigned long long y = __shfl_sync(0xffffffffu, x, i);
          const unsigned long long v = __shfl_sync(0xffffffffu, w, i);
          if (y > x) before += v;
        }
        if (before < target && before + w >= target)
          for (int z = 0; z < Z; ++z) tc::st_dsmem_u64(remote(&sh.cut[slot], z), x);
      }
      return;
    }
    int n = 2;
    while (n < m) n <<= 1;
    for (int i = m + tid; i < n; i += kST) sh.list[i] = 0;
    for (int size = 2; size <= n; size <<= 1) {
      for (int gap = size >> 1; gap > 0; gap >>= 1) {
        __syncthreads();
        for (int t = tid; t < n / 2; t += kST) {
          const int i = 2 * t - (t & (gap - 1)), j = i + gap;
          const unsigned long long x = sh.list[i], y = sh.list[j];
          if ((x < y) == ((i & size) == 0)) {  // descending
            sh.list[i] = y;
            sh.list[j] = x;
          }
        }
      }
    }
    __syncthreads();
    unsigned long long x[2], w[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = 2 * tid + q;
      x[q] = i < m ? sh.list[i] : 0;
      w[q] = i < m ? w_in(x[q]) : 0;
    }
    unsigned long long f = above + block_exclusive_scan(w[0] + w[1], sh.scratch, &all);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (f < target && f + w[q] >= target)
        for (int z = 0; z < Z; ++z) tc::st_dsmem_u64(remote(&sh.cut[slot], z), x[q]);
      f += w[q];
    }
  }
};

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kST, 2)
k_sample(const __grid_constant__ SampleArgs a) {
  pdl_prologue();
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  T* stage = reinterpret_cast<T*>(smem + ((sizeof(Shared) + 15) & ~size_t(15)));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Z = a.Z, r = blockIdx.x / Z, rank = blockIdx.x - r * Z;
  const T* logits = static_cast<const T*>(a.logits) + (long)r * a.ld;
  const int from = rank * a.slice, num = max(0, min(a.slice, a.V - from));
  for (int i = tid; i < 256; i += kST) sh.table[i] = kExp2.v[i];
  if (tid == 0) sh.left = 0;
  if (tid == kST - 32) sh.f = filters(a, r);  // (slow: while the others load)
  if (tid < kRounds) {
    sh.listed[tid] = 0;
    sh.low[tid] = 0xffffffffu;
    sh.high[tid] = 0;
  }
  // ---- the slice, its maximum and its least finite logit (NaN counts for neither)
  float top = -INFINITY, least = INFINITY;
  auto see = [&](float x) {
    top = fmaxf(top, x);
    least = fminf(least, x > -INFINITY ? x : INFINITY);
  };
  constexpr int L = Vec<T>::n;
  if (a.vec) {
#pragma unroll 4
    for (int i = tid * L; i < num; i += kST * L) {
      if (i + L <= num) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(logits + from + i));
        if (STAGED) *reinterpret_cast<uint4*>(stage + i) = v;
        float x[L];
        unpack16(v, x, T{});
#pragma unroll
        for (int q = 0; q < L; ++q) see(x[q]);
      } else {
        for (int q = i; q < num; ++q) {
          const T v = logits[from + q];
          if (STAGED) stage[q] = v;
          see(to_f32(v));
        }
      }
    }
  } else {
#pragma unroll 4
    for (int i = tid; i < num; i += kST) {
      const T v = logits[from + i];
      if (STAGED) stage[i] = v;
      see(to_f32(v));
    }
  }
  top = warp_max(top);
  least = -warp_max(-least);
  __shared__ float s_top[kWarps], s_least[kWarps];
  if (lane == 0) {
    s_top[warp] = top;
    s_least[warp] = least;
  }
  sync_cluster();  // (the first: the other CTAs' shared memory is there)
  if (tid < Z) {
    for (int w = 0; w < kWarps; ++w) {
      top = w == 0 ? s_top[0] : fmaxf(top, s_top[w]);
      least = w == 0 ? s_least[0] : fminf(least, s_least[w]);
    }
    tc::st_dsmem_f32(tc::cluster_map(tc::smem_u32(&sh.best[rank]), tid), top);
    tc::st_dsmem_f32(tc::cluster_map(tc::smem_u32(&sh.least[rank]), tid), least);
  }
  sync_cluster();
  top = -INFINITY;
  least = INFINITY;
  for (int z = 0; z < Z; ++z) {
    top = fmaxf(top, sh.best[z]);
    least = fminf(least, sh.least[z]);
  }
  if (!(top > -INFINITY)) {  // the row holds nothing (every CTA of it sees that)
    if (rank == 0 && tid == 0) {
      a.token[r] = -1;
      if (a.prob != nullptr) a.prob[r] = 0.f;
      if (a.n != nullptr) a.n[r] = 0;
    }
    sync_cluster();
    return;
  }
  // an infinite maximum counts as 0, the others as -inf
  const bool inf_top = top == INFINITY;
  if (inf_top) {
    top = 0.f;
    least = 0.f;
  }
  // ---- the row's filters
  if (tid == 0) place_filters(sh.f, top, least);
  __syncthreads();
  const Filters f = sh.f;
  Row<T, STAGED> row{STAGED ? stage : logits + from, from, num, inf_top};
  if (inf_top && STAGED) {
    for (int i = tid; i < num; i += kST) {
      const float x = to_f32(stage[i]);
      Store<T>::put(stage + i, x == INFINITY ? 0.f : -INFINITY);
    }
    __syncthreads();
  }
  Sampler<T, STAGED> s{sh, row, f.w, rank, Z};
  Cut cut{-INFINITY, -1};
  int round = 0;
  bool done = false;
  if ((f.k > 0 || f.some_p) && a.V <= kList && f.range_k > 1e-30f && f.range_p > 1e-30f &&
      f.range_p < 1e30f) {
    // (1000 rows of 1000 with top-p: fp32 92 us by narrow, bf16 76 by value, 43 so)
    s.by_list(f.k, f.some_p, f.p, f.range_k, f.range_p, cut);
    done = true;
  }
  if constexpr (sizeof(T) == 2)  // (a bin's count has 16 bits)
    done = done || ((f.k > 0 || f.some_p) && a.slice < 65536 &&
                    s.by_value(f.k, f.some_p, f.p, cut));
  if (f.k > 0 && !done) {
    s.template select<false>(0, cut, f.k, f.range_k, round);
    cut = cut_of(sh.cut[0]);
  }
  int left = 0;
  bool summed = false;  // sh.kept has the sums of what is left
  if (f.some_p && !done) {
    if constexpr (sizeof(T) == 4)  // (a bin's count has 16 bits; 12288 / range is finite)
      summed = a.slice < 65536 && f.range_p > 1e-30f && f.range_p < 1e30f &&
               s.narrow(1, cut, f.p, f.range_p, round, left);
    if (!summed) s.template select<true>(1, cut, f.p, f.range_p, round);
    cut = cut_of(sh.cut[1]);
  }
  if (f.least > cut.l) {
    cut = Cut{f.least, INT_MAX};  // (all of its ties)
    summed = false;
    left = 0;
  }
  // ---- the draw
  constexpr int W = kW;
  const bool whole = cut.l == -INFINITY;
  bool counting = !summed;  // in the first pass
  auto weights = [&](const float* l, int i, unsigned long long* w) {
    if (whole) {  // (w of -inf and NaN is 0)
      s.w_of_all(l, w);
      if (counting) {
#pragma unroll
        for (int q = 0; q < W; ++q) left += l[q] > -INFINITY;
      }
      return;
    }
    bool live[W], any = false;
#pragma unroll
    for (int q = 0; q < W; ++q) {
      live[q] = cut.has(l[q], i + q);
      any = any || live[q];
      w[q] = 0;
    }
    if (__any_sync(0xffffffffu, any)) {
      unsigned long long x[W];
      s.w_of_all(l, x);
#pragma unroll
      for (int q = 0; q < W; ++q) {
        w[q] = live[q] ? x[q] : 0;
        if (counting) left += live[q];
      }
    }
  };
  auto drawn = [&](unsigned long long all) {
    counting = false;
    return f.greedy ? ~0ull : __umul64hi(f.u, all);
  };
  if (summed) {
    if (tid < kWarps) sh.scratch[tid] = sh.kept[tid];
    __syncthreads();
  } else {
    s.add_up(weights);
  }
  s.locate(2, weights, drawn, [&](int i, unsigned long long w, unsigned long long all) {
    a.token[r] = i;
    if (a.prob != nullptr) a.prob[r] = (float)w / (float)all;
  });
  if (f.greedy)  // the first of the maximum
    s.find(3,
           [&](const float* l, int, unsigned long long* w) {
#pragma unroll
             for (int q = 0; q < W; ++q) w[q] = l[q] == top;
           },
           [](unsigned long long) { return 0ull; },
           [&](int i, unsigned long long, unsigned long long) {
             unsigned long long all = 0;
             for (int z = 0; z < Z; ++z) all += sh.sum[2][z];
             a.token[r] = i;
             if (a.prob != nullptr) a.prob[r] = (float)(1ull << kOne) / (float)all;
           });
  left = __reduce_add_sync(0xffffffffu, left);
  if (lane == 0) atomicAdd(&sh.left, left);
  __syncthreads();
  if (tid == 0)
    tc::st_dsmem_u32(tc::cluster_map(tc::smem_u32(&sh.count[rank]), 0), (uint32_t)sh.left);
  sync_cluster();  // no CTA leaves while another may still write to it
  if (rank == 0 && tid == 0 && a.n != nullptr) {
    int n = 0;
    for (int z = 0; z < Z; ++z) n += sh.count[z];
    a.n[r] = n;
  }
}

template <typename T, bool STAGED>
cudaError_t launch(const SampleArgs& a, cudaStream_t s) {
  auto kern = k_sample<T, STAGED>;
  const size_t smem = align_up(sizeof(Shared), 16) + (STAGED ? (size_t)a.slice * sizeof(T) : 0);
  static DeviceOnce once;
  const cudaError_t e = allow_smem(kern, 227 * 1024 - 256, once);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.R * a.Z);
  cfg.blockDim = dim3(kST);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)a.Z, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_ex(cfg, kern, a);
}

template <typename T>
cudaError_t run(SampleArgs a, cudaStream_t s) {
  // CTAs a row: slices of at most 48 KB, so that two CTAs share an SM; for few rows
  // more, down to slices of 2048 logits, until the SMs are covered.
  a.Z = 1;
  while (a.Z < kMaxZ && ((size_t)a.V * sizeof(T) > a.Z * size_t(48 << 10) ||
                         ((long)a.R * a.Z < kSmTarget && a.V > a.Z * 2048)))
    a.Z *= 2;
  a.slice = ceil_div(ceil_div(a.V, a.Z), 16) * 16;
  a.vec = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
          (a.R == 1 || a.ld * (long)sizeof(T) % 16 == 0);
  return (size_t)a.slice * sizeof(T) <= kStage ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

cudaError_t sample_run(SampleArgs a, cudaStream_t s) {
  return a.dtype == PS_F32 ? run<float>(a, s) : run<__nv_bfloat16>(a, s);
}

}  // namespace ps
