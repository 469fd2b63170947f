// Attention over a 4-bit KV cache, and the weight it puts on each slot.
//
//   k_kv4_attn     online-softmax attention of 8 or 16 rows of one KV head's
//                  queries over a share of its slots
//   k_kv4_combine  the shares of a row joined
//   k_kv4_weight   column sums of exp(s - lse), K only
//
// The rows of a KV head are its T tokens times the G = Hq / Hkv query heads it
// serves (row t G + j), so a head's K and V are read once for all of them.
//
// A warp works alone on 16 slots at a time, from its own cp.async ring into
// m16n8k16 operand fragments (f16, fp32 accumulators), the slots as the 16 and
// the query rows as the 8, since one token has few rows (the rows as the 16 took
// 118 us where this takes 94, without the ring):
//   S^T = K Q^T  the 16 contraction indices of a step may be any 16 elements as
//     long as Q and K agree: lane (g, t) = (lane / 4, lane % 4) takes elements
//     [t dh/4, (t+1) dh/4) of slots g and g + 8, one contiguous piece each, and
//     step ks uses elements 4 ks .. 4 ks + 3 of them.  Q is laid out in that
//     order in shared memory.
//   O^T = V^T P^T  P^T needs the slots where S^T has the rows: one 8 x 8
//     transpose instruction each 8 slots.  Lane (g, t) then multiplies V of
//     slots 2t, 2t+1, 2t+8, 2t+9, elements [g dh/8, (g+1) dh/8), which it loads
//     itself; the codes of two slots are interleaved before they are converted,
//     so that a conversion gives a pair of slots.
// Q is scaled by a power of two of its row's own (2^14 <= max |q| < 2^15), so
// bf16 queries are exact in f16 down to 2^-25 of the row's largest; fp32
// queries and P take two f16 terms (hi + lo).  P carries a factor 2^kPShift,
// which keeps small weights out of f16's subnormals.
//
// What bounds k_kv4_attn: the codes are read once, 0.56 bytes an element, and
// cost two conversions and a product an f16 pair, so a long cache is held up by
// instructions and the ring's waits before memory: 8 tokens on 64 K slots of 4
// heads (302 MB) 59 us, 5.1 TB/s, 75 % of a copy's rate; few slots by the launch
// and the length of one warp's chain (1024 slots: 6 us).  k_kv4_weight reads K
// alone and is bound by its instructions: 8 tokens on 32 K slots (84 MB with the
// weights) 21 us, 4 TB/s.
#include "kv4.cuh"
#include "tc.cuh"

namespace ps {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kGrow = 4.f;      // log2 growth of a maximum before O is rescaled
constexpr int kMaxCluster = 8;    // CTAs of a portable cluster
constexpr float kNoMax = -FLT_MAX;  // a maximum that every score outgrows
// Rows [m0, m0 + rows) of (b, hkv) into shared memory as B fragments
// [row / 8][part][ks / 2][lane] (uint4: two steps' pairs), with their constants;
// rows past M are zero and see nothing.  DH / 8 lanes a row, every load of a
// thread issued before the first is used.
template <int DH, bool F32>
__device__ __forceinline__ void stage_rows(const Kv4AttnArgs& a, int b, int hkv, int m0, int rows,
                                           uint4* qs, RowPar* par) {
  constexpr int KS = DH / 16, LN = DH / 8, P = F32 ? 2 : 1;
  const int sub = threadIdx.x % LN, step = blockDim.x / LN;
  for (int r = threadIdx.x / LN; r < rows; r += step) {
    const int m = m0 + r;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    RowPar p{0.f, INFINITY, 0.f, 0, INT32_MAX, INT32_MIN};
    if (m < a.M) {
      const int t = row_token(a, m), h = hkv * a.G + (m - t * a.G);
      const long tok = (long)b * a.T + t;
      const long at = (long)b * a.q_bld + (long)t * a.q_ld + (long)h * DH + sub * 8;
      if constexpr (F32) {
        load16(static_cast<const float*>(a.Q) + at, x);
        load16(static_cast<const float*>(a.Q) + at + 4, x + 4);
      } else {
        load16(static_cast<const __nv_bfloat16*>(a.Q) + at, x);
      }
      p.slope = a.slope != nullptr ? a.slope[h] : 0.f;
      const int lo = a.span != nullptr ? a.span[2 * tok] : INT32_MIN;
      const int hi = a.span != nullptr ? a.span[2 * tok + 1] : INT32_MAX;
      if (a.span == nullptr || lo < hi) {
        p.lo = lo;
        p.last = a.span != nullptr ? hi - 1 : INT32_MAX;
      }
      p.qpos = a.qpos != nullptr ? a.qpos[tok] : 0;
      p.lse = a.lse_in != nullptr ? a.lse_in[tok * a.Hq + h] : -INFINITY;
    }
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
    const uint32_t mask = (uint32_t)((1ull << LN) - 1) << ((threadIdx.x & 31) & ~(LN - 1));
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(mask, mx, o));
    float up;
    float f;
    row_scale(mx, a.scale, &up, &f);
    if (m < a.M) p.f = f;
    if (sub == 0) par[r] = p;
    // elements 8 sub .. 8 sub + 7: lane t = d / (DH / 4) of the fragment, steps
    // ks = d % (DH / 4) / 4 and the next, two pairs each
    const int t = 8 * sub / (DH / 4), ks = 8 * sub % (DH / 4) / 4;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v0 = x[2 * e] * up, v1 = x[2 * e + 1] * up;
      const __half2 h = __floats2half2_rn(v0, v1);
      hi[e] = h2_bits(h);
      if constexpr (F32) {
        const float2 back = __half22float2(h);
        lo[e] = h2_bits(__floats2half2_rn(v0 - back.x, v1 - back.y));
      }
    }
    uint4* at = qs + ((size_t)(r / 8) * P * (KS / 2) + ks / 2) * 32 + (r % 8) * 4 + t;
    *at = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (F32) at[(KS / 2) * 32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// A warp's own two stages of 32 slots (two 16-slot steps) in shared memory, one
// filled with cp.async while the other is used: codes and scales as they lie in
// the cache.  (Loaded straight into registers one step ahead, too few bytes were
// in flight: 90 us against 54 with V left out, on 64 K slots x 8 sequences x 4
// heads.)
constexpr int kStep = 32;
template <int DH, bool WITH_V>
struct Ring {
  static constexpr int kCode = kStep * (DH / 2), kScale = kStep * (DH / 16);
  static constexpr int kV = kCode + kScale;            // V's codes, then its scales
  static constexpr int kStage = WITH_V ? 2 * kV : kV;
  static constexpr int kBytes = 2 * kStage;
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool in) {
  const int n = in ? BYTES : 0;  // nothing read, zeros written
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Fills a lane's part of the stages, kStep slots at a time, `stride` slots on each
// time: the 16-byte pieces of codes lane, lane + 32, ..., and the scales of slot
// `lane`.  Zeros past the cache.
template <int DH, bool WITH_V>
struct RingFill {
  using R = Ring<DH, WITH_V>;
  static constexpr int kPieces = DH / 32;  // of codes a lane
  const uint8_t *kc, *vc, *ks, *vs;
  int left;

  __device__ __forceinline__ RingFill(const Kv4AttnArgs& a, long bh, int n) {
    const int lane = threadIdx.x & 31;
    const long row = bh * a.Ncache + n;
    left = a.Ncache - n;
    kc = a.kcode + row * (DH / 2) + lane * 16;
    vc = a.vcode + row * (DH / 2) + lane * 16;
    ks = a.kscale + (row + lane) * (DH / 16);
    vs = a.vscale + (row + lane) * (DH / 16);
  }
  __device__ __forceinline__ void next(uint32_t dst, int stride) {
    const int lane = threadIdx.x & 31;
    const uint32_t d = dst + lane * 16, sd = dst + R::kCode + lane * (DH / 16);
    if (left >= kStep) {  // warp-uniform
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        cp_async<16>(d + 512 * i, kc + 512 * i, true);
        if constexpr (WITH_V) cp_async<16>(d + R::kV + 512 * i, vc + 512 * i, true);
      }
      cp_async<DH / 16>(sd, ks, true);
      if constexpr (WITH_V) cp_async<DH / 16>(sd + R::kV, vs, true);
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const bool in = lane / (DH / 32) + i * (1024 / DH) < left;
        cp_async<16>(d + 512 * i, in ? kc + 512 * i : kc - lane * 16, in);
        if constexpr (WITH_V)
          cp_async<16>(d + R::kV + 512 * i, in ? vc + 512 * i : vc - lane * 16, in);
      }
      const bool in = lane < left;
      const int back = in ? 0 : lane * (DH / 16);
      cp_async<DH / 16>(sd, ks - back, in);
      if constexpr (WITH_V) cp_async<DH / 16>(sd + R::kV, vs - back, in);
    }
    kc += (long)stride * (DH / 2);
    ks += (long)stride * (DH / 16);
    if constexpr (WITH_V) {
      vc += (long)stride * (DH / 2);
      vs += (long)stride * (DH / 16);
    }
    left -= stride;
  }
};

// The slot that stands at index r of a 16-slot step: 0 4 1 5 2 6 3 7, and 8 more
// for the second half.  Indices 2t, 2t+1, 2t+8, 2t+9 are then slots t, t+4, t+8,
// t+12, so that the lanes of a V load read neighbouring rows (no bank is hit
// twice).
__device__ __forceinline__ int slot_at(int r) { return (r & 8) | ((r & 1) << 2) | ((r & 7) >> 1); }

// What a lane reads of step h of a stage: K of slots slot_at(g) and slot_at(g) + 8,
// elements [t dh/4, (t+1) dh/4); V of slots t + 4 j, elements [g dh/8, (g+1)
// dh/8); the block scales that go with them.
template <int DH>
struct RawK {
  uint32_t c[2][DH / 32];
  uint32_t s[2];
};
template <int DH>
struct RawV {
  uint32_t c[4][DH / 64];
  uint32_t s[4];
};

template <int DH>
__device__ __forceinline__ void read_k(const uint8_t* st, int h, int g, int t, RawK<DH>& o) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int slot = 16 * h + slot_at(g) + 8 * j;
    const uint8_t* p = st + slot * (DH / 2) + t * (DH / 8);
    const uint8_t* q = st + kStep * (DH / 2) + slot * (DH / 16) + t * (DH / 64);
    if constexpr (DH == 64) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      o.c[j][0] = v.x; o.c[j][1] = v.y;
      o.s[j] = *q;
    } else {
#pragma unroll
      for (int i = 0; i < DH / 128; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        o.c[j][4 * i] = v.x; o.c[j][4 * i + 1] = v.y;
        o.c[j][4 * i + 2] = v.z; o.c[j][4 * i + 3] = v.w;
      }
      if constexpr (DH == 128) o.s[j] = *reinterpret_cast<const uint16_t*>(q);
      else o.s[j] = *reinterpret_cast<const uint32_t*>(q);
    }
  }
}

template <int DH>
__device__ __forceinline__ void read_v(const uint8_t* st, int h, int g, int t, RawV<DH>& o) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int slot = 16 * h + t + 4 * j;
    const uint8_t* p = st + slot * (DH / 2) + g * (DH / 16);
    const uint8_t* q = st + kStep * (DH / 2) + slot * (DH / 16);
    if constexpr (DH == 64) {
      o.c[j][0] = *reinterpret_cast<const uint32_t*>(p);
      o.s[j] = q[g >> 1];
    } else if constexpr (DH == 128) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      o.c[j][0] = v.x; o.c[j][1] = v.y;
      o.s[j] = q[g];
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      o.c[j][0] = v.x; o.c[j][1] = v.y; o.c[j][2] = v.z; o.c[j][3] = v.w;
      o.s[j] = reinterpret_cast<const uint16_t*>(q)[g];
    }
  }
}

// Word w of the lane's K as A fragments of steps 2 w and 2 w + 1.
template <int DH>
__device__ __forceinline__ void dequant_k(const RawK<DH>& r, int w, uint32_t* a0, uint32_t* a1) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    // eight elements a word, two words a scale, two scales a conversion
    const uint32_t two = h2_bits(e4m3x2_f16(DH == 64 ? r.s[j] : r.s[j] >> (16 * (w / 4))));
    const __half2 s = h2_of(__byte_perm(two, two, (w / 2) & 1 ? 0x3232u : 0x1010u));
    uint32_t h[4];
    e2m1x8_f16(r.c[j][w], h);
    a0[j] = h2_bits(__hmul2(h2_of(h[0]), s));
    a0[2 + j] = h2_bits(__hmul2(h2_of(h[1]), s));
    a1[j] = h2_bits(__hmul2(h2_of(h[2]), s));
    a1[2 + j] = h2_bits(__hmul2(h2_of(h[3]), s));
  }
}

// s += two steps' products of K with the queries: hi (and for fp32 queries lo).
// The tensor cores truncate what they add to an accumulator, by up to 2^-23 of
// it each time, and a chain of 16 of them showed in fp32 weights (1.4e-6): fp32
// products of 32 elements are added by a rounding instruction.
template <bool F32>
__device__ __forceinline__ void add_products(float* s, const uint32_t* a0, const uint32_t* a1,
                                             const uint4& hi, const uint4& lo) {
  if constexpr (F32) {
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    mma_f16(d, a0, lo.x, lo.y);
    mma_f16(d, a1, lo.z, lo.w);
    mma_f16(d, a0, hi.x, hi.y);
    mma_f16(d, a1, hi.z, hi.w);
#pragma unroll
    for (int c = 0; c < 4; ++c) s[c] += d[c];
  } else {
    mma_f16(s, a0, hi.x, hi.y);
    mma_f16(s, a1, hi.z, hi.w);
  }
}

// Codes of word w of slots a and b interleaved before they are converted: byte q
// of *even holds element 2 q of both, of *odd element 2 q + 1.
__device__ __forceinline__ void pair_codes(uint32_t a, uint32_t b, uint32_t* even, uint32_t* odd) {
  *even = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
  *odd = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
}

// The 8 x 8 matrix of 16-bit values that a warp holds (lane 4 i + j: row i,
// columns 2 j and 2 j + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// tanh of four scores / cap to fp32's precision, for a whole warp.
__device__ __forceinline__ void tanh4(float* y) {
  const float top = max3(fmaxf(fabsf(y[0]), fabsf(y[1])), fabsf(y[2]), fabsf(y[3]));
  if (__all_sync(0xffffffffu, top <= kTanhTop)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = tanh_small(y[c]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = tanhf(y[c]);
  }
}

// What an instance takes: no bias nor explicit positions; those too; and, of bf16
// queries, caps past kCapAbs (whose formula in every instance made 8 tokens on 64 K
// slots under a cap 53.5 us for 51.9, with positions on 16 K slots 28.7 for 26.7).
enum RowKind { kPlainRows, kAnyRows, kLargeCap };

template <int DH, int NB, bool F32, RowKind KIND>
__global__ void __launch_bounds__(kThreads, DH <= 128 && NB == 1 && !F32 ? 5 : 1)
k_kv4_attn(const __grid_constant__ Kv4AttnArgs a) {
  constexpr bool GEN = KIND != kPlainRows;
  constexpr int KS = DH / 16, MT = DH / 16, P = F32 ? 2 : 1;  // QK steps; O tiles of 16 elements
  constexpr int kRows = 8 * NB;
  pdl_prologue();
  extern __shared__ uint4 smem4[];
  using R = Ring<DH, true>;
  uint4* qs = smem4;                               // NB * P * KS / 2 * 32
  float* obuf = reinterpret_cast<float*>(smem4);   // kWarps * kRows * DH, after the loop
  float* cbuf = obuf + kWarps * kRows * DH;        // kRows * DH, the CTA's sums
  __shared__ float cml[2 * kRows];
  __shared__ RowPar par[kRows];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % a.nsplit;
  const int tile = blockIdx.x / a.nsplit % a.ntile;
  const int bh = blockIdx.x / a.nsplit / a.ntile;
  const int b = bh / a.Hkv, hkv = bh % a.Hkv, m0 = tile * kRows;
  const int rows = min(kRows, a.M - m0);
  const int len = kv4_len(a, b);

  stage_rows<DH, F32>(a, b, hkv, m0, kRows, qs, par);
  __syncthreads();
  // positions that some row sees, and that every row sees
  int n_lo = 0, n_hi = len, all_lo = 0, all_hi = len;
  const int32_t* kpos = GEN && a.kpos != nullptr ? a.kpos + (long)bh * a.Ncache : nullptr;
  if (kpos != nullptr) {
    if (a.span != nullptr) all_hi = -1;
  } else if (a.span != nullptr) {  // slots are positions: skip what no row sees
    const bool row = lane < rows;
    const int lo = row ? par[lane].lo : 0, hi = row ? par[lane].last + 1 : 0;
    const bool in = lo < hi;
    n_lo = max(0, __reduce_min_sync(0xffffffffu, in ? lo : INT32_MAX));
    n_hi = min(len, __reduce_max_sync(0xffffffffu, in ? hi : INT32_MIN));
    all_lo = __reduce_max_sync(0xffffffffu, row ? lo : INT32_MIN);
    all_hi = min(len, __reduce_min_sync(0xffffffffu, row ? hi : INT32_MAX));
  }
  // This CTA's share of the slots seen, whole 64-slot groups
  if (n_lo >= n_hi) {
    n_lo = n_hi = 0;
  } else if (a.nsplit > 1) {
    const int share = ceil_div(ceil_div(n_hi - n_lo, 64), a.nsplit) * 64;
    n_lo = (int)min((long)n_hi, n_lo + (long)split * share);
    n_hi = (int)min((long)n_hi, (long)n_lo + share);
  }

  if (a.nsplit > 1 && !a.cluster && n_lo >= n_hi) {  // an empty share
    if (tid < rows) {
      const size_t at = ((size_t)bh * a.M + m0 + tid) * a.nsplit + split;
      a.pml[2 * at] = -INFINITY;
      a.pml[2 * at + 1] = 0.f;
    }
    return;
  }

  const int last = a.Ncache - 1;
  uint8_t* ring = reinterpret_cast<uint8_t*>(qs + NB * P * (KS / 2) * 32) + warp * R::kBytes;
  const uint32_t ring32 = tc::smem_u32(ring);

  // O of rows 8 nb + 2 t + (c & 1), elements [g dh/8, (g+1) dh/8): element
  // 2 i + c / 2 in o[nb][i][c].  Scores are in log2 units: a raw product times
  // fa (of score / cap where scores are capped, for bf16 queries 2 log2(e) times
  // that); `base` is subtracted, the maximum so far less kPShift.
  float o[NB][MT][4], fa[NB][2], base[NB][2], lrow[NB][2];
  const float cap2 = a.cap * kLog2e;
  const bool capped = a.cap > 0.f;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[nb][i][c] = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float f = par[nb * 8 + 2 * t + u].f;
      fa[nb][u] = capped ? fminf(f * (F32 ? a.inv_cap : a.inv_cap * kTwoLog2e), FLT_MAX)
                         : f * (F32 ? 1.f : kLog2e);
      base[nb][u] = kNoMax;
      lrow[nb][u] = 0.f;
    }
  }
  RingFill<DH, true> fill(a, bh, n_lo + kStep * warp);
  if (n_lo + kStep * warp < n_hi) fill.next(ring32, kStep * kWarps);
  cp_commit();
  const int sg = slot_at(g);
  uint32_t at = 0;  // the stage to read
  for (int n2 = n_lo + kStep * warp; n2 < n_hi; n2 += kStep * kWarps) {
    cp_wait<0>();
    __syncwarp();  // the stage has arrived, and the other has been read by every lane
    if (n2 + kStep * kWarps < n_hi) fill.next(ring32 + (at ^ R::kStage), kStep * kWarps);
    cp_commit();
    const uint8_t* st = ring + at;
    at ^= R::kStage;
#pragma unroll
    for (int half = 0; half < kStep / 16; ++half) {
      const int n = n2 + 16 * half;
      if (n >= n_hi) break;
      RawK<DH> rk;
      read_k<DH>(st, half, g, t, rk);
      // S^T: slots sg and sg + 8 (c / 2), rows 2 t and 2 t + 1 (c & 1) of block nb
      float s[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nb][c] = 0.f;
#pragma unroll
      for (int w = 0; w < KS / 2; ++w) {
        uint32_t a0[4], a1[4];
        dequant_k<DH>(rk, w, a0, a1);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint4* q = qs + (nb * P * (KS / 2) + w) * 32 + lane;
          add_products<F32>(s[nb], a0, a1, q[0], q[(P - 1) * (KS / 2) * 32]);
        }
      }
      const bool masked = n < all_lo || n + 16 > all_hi;
      int pos[2] = {n + sg, n + sg + 8};
      if (GEN && kpos != nullptr) {
        pos[0] = __ldg(kpos + min(pos[0], last));
        pos[1] = __ldg(kpos + min(pos[1], last));
      }
      uint32_t ph[NB][2], pl[NB][F32 ? 2 : 1];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // the four scores less sub
        auto scores = [&](const float* sub, float* x) {
          if (F32) {
            float y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = s[nb][c] * fa[nb][c & 1];
            if (capped) tanh4(y);
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = fmaf(y[c], capped ? cap2 : kLog2e, -sub[c & 1]);
          } else if (KIND == kLargeCap) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              x[c] = fmaf(tanh_any(s[nb][c] * fa[nb][c & 1] * (1.f / kTwoLog2e)), cap2,
                          -sub[c & 1]);
          } else if (capped) {  // tanh_abs, times the cap in its last step
#pragma unroll
            for (int c = 0; c < 4; ++c)
              x[c] = fmaf(-2.f * cap2, rcp_approx(exp2_approx(s[nb][c] * fa[nb][c & 1]) + 1.f),
                          cap2 - sub[c & 1]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = fmaf(s[nb][c], fa[nb][c & 1], -sub[c & 1]);
          }
          if (GEN && a.slope != nullptr) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const RowPar& rp = par[nb * 8 + 2 * t + (c & 1)];
              x[c] = fmaf(-rp.slope * kLog2e, fabsf((float)(rp.qpos - pos[c >> 1])), x[c]);
            }
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const RowPar& rp = par[nb * 8 + 2 * t + (c & 1)];
              if (n + sg + 8 * (c >> 1) >= len || pos[c >> 1] < rp.lo || pos[c >> 1] > rp.last)
                x[c] = -INFINITY;
            }
          }
        };
        float x[4];
        scores(base[nb], x);
        // The running maximum follows only when some row has outgrown it by
        // 2^kGrow; until then P carries a factor up to that.  Scores from 2^24 on
        // lie further apart than these shifts: rounded so that P stays in f16.
        if (__any_sync(0xffffffffu,
                       fmaxf(fmaxf(x[0], x[2]), fmaxf(x[1], x[3])) > kPShift + kGrow)) {
          const float zero[2] = {0.f, 0.f};
          scores(zero, x);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float mx = fmaxf(x[u], x[2 + u]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = __fsub_ru(fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16)), kPShift);
            if (mx > __fadd_rd(base[nb][u], kGrow)) {
              const float corr = exp2_approx(base[nb][u] - mx);
              base[nb][u] = mx;
              lrow[nb][u] *= corr;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[nb][i][u] *= corr;
                o[nb][i][2 + u] *= corr;
              }
            }
            x[u] -= base[nb][u];
            x[2 + u] -= base[nb][u];
          }
        }
        float p[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          p[c] = exp2_approx(x[c]);
          lrow[nb][c & 1] += p[c];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // slots 8 j .. 8 j + 7: (slot, rows) -> (row, slots)
          const __half2 h = __floats2half2_rn(p[2 * j], p[2 * j + 1]);
          ph[nb][j] = transpose8(h2_bits(h));
          if constexpr (F32) {
            const float2 back = __half22float2(h);
            pl[nb][j] =
                transpose8(h2_bits(__floats2half2_rn(p[2 * j] - back.x, p[2 * j + 1] - back.y)));
          }
        }
      }
      // O^T += V^T P^T
      RawV<DH> rv;
      read_v<DH>(st + R::kV, half, g, t, rv);
#pragma unroll
      for (int w = 0; w < DH / 64; ++w) {
        uint32_t v[2][2][4];  // [even, odd element][slots t and t + 4, t + 8 and t + 12][byte]
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t even, odd;
          pair_codes(rv.c[2 * j][w], rv.c[2 * j + 1][w], &even, &odd);
          const int sh = DH == 256 ? 8 * (w / 2) : 0;
          const __half2 sc =
              e4m3x2_f16(((rv.s[2 * j] >> sh) & 0xffu) | ((rv.s[2 * j + 1] >> sh) & 0xffu) << 8);
          e2m1x8_f16(even, v[0][j]);
          e2m1x8_f16(odd, v[1][j]);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[e][j][q] = h2_bits(__hmul2(h2_of(v[e][j][q]), sc));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t av[4] = {v[0][0][q], v[1][0][q], v[0][1][q], v[1][1][q]};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float* d = o[nb][4 * w + q];
            if constexpr (F32) {
              // added by a rounding instruction, as the scores
              float e[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(e, av, ph[nb][0], ph[nb][1]);
              mma_f16(e, av, pl[nb][0], pl[nb][1]);
#pragma unroll
              for (int c = 0; c < 4; ++c) d[c] += e[c];
            } else {
              mma_f16(d, av, ph[nb][0], ph[nb][1]);
            }
          }
        }
      }
    }
  }

  // the four warps' shares of each row joined
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float l = lrow[nb][u];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (g == 0) {
        s_m[warp][nb * 8 + 2 * t + u] = base[nb][u] == kNoMax ? -INFINITY : base[nb][u] + kPShift;
        s_l[warp][nb * 8 + 2 * t + u] = l;
      }
    }
  cp_wait<0>();
  __syncthreads();  // Q and the rings are no longer read
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = nb * 8 + 2 * t + u;
      if (r < rows) {
        float* dst = obuf + ((size_t)warp * kRows + r) * DH + g * (DH / 8);
#pragma unroll
        for (int i = 0; i < MT; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(
              o[nb][i][u], o[nb][i][2 + u], o[nb][i + 1][u], o[nb][i + 1][2 + u]);
      }
    }
  __syncthreads();
  for (int e = tid; e < rows * (DH / 4); e += kThreads) {
    const int r = e / (DH / 4), d = e % (DH / 4) * 4, m = m0 + r;
    float mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      // a warp that saw nothing (or NaN only) keeps factor 1: its sums are 0 (NaN)
      const float c = s_m[w][r] == -INFINITY ? 1.f : exp2_approx(s_m[w][r] - mx);
      const float4 v = *reinterpret_cast<const float4*>(obuf + ((size_t)w * kRows + r) * DH + d);
      l += c * s_l[w][r];
      acc.x += c * v.x; acc.y += c * v.y; acc.z += c * v.z; acc.w += c * v.w;
    }
    if (a.cluster) {
      *reinterpret_cast<float4*>(cbuf + r * DH + d) = acc;
      if (d == 0) {
        cml[2 * r] = mx;
        cml[2 * r + 1] = l;
      }
    } else if (a.nsplit > 1) {
      const size_t at = ((size_t)bh * a.M + m) * a.nsplit + split;
      if (l != 0.f) *reinterpret_cast<float4*>(a.po + at * DH + d) = acc;
      if (d == 0) {
        a.pml[2 * at] = mx;
        a.pml[2 * at + 1] = l;
      }
    } else {
      kv4_finish<F32>(a, b, hkv, m, DH, d, acc, mx, l);
    }
  }
  if (a.cluster) {
    // The shares of these rows are the CTAs of a thread-block cluster: each
    // joins its part of the elements from all of them, in order.
    tc::cluster_sync_all();
    const uint32_t cb = tc::smem_u32(cbuf), cm = tc::smem_u32(cml);
    for (int e = tid + split * kThreads; e < rows * (DH / 4); e += kThreads * a.nsplit) {
      const int r = e / (DH / 4), d = e % (DH / 4) * 4;
      float ms[kMaxCluster], ls[kMaxCluster], mx = -INFINITY, l = 0.f;
      float4 v[kMaxCluster];
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        if (q >= a.nsplit) break;
        const uint32_t mq = tc::cluster_map(cm, q) + r * 8;
        ms[q] = tc::ld_dsmem_f32(mq);
        ls[q] = tc::ld_dsmem_f32(mq + 4);
        v[q] = tc::ld_dsmem_v4(tc::cluster_map(cb, q) + (r * DH + d) * 4);
      }
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q)
        if (q < a.nsplit) mx = fmaxf(mx, ms[q]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        if (q >= a.nsplit) break;
        const float c = ms[q] == -INFINITY ? 1.f : exp2_approx(ms[q] - mx);
        l += c * ls[q];
        acc.x += c * v[q].x; acc.y += c * v[q].y; acc.z += c * v[q].z; acc.w += c * v[q].w;
      }
      kv4_finish<F32>(a, b, hkv, m0 + r, DH, d, acc, mx, l);
    }
    tc::cluster_sync_all();  // no CTA leaves while another still reads its sums
  }
}

// One CTA a row: dh / 4 threads take four elements each of every (4 NT / dh)-th
// share, and the groups are joined in order.
template <int DH, bool F32, int NT>
__global__ void __launch_bounds__(NT)
k_kv4_combine(const __grid_constant__ Kv4AttnArgs a) {
  constexpr int LN = DH / 4, NG = NT / LN;  // threads a share, shares at a time
  pdl_prologue();
  __shared__ float s_part[NG][DH], s_l[NG], s_w[NT / 32];
  const int idx = blockIdx.x, bh = idx / a.M, m = idx - bh * a.M;
  const int tid = threadIdx.x, grp = tid / LN, d = (tid % LN) * 4;
  const float* ml = a.pml + (size_t)idx * a.nsplit * 2;
  const float* po = a.po + (size_t)idx * a.nsplit * DH + d;
  float mx = -INFINITY;
  for (int s = tid; s < a.nsplit; s += NT) mx = fmaxf(mx, ml[2 * s]);
  mx = warp_max(mx);
  if ((tid & 31) == 0) s_w[tid >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) mx = fmaxf(mx, s_w[w]);
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = grp; s < a.nsplit; s += NG) {
    const float ms = ml[2 * s], ls = ml[2 * s + 1];
    const float4 v = *reinterpret_cast<const float4*>(po + (size_t)s * DH);
    const float c = ms == -INFINITY ? 1.f : exp2_approx(ms - mx);
    if (ls != 0.f) {  // else it saw nothing, and its sums may not have been written
      l += c * ls;
      acc.x += c * v.x; acc.y += c * v.y; acc.z += c * v.z; acc.w += c * v.w;
    }
  }
  *reinterpret_cast<float4*>(&s_part[grp][d]) = acc;
  if (d == 0) s_l[grp] = l;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int q = 1; q < NG; ++q) {
    const float4 v = *reinterpret_cast<const float4*>(&s_part[q][d]);
    acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    l = q == 1 ? s_l[0] + s_l[1] : l + s_l[q];
  }
  kv4_finish<F32>(a, bh / a.Hkv, bh % a.Hkv, m, DH, d, acc, mx, l);
}

// K only: a warp owns 16 slots at a time, whose K fragments stay in registers
// while all rows of the head pass by (kWRows at a time through shared memory);
// every slot's sum is one warp's, in row order, so the result does not depend
// on timing.
// Rows from which k_kv4_weight_tc takes over.  It pays more a slot and less a row:
// 4 x 32 heads, 4096 slots: 64 rows 71 us there and 42 here, 96 rows 67 and 121;
// 2 x 8 heads, 16 K slots: 36 and 22, 35 and 65.
constexpr int kTcWeight = 64;
constexpr int kWRows = 64;
constexpr int kGroup = kStep * kWarps;  // slots that a CTA takes at a time

// The slots that some row, and that every row, of those in shared memory sees.
struct SeenRange {
  int any_lo, any_hi, all_lo, all_hi;
};
__device__ __forceinline__ SeenRange seen_range(const RowPar* par, int rows, int len) {
  int lo = INT32_MAX, hi = INT32_MIN, lo_all = INT32_MIN, hi_all = INT32_MAX;
  for (int r = threadIdx.x & 31; r < rows; r += 32) {
    const int x = par[r].lo, y = par[r].last + 1;
    if (x < y) {
      lo = min(lo, x);
      hi = max(hi, y);
    }
    lo_all = max(lo_all, x);
    hi_all = min(hi_all, y);
  }
  SeenRange s;
  s.any_lo = __reduce_min_sync(0xffffffffu, lo);
  s.any_hi = min(len, __reduce_max_sync(0xffffffffu, hi));
  s.all_lo = __reduce_max_sync(0xffffffffu, lo_all);
  s.all_hi = min(len, __reduce_min_sync(0xffffffffu, hi_all));
  return s;
}

// acc[j] += sum over nbs blocks of 8 rows of exp(score - lse), slots n + sg + 8 j.
template <int DH, bool F32, bool GEN>
__device__ __forceinline__ void weigh(const Kv4AttnArgs& a, const uint32_t (*kf)[4],
                                      const uint4* qp, const RowPar* rp, int nbs, int n_sg,
                                      int len, const int* pos, bool masked, float* acc) {
  constexpr int KS = DH / 16, P = F32 ? 2 : 1;
#pragma unroll 1
  for (; nbs > 0; --nbs, qp += P * (KS / 2) * 32, rp += 8) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < KS / 2; ++w)
      add_products<F32>(s, kf[2 * w], kf[2 * w + 1], qp[w * 32], qp[((P - 1) * (KS / 2) + w) * 32]);
    // score - lse of slots sg, sg + 8 (c / 2), rows 2 t, 2 t + 1 (c & 1)
    float x[4];
    const float f0 = rp[0].f, l0 = -rp[0].lse, f1 = rp[1].f, l1 = -rp[1].lse;
    if (GEN && a.cap > 0.f) {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = s[c] * (c & 1 ? f1 : f0) * a.inv_cap;
      tanh4(x);
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = fmaf(x[c], a.cap, c & 1 ? l1 : l0);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = fmaf(s[c], c & 1 ? f1 : f0, c & 1 ? l1 : l0);
    }
    if (GEN && a.slope != nullptr) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[c] = fmaf(-rp[c & 1].slope, fabsf((float)(rp[c & 1].qpos - pos[c >> 1])), x[c]);
    }
    if (masked) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n_sg + 8 * (c >> 1) >= len || pos[c >> 1] < rp[c & 1].lo ||
            pos[c >> 1] > rp[c & 1].last)
          x[c] = -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c >> 1] += exp2_approx(x[c] * kLog2e);
  }
}

// GEN: capped scores, a distance bias or explicit positions.  ONE: all rows fit
// shared memory and are staged once.
template <int DH, bool F32, bool GEN, bool ONE>
__global__ void __launch_bounds__(kThreads)
k_kv4_weight(const __grid_constant__ Kv4AttnArgs a, int steps) {
  constexpr int KS = DH / 16, P = F32 ? 2 : 1;
  pdl_prologue();
  extern __shared__ uint4 smem4[];
  using R = Ring<DH, false>;
  uint4* qs = smem4;  // (kWRows / 8) * P * KS / 2 * 32
  __shared__ RowPar par[kWRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int bh = blockIdx.y, b = bh / a.Hkv, hkv = bh % a.Hkv;
  const int len = kv4_len(a, b), last = a.Ncache - 1;
  const int32_t* kpos = GEN && a.kpos != nullptr ? a.kpos + (long)bh * a.Ncache : nullptr;
  const int chunks = ONE ? 1 : ceil_div(a.M, kWRows);
  const int n0 = (blockIdx.x * steps) * kGroup + kStep * warp;
  // the warp's steps that hold slots of the sequence; all warps' for the barriers
  const int live = max(0, min(steps, ceil_div(len - n0, kGroup)));
  const int sg = slot_at(g);
  // lanes t < 2 write slot sg + 8 t
  const float* w_in = a.w_in != nullptr ? a.w_in + (long)bh * a.Ncache + n0 + sg + 8 * t : nullptr;
  float* w_out = a.w_out + (long)bh * a.Ncache + n0 + sg + 8 * t;
  int room = t < 2 ? a.Ncache - (n0 + sg + 8 * t) : 0;  // > 0: the slot exists
  uint8_t* ring =
      reinterpret_cast<uint8_t*>(qs + (kWRows / 8) * P * (KS / 2) * 32) + warp * R::kBytes;
  const uint32_t ring32 = tc::smem_u32(ring);
  RingFill<DH, false> fill(a, bh, n0);
  if (live > 0) fill.next(ring32, kGroup);
  cp_commit();
  uint32_t at = 0;  // the stage to read
  const bool spans = a.span != nullptr && kpos == nullptr;
  SeenRange seen{0, len, 0, kpos != nullptr && a.span != nullptr ? -1 : len};
  int nbs = 0;
  if constexpr (ONE) {
    stage_rows<DH, F32>(a, b, hkv, 0, (a.M + 7) & ~7, qs, par);
    __syncthreads();
    if (spans) seen = seen_range(par, a.M, len);
    nbs = ceil_div(a.M, 8);
  }
  const int all = ONE ? live : steps;
  int n2 = n0;
  for (int st = 0; st < all; ++st, n2 += kGroup) {
    float old[kStep / 16];  // asked for early
#pragma unroll
    for (int h = 0; h < kStep / 16; ++h)
      old[h] = w_in != nullptr && room > 16 * h ? w_in[16 * h] : 0.f;
    cp_wait<0>();
    __syncwarp();
    if (st + 1 < live) fill.next(ring32 + (at ^ R::kStage), kGroup);
    cp_commit();
#pragma unroll
    for (int h = 0; h < kStep / 16; ++h) {
      const int n = n2 + 16 * h;
      uint32_t kf[KS][4];
      int pos[2] = {n + sg, n + sg + 8};
      float acc[2] = {0.f, 0.f};  // slots sg and sg + 8
      const bool here = n < len;  // warp-uniform
      if (here) {
        RawK<DH> rk;
        read_k<DH>(ring + at, h, g, t, rk);
#pragma unroll
        for (int w = 0; w < KS / 2; ++w) dequant_k<DH>(rk, w, kf[2 * w], kf[2 * w + 1]);
        if (GEN && kpos != nullptr) {
          pos[0] = __ldg(kpos + min(pos[0], last));
          pos[1] = __ldg(kpos + min(pos[1], last));
        }
      }
      if constexpr (ONE) {
        if (here && n < seen.any_hi && n + 16 > seen.any_lo)
          weigh<DH, F32, GEN>(a, kf, qs + lane, par + 2 * t, nbs, n + sg, len, pos,
                              n < seen.all_lo || n + 16 > seen.all_hi, acc);
      } else {
        for (int ch = 0; ch < chunks; ++ch) {
          const int m0 = ch * kWRows, rows = min(kWRows, a.M - m0);
          __syncthreads();
          stage_rows<DH, F32>(a, b, hkv, m0, (rows + 7) & ~7, qs, par);
          __syncthreads();
          if (spans) seen = seen_range(par, rows, len);
          if (here && n < seen.any_hi && n + 16 > seen.any_lo)
            weigh<DH, F32, GEN>(a, kf, qs + lane, par + 2 * t, ceil_div(rows, 8), n + sg, len, pos,
                                n < seen.all_lo || n + 16 > seen.all_hi, acc);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 1);
        acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 2);
      }
      if (room > 16 * h) w_out[16 * h] = old[h] + (t == 0 ? acc[0] : acc[1]);
    }
    at ^= R::kStage;
    if (w_in != nullptr) w_in += kGroup;
    w_out += kGroup;
    room -= kGroup;
  }
  for (int st = all; st < steps; ++st) {  // past the sequence
#pragma unroll
    for (int h = 0; h < kStep / 16; ++h)
      if (room > 16 * h) w_out[16 * h] = w_in != nullptr ? w_in[16 * h] : 0.f;
    if (w_in != nullptr) w_in += kGroup;
    w_out += kGroup;
    room -= kGroup;
  }
  cp_wait<0>();  // no copy is under way when the CTA leaves
}

template <int DH, bool F32>
cudaError_t launch_combine(const Kv4AttnArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(a.B * a.Hkv * a.M));
  // many threads a row where there are few rows with many shares: a token on 30 K
  // slots 13.4 us for 16.6, 64 K slots x 1 head 12.7 for 17.6; 800 rows 25.6 for 23.7
  return a.nsplit > 16 && grid.x <= 4 * kSmTarget
             ? launch_pdl(k_kv4_combine<DH, F32, 512>, grid, dim3(512), 0, s, a)
             : launch_pdl(k_kv4_combine<DH, F32, 128>, grid, dim3(128), 0, s, a);
}

template <int DH, int NB, bool F32, RowKind KIND>
cudaError_t launch_attn(const Kv4AttnArgs& a, cudaStream_t s) {
  constexpr size_t q_bytes =
      (size_t)NB * (F32 ? 2 : 1) * (DH / 32) * 32 * 16 + kWarps * Ring<DH, true>::kBytes;
  constexpr size_t o_bytes = (size_t)(kWarps + 1) * 8 * NB * DH * 4;
  constexpr size_t smem = q_bytes > o_bytes ? q_bytes : o_bytes;
  auto kern = k_kv4_attn<DH, NB, F32, KIND>;
  static bool attr_set = false;
  if (!attr_set && smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  const unsigned grid = (unsigned)((long)a.B * a.Hkv * a.nsplit * a.ntile);
  if (a.cluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.nsplit;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_ex(cfg, kern, a);
  }
  cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kThreads), smem, s, a);
  if (e != cudaSuccess || a.nsplit == 1) return e;
  return launch_combine<DH, F32>(a, s);
}

template <int DH, bool F32, bool GEN, bool ONE>
cudaError_t launch_weight(const Kv4AttnArgs& a, cudaStream_t s) {
  constexpr size_t smem =
      (size_t)(kWRows / 8) * (F32 ? 2 : 1) * (DH / 32) * 32 * 16 + kWarps * Ring<DH, false>::kBytes;
  auto kern = k_kv4_weight<DH, F32, GEN, ONE>;
  static bool attr_set = false;
  if (!attr_set && smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  // rows that fit shared memory are staged once for all the slot groups of
  // a CTA, as many as leave five CTAs an SM, which is what its registers hold
  // (against eight: a token on 64 K slots 7.6 us for 9.3, on 4 sequences of 12 K
  // 6.0 for 7.3, on 8 of 32 K 18.6 for 19.1, 32-token blocks on 4 K 25.7 for 24.3)
  const int groups = ceil_div(a.Ncache, kGroup);
  int steps = 1;
  if (ONE) {
    steps = ceil_div((long)groups * a.B * a.Hkv, 5 * kSmTarget);
    if (steps > 64) steps = 64;
  }
  return launch_pdl(kern, dim3((unsigned)ceil_div(groups, steps), a.B * a.Hkv), dim3(kThreads),
                    smem, s, a, steps);
}

// The kernel, rows of a tile, tiles and shares of the slots for these sizes.
struct AttnPlan {
  bool tc;  // k_kv4_attn_tc: 256-row tiles; else k_kv4_attn: 8 nb
  int nb, ntile, nsplit;
};
AttnPlan attn_plan(int dtype, int B, int N, int Hq, int Hkv, int dh, int T) {
  AttnPlan p;
  const int M = T * (Hq / Hkv);
  // From 33 rows on the tcgen05 kernel reads the slots fewer times.  4 x 32 heads,
  // 768 slots: 32 rows 17.2 us there and 15.6 here, 48 rows 17.2 and 28; 4 x 8
  // heads, 4096 slots: 32 rows 23.5 and 19.5, 64 rows 24 and 31.
  p.tc = dtype == PS_BF16 && dh <= 128 && M > 32;
  if (p.tc) {
    p.nb = 0;
    p.ntile = ceil_div(M, 256);
    // rounds of CTAs (one an SM) times the steps of each, set-up and join
    // counted as four steps
    const long base = (long)B * Hkv * p.ntile;
    const int steps = ceil_div(N, 128);
    p.nsplit = 1;
    long best = ceil_div(base, kSmTarget) * (long)(steps + 4);
    for (int ns = 2; ns <= 64 && ns <= steps; ++ns) {
      const long cost = ceil_div(base * ns, kSmTarget) * (long)(ceil_div(steps, ns) + 4) + 4;
      if (cost < best) {
        best = cost;
        p.nsplit = ns;
      }
    }
    return p;
  }
  // 16-row tiles from 9 rows on: 16 rows, 4 x 8 heads, 4096 slots 15.6 us against
  // 16.2 as two of 8, 64 fp32 rows 42 against 57; 8 rows in a 16-row tile 14.5
  // against 13.4.  (32-row tiles for fp32: 70, too few warps an SM.)
  p.nb = M <= 8 ? 1 : 2;
  p.ntile = ceil_div(M, 8 * p.nb);
  const long base = (long)B * Hkv * p.ntile;
  const int most = ceil_div(N, 128);  // at least 128 slots a share
  // CTAs that run side by side, 4 a SM of 8 rows and 2 of more: no second round
  // of them that leaves SMs idle.  Against 7 a SM in rounds: 8 sequences of 64 K
  // slots 59 us for 71 (lengths of 1/2 to 1: 51 for 50), of 6000 slots 14.5 for
  // 20; 16 rows and 32 K slots 53 for 73; with 5 and 3 a SM 62, 16 and 68.
  long want = (p.nb == 1 ? 4 : 2) * kSmTarget / base;
  if (want > most) want = most;
  if (want > 256) want = 256;
  p.nsplit = (int)(want < 1 ? 1 : want);
  return p;
}

// Few shares are joined inside a thread-block cluster, without a second kernel.
bool in_cluster(const AttnPlan& p) { return !p.tc && p.nsplit > 1 && p.nsplit <= kMaxCluster; }

}  // namespace

size_t kv4_attn_ws(int B, int N, int Hq, int Hkv, int dh, int T) {
  // either type's: the size does not name it
  size_t most = 0;
  for (int dtype : {PS_F32, PS_BF16}) {
    const AttnPlan p = attn_plan(dtype, B, N, Hq, Hkv, dh, T);
    if (p.nsplit == 1 || in_cluster(p)) continue;
    Carver c(nullptr);
    const size_t rows = (size_t)B * T * Hq * p.nsplit;
    c.take<float>(rows * dh);
    c.take<float>(rows * 2);
    if (c.bytes() > most) most = c.bytes();
  }
  return most;
}

size_t kv4_weight_ws(int, int, int, int, int, int) { return 0; }

cudaError_t kv4_attn_run(Kv4AttnArgs a, cudaStream_t s) {
  const AttnPlan p = attn_plan(a.dtype, a.B, a.Ncache, a.Hq, a.Hkv, a.dh, a.T);
  a.ntile = p.ntile;
  a.nsplit = p.nsplit;
  a.cluster = in_cluster(p);
  if (a.nsplit > 1 && !a.cluster) {
    Carver c(a.ws);
    const size_t rows = (size_t)a.B * a.T * a.Hq * a.nsplit;
    a.po = c.take<float>(rows * a.dh);
    a.pml = c.take<float>(rows * 2);
  }
  const bool f32 = a.dtype == PS_F32;
  if (p.tc) {
    cudaError_t e = kv4_attn_tc_launch(a, s);
    if (e != cudaSuccess || a.nsplit == 1) return e;
    return a.dh == 64 ? launch_combine<64, false>(a, s) : launch_combine<128, false>(a, s);
  }
  const bool gen = a.slope != nullptr || a.kpos != nullptr;
#define PS_KV4_CASE(DH, NB)                                           \
  if (a.dh == DH && p.nb == NB) {                                     \
    if (f32) return launch_attn<DH, NB, true, kAnyRows>(a, s);        \
    if (a.cap > kCapAbs) return launch_attn<DH, NB, false, kLargeCap>(a, s); \
    return gen ? launch_attn<DH, NB, false, kAnyRows>(a, s)           \
               : launch_attn<DH, NB, false, kPlainRows>(a, s);        \
  }
  PS_KV4_CASE(64, 1)
  PS_KV4_CASE(64, 2)
  PS_KV4_CASE(128, 1)
  PS_KV4_CASE(128, 2)
  PS_KV4_CASE(256, 1)
  PS_KV4_CASE(256, 2)
#undef PS_KV4_CASE
  return cudaErrorInvalidValue;
}

cudaError_t kv4_weight_run(const Kv4AttnArgs& a, cudaStream_t s) {
  if (a.dtype == PS_BF16 && a.dh <= 128 && a.M > kTcWeight) return kv4_weight_tc_launch(a, s);
  const bool gen = a.cap > 0.f || a.slope != nullptr || a.kpos != nullptr;
  const bool one = a.M <= kWRows;
#define PS_KV4_CASE(DH)                                                       \
  if (a.dh == DH) {                                                           \
    if (a.dtype == PS_F32)                                                    \
      return one ? launch_weight<DH, true, true, true>(a, s)                  \
                 : launch_weight<DH, true, true, false>(a, s);                \
    if (gen)                                                                  \
      return one ? launch_weight<DH, false, true, true>(a, s)                 \
                 : launch_weight<DH, false, true, false>(a, s);               \
    return one ? launch_weight<DH, false, false, true>(a, s)                  \
               : launch_weight<DH, false, false, false>(a, s);                \
  }
  PS_KV4_CASE(64)
  PS_KV4_CASE(128)
  PS_KV4_CASE(256)
#undef PS_KV4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace ps
