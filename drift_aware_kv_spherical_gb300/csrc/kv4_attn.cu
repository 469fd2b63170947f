// Attention over a 4-bit KV cache, and the weight it puts on each slot.
//
//   k_kv4_attn     online-softmax attention of a 16- or 32-row tile of one KV
//                  head's queries over a share of its slots
//   k_kv4_combine  the shares of a row joined
//   k_kv4_weight   column sums of exp(s - lse), K only
//
// The rows of a KV head are its T tokens times the G = Hq / Hkv query heads it
// serves (row t G + j), so a head's K and V are read once for all of them.
//
// A warp works alone on 16 slots at a time, straight from global memory into
// m16n8k16 operand fragments (f16, fp32 accumulators):
//   S = Q K^T   the 16 contraction indices of a step may be any 16 elements as
//     long as Q and K agree: lane (g, t) = (lane / 4, lane % 4) takes elements
//     [t dh/4, (t+1) dh/4) of the slot of its column g, one contiguous load,
//     and step ks uses elements 4 ks .. 4 ks + 3 of it.  Q is laid out in that
//     order in shared memory, one 16-byte load a step.
//   O = P V     column c of S stands for slot 4 (c/2) + c%2 (first n8 tile) or
//     that + 2 (second), so lane t's four scores belong to slots 4t .. 4t+3,
//     whose V rows it loads itself: elements [g dh/8, (g+1) dh/8), one n8 tile
//     of O a code.  The slot pairs are joined by byte permutes.
// Q is scaled by a power of two of its row's own (2^14 <= max |q| < 2^15), so
// bf16 queries are exact in f16 down to 2^-25 of the row's largest; fp32
// queries and P take two f16 terms (hi + lo).  P carries a factor 2^12, which
// keeps weights down to 2^-26 of the row's largest out of f16's subnormals.
#include "kv4.cuh"

namespace ps {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Rows [m0, m0 + rows) of (b, hkv) into shared memory as A fragments
// [mt][part][ks][lane] (uint4), with their constants; rows past M are zero
// and see nothing.  One warp a row.
template <int DH, bool F32>
__device__ __forceinline__ void stage_rows(const Kv4AttnArgs& a, int b, int hkv, int m0, int rows,
                                           uint4* qs, RowPar* par, int nwarps) {
  constexpr int KS = DH / 16, E = DH / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = warp; r < rows; r += nwarps) {
    const int m = m0 + r;
    float x[E];
    RowPar p{0.f, 0.f, 0, 0, 0, -INFINITY};
    if (m < a.M) {
      const int t = row_token(a, m), h = hkv * a.G + (m - t * a.G);
      const long tok = (long)b * a.T + t;
      const long at = tok * a.q_ld + (long)h * DH + lane * E;
      if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = static_cast<const float*>(a.Q)[at + e];
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          x[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.Q)[at + e]);
      }
      p.slope = a.slope != nullptr ? a.slope[h] : 0.f;
      p.lo = a.span != nullptr ? a.span[2 * tok] : 0;
      p.hi = a.span != nullptr ? a.span[2 * tok + 1] : INT32_MAX;
      p.qpos = a.qpos != nullptr ? a.qpos[tok] : 0;
      p.lse = a.lse_in != nullptr ? a.lse_in[tok * a.Hq + h] : -INFINITY;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = 0.f;
    }
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(x[e]));
    mx = warp_max(mx);
    float up;
    row_scale(mx, a.scale, &up, &p.f);
    if (lane == 0) par[r] = p;
    __half* hq = reinterpret_cast<__half*>(qs);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane * E + e, t = d / (DH / 4), rem = d % (DH / 4);
      const int ks = rem / 4, j = rem % 4;
      const int reg = (j / 2) * 2 + (r % 16) / 8, fl = (r % 8) * 4 + t;
      const float v = x[e] * up;
      const __half hi = __float2half_rn(v);
      constexpr int P = F32 ? 2 : 1;
      const size_t base = ((((size_t)(r / 16) * P) * KS + ks) * 32 + fl) * 8 + reg * 2 + (j & 1);
      hq[base] = hi;
      if constexpr (F32) hq[base + (size_t)KS * 32 * 8] = __float2half_rn(v - __half2float(hi));
    }
  }
}

// K of the lane's two slots of a 16-slot step (raw codes and scale bytes).
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
__device__ __forceinline__ void load_k(const uint8_t* kc, const uint8_t* ks, int n, int last,
                                       int g, int t, RawK<DH>& o) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long slot = min(n + 4 * (g >> 1) + (g & 1) + 2 * j, last);
    const uint8_t* p = kc + slot * (DH / 2) + t * (DH / 8);
    const uint8_t* q = ks + slot * (DH / 16) + t * (DH / 64);
    if constexpr (DH == 64) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      o.c[j][0] = v.x; o.c[j][1] = v.y;
      o.s[j] = __ldg(q);
    } else {
#pragma unroll
      for (int i = 0; i < DH / 128; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        o.c[j][4 * i] = v.x; o.c[j][4 * i + 1] = v.y;
        o.c[j][4 * i + 2] = v.z; o.c[j][4 * i + 3] = v.w;
      }
      if constexpr (DH == 128) o.s[j] = __ldg(reinterpret_cast<const uint16_t*>(q));
      else o.s[j] = __ldg(reinterpret_cast<const uint32_t*>(q));
    }
  }
}

template <int DH>
__device__ __forceinline__ void load_v(const uint8_t* vc, const uint8_t* vs, int n, int last,
                                       int g, int t, RawV<DH>& o) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long slot = min(n + 4 * t + j, last);
    const uint8_t* p = vc + slot * (DH / 2) + g * (DH / 16);
    const uint8_t* q = vs + slot * (DH / 16);
    if constexpr (DH == 64) {
      o.c[j][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      o.s[j] = __ldg(q + (g >> 1));
    } else if constexpr (DH == 128) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      o.c[j][0] = v.x; o.c[j][1] = v.y;
      o.s[j] = __ldg(q + g);
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      o.c[j][0] = v.x; o.c[j][1] = v.y; o.c[j][2] = v.z; o.c[j][3] = v.w;
      o.s[j] = __ldg(reinterpret_cast<const uint16_t*>(q) + g);
    }
  }
}

// B fragments of K: kf[j][ks][0..1] for the lane's slot of n8 tile j.
template <int DH>
__device__ __forceinline__ void dequant_k(const RawK<DH>& r, uint32_t (*kf)[DH / 16][2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int w = 0; w < DH / 32; ++w) {
      uint32_t h[4];
      e2m1x8_f16(r.c[j][w], h);
      // word w holds elements 8 w .. 8 w + 7 of the lane's dh / 4: two a scale
      const __half2 s = e4m3_pair((r.s[j] >> (8 * (w / 2))) & 0xffu);
      kf[j][2 * w][0] = h2_bits(__hmul2(h2_of(h[0]), s));
      kf[j][2 * w][1] = h2_bits(__hmul2(h2_of(h[1]), s));
      kf[j][2 * w + 1][0] = h2_bits(__hmul2(h2_of(h[2]), s));
      kf[j][2 * w + 1][1] = h2_bits(__hmul2(h2_of(h[3]), s));
    }
}

template <int DH, int MT, bool F32>
__global__ void __launch_bounds__(kThreads)
k_kv4_attn(const __grid_constant__ Kv4AttnArgs a) {
  constexpr int KS = DH / 16, NT = DH / 8, P = F32 ? 2 : 1;
  constexpr int kRows = 16 * MT;
  pdl_prologue();
  extern __shared__ uint4 smem4[];
  uint4* qs = smem4;                                             // MT * P * KS * 32
  float* obuf = reinterpret_cast<float*>(smem4);                 // kWarps * kRows * DH, after the loop
  __shared__ RowPar par[kRows];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ int s_range[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int tile = blockIdx.x % a.ntile;
  const int split = blockIdx.x / a.ntile % a.nsplit;
  const int bh = blockIdx.x / a.ntile / a.nsplit;
  const int b = bh / a.Hkv, hkv = bh % a.Hkv, m0 = tile * kRows;
  const int rows = min(kRows, a.M - m0);
  const int len = kv4_len(a, b);

  stage_rows<DH, F32>(a, b, hkv, m0, kRows, qs, par, kWarps);
  __syncthreads();
  // positions that some row sees, and that every row sees
  if (warp == 0) {
    int lo = INT32_MAX, hi = INT32_MIN, lo_all = INT32_MIN, hi_all = INT32_MAX;
    for (int r = lane; r < rows; r += 32) {
      if (par[r].lo < par[r].hi) {
        lo = min(lo, par[r].lo);
        hi = max(hi, par[r].hi);
      }
      lo_all = max(lo_all, par[r].lo);
      hi_all = min(hi_all, par[r].hi);
    }
    for (int o = 16; o > 0; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo_all = max(lo_all, __shfl_xor_sync(0xffffffffu, lo_all, o));
      hi_all = min(hi_all, __shfl_xor_sync(0xffffffffu, hi_all, o));
    }
    if (lane == 0) {
      s_range[0] = lo; s_range[1] = hi; s_range[2] = lo_all; s_range[3] = hi_all;
    }
  }
  __syncthreads();
  const int32_t* kpos = a.kpos != nullptr ? a.kpos + (long)bh * a.Ncache : nullptr;
  int n_lo = 0, n_hi = len, all_lo = 0, all_hi = len;
  if (kpos == nullptr) {  // slots are positions: skip what no row sees
    n_lo = max(0, s_range[0]) & ~15;
    n_hi = min(len, s_range[1]);
    all_lo = s_range[2];
    all_hi = min(len, s_range[3]);
  } else if (a.span != nullptr) {
    all_hi = -1;
  }
  // this CTA's share: whole 64-slot groups
  if (n_lo >= n_hi) {
    n_lo = n_hi = 0;
  } else {
    const int share = ceil_div(ceil_div(n_hi - n_lo, 64), a.nsplit) * 64;
    n_lo = min(n_hi, n_lo + split * share);
    n_hi = min(n_hi, n_lo + share);
  }

  const uint8_t* kc = a.kcode + (long)bh * a.Ncache * (DH / 2);
  const uint8_t* ks = a.kscale + (long)bh * a.Ncache * (DH / 16);
  const uint8_t* vc = a.vcode + (long)bh * a.Ncache * (DH / 2);
  const uint8_t* vs = a.vscale + (long)bh * a.Ncache * (DH / 16);
  const int last = a.Ncache - 1;

  float o[MT][NT][4], mrow[MT][2], lrow[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[mt][i][c] = 0.f;
    mrow[mt][0] = mrow[mt][1] = -INFINITY;
    lrow[mt][0] = lrow[mt][1] = 0.f;
  }
  for (int n = n_lo + 16 * warp; n < n_hi; n += 16 * kWarps) {
    RawK<DH> rk;
    RawV<DH> rv;
    load_k<DH>(kc, ks, n, last, g, t, rk);
    load_v<DH>(vc, vs, n, last, g, t, rv);
    // scores
    float s[MT][2][4];
    {
      uint32_t kf[2][KS][2];
      dequant_k<DH>(rk, kf);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[mt][j][c] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint4 q = qs[((mt * P + p) * KS + k) * 32 + lane];
            mma_f16(s[mt][0], &q.x, kf[0][k][0], kf[0][k][1]);
            mma_f16(s[mt][1], &q.x, kf[1][k][0], kf[1][k][1]);
          }
    }
    const bool masked = n < all_lo || n + 16 > all_hi;
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int slot = min(n + 4 * t + i, last);
      pos[i] = kpos != nullptr ? __ldg(kpos + slot) : slot;
    }
    uint32_t ph[MT][4], pl[MT][F32 ? 4 : 1];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {  // rows g and g + 8
        const RowPar& rp = par[mt * 16 + g + 8 * u];
        const float f = rp.f, slope = rp.slope;
        const int qpos = rp.qpos, lo = rp.lo, hi = rp.hi;
        float x[4], mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = kv4_score<F32>(a, s[mt][i >> 1][2 * u + (i & 1)], f, slope, qpos, pos[i]) * kLog2e;
          if (masked && (n + 4 * t + i >= len || pos[i] < lo || pos[i] >= hi)) x[i] = -INFINITY;
          mx = fmaxf(mx, x[i]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(mrow[mt][u], mx);
        if (__any_sync(0xffffffffu, m_new > mrow[mt][u])) {
          const float corr = m_new > mrow[mt][u] ? exp2_approx(mrow[mt][u] - m_new) : 1.f;
          lrow[mt][u] *= corr;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            o[mt][i][2 * u] *= corr;
            o[mt][i][2 * u + 1] *= corr;
          }
          mrow[mt][u] = m_new;
        }
        const float base = m_new == -INFINITY ? 0.f : m_new - kPShift;
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = exp2_approx(x[i] - base);
          lrow[mt][u] += p[i];
        }
        // A fragment: a0/a1 first n8 tile (rows g, g + 8), a2/a3 the second
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const __half2 h = __floats2half2_rn(p[2 * j], p[2 * j + 1]);
          ph[mt][2 * j + u] = h2_bits(h);
          if constexpr (F32) {
            const float2 back = __half22float2(h);
            pl[mt][2 * j + u] = h2_bits(__floats2half2_rn(p[2 * j] - back.x, p[2 * j + 1] - back.y));
          }
        }
      }
    }
    // O += P V
#pragma unroll
    for (int w = 0; w < DH / 64; ++w) {
      uint32_t v[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e2m1x8_f16(rv.c[j][w], v[j]);
        const __half2 sc = e4m3_pair((rv.s[j] >> (DH == 256 ? 8 * (w / 2) : 0)) & 0xffu);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[j][q] = h2_bits(__hmul2(h2_of(v[j][q]), sc));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half == 0 ? 0x5410u : 0x7632u;
          const uint32_t b0 = __byte_perm(v[0][q], v[1][q], sel);
          const uint32_t b1 = __byte_perm(v[2][q], v[3][q], sel);
          const int i = 8 * w + 2 * q + half;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if constexpr (F32) {
              // the tensor cores truncate what they add to an accumulator:
              // over thousands of steps that shows in fp32, so each step's
              // product is added by a rounding instruction
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(d, ph[mt], b0, b1);
              mma_f16(d, pl[mt], b0, b1);
#pragma unroll
              for (int c = 0; c < 4; ++c) o[mt][i][c] += d[c];
            } else {
              mma_f16(o[mt][i], ph[mt], b0, b1);
            }
          }
        }
    }
  }

  // the four warps' shares of each row joined
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float l = lrow[mt][u];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (t == 0) {
        s_m[warp][mt * 16 + g + 8 * u] = mrow[mt][u];
        s_l[warp][mt * 16 + g + 8 * u] = l;
      }
    }
  __syncthreads();  // Q is no longer read
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* dst = obuf + ((size_t)warp * kRows + mt * 16 + g + 8 * u) * DH + (2 * t + c) * NT;
#pragma unroll
        for (int i = 0; i < NT; i += 4)
          *reinterpret_cast<float4*>(dst + i) =
              make_float4(o[mt][i][2 * u + c], o[mt][i + 1][2 * u + c], o[mt][i + 2][2 * u + c],
                          o[mt][i + 3][2 * u + c]);
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
    if (a.nsplit > 1) {
      const size_t at = ((size_t)bh * a.M + m) * a.nsplit + split;
      *reinterpret_cast<float4*>(a.po + at * DH + d) = acc;
      if (d == 0) {
        a.pml[2 * at] = mx;
        a.pml[2 * at + 1] = l;
      }
    } else {
      kv4_finish<F32>(a, b, hkv, m, DH, d, acc, mx, l);
    }
  }
}

// dh / 4 threads a row, four elements each.
template <int DH, bool F32>
__global__ void __launch_bounds__(128)
k_kv4_combine(const __grid_constant__ Kv4AttnArgs a) {
  pdl_prologue();
  constexpr int LN = DH / 4;  // threads a row
  const long idx = ((long)blockIdx.x * 128 + threadIdx.x) / LN;
  const int d = (threadIdx.x % LN) * 4;
  if (idx >= (long)a.B * a.Hkv * a.M) return;
  const int bh = (int)(idx / a.M), m = (int)(idx % a.M);
  const float* ml = a.pml + (size_t)idx * a.nsplit * 2;
  const float* po = a.po + (size_t)idx * a.nsplit * DH + d;
  float mx = -INFINITY;
  for (int s = 0; s < a.nsplit; ++s) mx = fmaxf(mx, ml[2 * s]);
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < a.nsplit; ++s) {
    const float c = ml[2 * s] == -INFINITY ? 1.f : exp2_approx(ml[2 * s] - mx);
    const float4 v = *reinterpret_cast<const float4*>(po + (size_t)s * DH);
    l += c * ml[2 * s + 1];
    acc.x += c * v.x; acc.y += c * v.y; acc.z += c * v.z; acc.w += c * v.w;
  }
  kv4_finish<F32>(a, bh / a.Hkv, bh % a.Hkv, m, DH, d, acc, mx, l);
}

// K only: a CTA owns 64 slots at a time (16 a warp), their K fragments stay in
// registers while all rows of the head pass by (64 at a time through shared
// memory); every slot's sum is one CTA's, in row order, so the result does not
// depend on timing.
constexpr int kWRows = 64;

template <int DH, bool F32>
__global__ void __launch_bounds__(kThreads)
k_kv4_weight(const __grid_constant__ Kv4AttnArgs a, int steps) {
  constexpr int KS = DH / 16, P = F32 ? 2 : 1;
  pdl_prologue();
  extern __shared__ uint4 smem4[];
  uint4* qs = smem4;  // (kWRows / 16) * P * KS * 32
  __shared__ RowPar par[kWRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int bh = blockIdx.y, b = bh / a.Hkv, hkv = bh % a.Hkv;
  const int len = kv4_len(a, b), last = a.Ncache - 1;
  const uint8_t* kc = a.kcode + (long)bh * a.Ncache * (DH / 2);
  const uint8_t* ks = a.kscale + (long)bh * a.Ncache * (DH / 16);
  const int32_t* kpos = a.kpos != nullptr ? a.kpos + (long)bh * a.Ncache : nullptr;
  const float* w_in = a.w_in != nullptr ? a.w_in + (long)bh * a.Ncache : nullptr;
  float* w_out = a.w_out + (long)bh * a.Ncache;
  const int chunks = ceil_div(a.M, kWRows);
  for (int st = 0; st < steps; ++st) {
    const int n = (blockIdx.x * steps + st) * 64 + 16 * warp;
    const bool live = n < len;  // warp-uniform
    uint32_t kf[2][KS][2];
    int pos[4];
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
      RawK<DH> rk;
      load_k<DH>(kc, ks, n, last, g, t, rk);
      dequant_k<DH>(rk, kf);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int slot = min(n + 4 * t + i, last);
        pos[i] = kpos != nullptr ? __ldg(kpos + slot) : slot;
      }
    }
    for (int ch = 0; ch < chunks; ++ch) {
      const int m0 = ch * kWRows, rows = min(kWRows, a.M - m0);
      if (st == 0 || chunks > 1) {
        __syncthreads();
        stage_rows<DH, F32>(a, b, hkv, m0, (rows + 15) & ~15, qs, par, kWarps);
        __syncthreads();
      }
      if (!live) continue;
      for (int mt = 0; mt * 16 < rows; ++mt) {
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint4 q = qs[((mt * P + p) * KS + k) * 32 + lane];
            mma_f16(s[0], &q.x, kf[0][k][0], kf[0][k][1]);
            mma_f16(s[1], &q.x, kf[1][k][0], kf[1][k][1]);
          }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const RowPar rp = par[mt * 16 + g + 8 * u];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x =
                kv4_score<true>(a, s[i >> 1][2 * u + (i & 1)], rp.f, rp.slope, rp.qpos, pos[i]);
            const bool see = n + 4 * t + i < len && pos[i] >= rp.lo && pos[i] < rp.hi &&
                             rp.lse != -INFINITY;
            acc[i] += see ? exp2_approx((x - rp.lse) * kLog2e) : 0.f;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 4);
      acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 8);
      acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 16);
    }
    if (g == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int slot = n + 4 * t + i;
        if (slot < a.Ncache) w_out[slot] = (w_in != nullptr ? w_in[slot] : 0.f) + acc[i];
      }
    }
  }
}

template <int DH, bool F32>
cudaError_t launch_combine(const Kv4AttnArgs& a, cudaStream_t s) {
  const long rows = (long)a.B * a.Hkv * a.M;
  return launch_pdl(k_kv4_combine<DH, F32>, dim3((unsigned)ceil_div(rows * (DH / 4), 128)),
                    dim3(128), 0, s, a);
}

template <int DH, int MT, bool F32>
cudaError_t launch_attn(const Kv4AttnArgs& a, cudaStream_t s) {
  constexpr size_t q_bytes = (size_t)MT * (F32 ? 2 : 1) * (DH / 16) * 32 * 16;
  constexpr size_t o_bytes = (size_t)kWarps * 16 * MT * DH * 4;
  constexpr size_t smem = q_bytes > o_bytes ? q_bytes : o_bytes;
  auto kern = k_kv4_attn<DH, MT, F32>;
  static bool attr_set = false;
  if (!attr_set && smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  const long grid = (long)a.B * a.Hkv * a.nsplit * a.ntile;
  cudaError_t e = launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), smem, s, a);
  if (e != cudaSuccess || a.nsplit == 1) return e;
  return launch_combine<DH, F32>(a, s);
}

template <int DH, bool F32>
cudaError_t launch_weight(const Kv4AttnArgs& a, cudaStream_t s) {
  constexpr size_t smem = (size_t)(kWRows / 16) * (F32 ? 2 : 1) * (DH / 16) * 32 * 16;
  auto kern = k_kv4_weight<DH, F32>;
  static bool attr_set = false;
  if (!attr_set && smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  // rows that fit shared memory are staged once for several 64-slot groups
  const int groups = ceil_div(a.Ncache, 64);
  int steps = 1;
  if (a.M <= kWRows)
    while (steps < 8 && (long)ceil_div(groups, 2 * steps) * a.B * a.Hkv >= 8 * kSmTarget) steps *= 2;
  return launch_pdl(kern, dim3((unsigned)ceil_div(groups, steps), a.B * a.Hkv), dim3(kThreads),
                    smem, s, a, steps);
}

// The kernel, rows of a tile, tiles and shares of the slots for these sizes.
struct AttnPlan {
  bool tc;  // k_kv4_attn_tc: 256-row tiles; else k_kv4_attn with 16 mt rows
  int mt, ntile, nsplit;
};
AttnPlan attn_plan(int dtype, int B, int N, int Hq, int Hkv, int dh, int T) {
  AttnPlan p;
  const int M = T * (Hq / Hkv);
  p.tc = dtype == PS_BF16 && dh <= 128 && M >= 64;
  if (p.tc) {
    p.mt = 0;
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
  p.mt = (M > 16 && dh <= 128) ? 2 : 1;
  p.ntile = ceil_div(M, 16 * p.mt);
  const long base = (long)B * Hkv * p.ntile;
  const int most = ceil_div(N, 128);  // at least 128 slots a share
  long want = ceil_div(4 * kSmTarget, base);
  if (want > most) want = most;
  if (want > 256) want = 256;
  p.nsplit = (int)(want < 1 ? 1 : want);
  return p;
}

}  // namespace

size_t kv4_attn_ws(int B, int N, int Hq, int Hkv, int dh, int T) {
  // either type's: the size does not name it
  const int a = attn_plan(PS_BF16, B, N, Hq, Hkv, dh, T).nsplit;
  const int b = attn_plan(PS_F32, B, N, Hq, Hkv, dh, T).nsplit;
  const int nsplit = a > b ? a : b;
  if (nsplit == 1) return 0;
  Carver c(nullptr);
  const size_t rows = (size_t)B * T * Hq * nsplit;
  c.take<float>(rows * dh);
  c.take<float>(rows * 2);
  return c.bytes();
}

size_t kv4_weight_ws(int, int, int, int, int, int) { return 0; }

cudaError_t kv4_attn_run(Kv4AttnArgs a, cudaStream_t s) {
  const AttnPlan p = attn_plan(a.dtype, a.B, a.Ncache, a.Hq, a.Hkv, a.dh, a.T);
  a.ntile = p.ntile;
  a.nsplit = p.nsplit;
  if (a.nsplit > 1) {
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
#define PS_KV4_CASE(DH, MT)                                                          \
  if (a.dh == DH && p.mt == MT)                                                      \
    return f32 ? launch_attn<DH, MT, true>(a, s) : launch_attn<DH, MT, false>(a, s);
  PS_KV4_CASE(64, 1)
  PS_KV4_CASE(64, 2)
  PS_KV4_CASE(128, 1)
  PS_KV4_CASE(128, 2)
  PS_KV4_CASE(256, 1)
#undef PS_KV4_CASE
  return cudaErrorInvalidValue;
}

cudaError_t kv4_weight_run(const Kv4AttnArgs& a, cudaStream_t s) {
  const bool f32 = a.dtype == PS_F32;
  switch (a.dh) {
    case 64: return f32 ? launch_weight<64, true>(a, s) : launch_weight<64, false>(a, s);
    case 128: return f32 ? launch_weight<128, true>(a, s) : launch_weight<128, false>(a, s);
    case 256: return f32 ? launch_weight<256, true>(a, s) : launch_weight<256, false>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ps
