// Rotary positions of query and key rows, fused with their way into the cache.
//
// A pair (x, y) of a head's elements is turned by the angle position * freq.  The
// angle is kept as a fraction of a turn in 64-bit fixed point: position * turns
// modulo 2^64 is exact at any position, where a product in fp32 is off by a tenth
// of a radian at a million.  Its nearest quarter turn is split off as an integer and
// the rest, at most an eighth of a turn, is a float good to 2^-28 of a turn, 2^-25.3
// radians.  (Added on by the derivatives, what that leaves took the worst mean error of an
// angle from 2.4e-8 to 1.5e-8 only: cosine and sine are rounded themselves.)
//
// A CTA takes a token of a sequence: its threads work out the cosine and sine of
// every pair once into shared memory, then move all heads of Q, K and V, each
// thread the same 2 W elements of one head after another: two W-element vectors
// that hold both partners of W pairs.  Memory bound: a row is read and written
// once.  2 x 4096 rows of 32 heads of Q, K and V, bf16: 65 us, 91 % of a copy's rate
// (four tokens a CTA 70, CTAs of 512 threads 81); 537 listed rows of 32 heads of K and V
// 8.5 (four tokens 12.9).  The first heads' loads put before the angles made both
// slower, 131 and 14.8.  A few tokens' rows are the latency of one list entry, one sine,
// one load and one store.
#include "ops.h"
#include "vec.cuh"

namespace ps {
namespace {

constexpr int kRT = 256;   // threads

// W elements, as one access.
template <typename T, int W>
struct alignas(sizeof(T) * W) Pack {
  T v[W];
};

__device__ __forceinline__ void put(float& d, float x) { d = x; }
__device__ __forceinline__ void put(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// cos and sin of t turns, t in units of 2^-64.
__device__ __forceinline__ float2 cos_sin(uint64_t t) {
  const uint32_t hi = (uint32_t)(t >> 32);
  const uint32_t quarter = (hi + 0x20000000u) >> 30;       // nearest
  const int32_t rest = (int32_t)(hi - (quarter << 30));    // of a turn, 2^-32: |rest| <= 2^29
  float s, c;
  sincospif((float)rest * 0x1p-31f, &s, &c);
  if (quarter & 1) {
    const float x = c;
    c = -s;
    s = x;
  }
  if (quarter & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c, s);
}

// Row j of sequence b's list: its row, position and slot; false where there is none.
__device__ __forceinline__ bool rope_row(const RopeArgs& a, int b, int j, int* r, long* pos,
                                         long* slot) {
  if (j >= a.T || (a.cnt != nullptr && j >= __ldg(a.cnt + b))) return false;
  const long base = (long)b * a.T;
  *r = a.rows != nullptr ? __ldg(a.rows + base + j) : j;
  if (*r < 0 || *r >= a.T) return false;
  const long next = (a.off != nullptr ? (long)__ldg(a.off + b) : 0L) + *r;
  *pos = a.pos != nullptr ? (long)__ldg(a.pos + base + *r) : next;
  *slot = a.dst != nullptr ? (long)__ldg(a.dst + base + *r) : next;
  return true;
}

template <typename T, int W, bool PAIRS>
__global__ void __launch_bounds__(kRT)
k_rope(const __grid_constant__ RopeArgs a) {
  pdl_prologue();
  __shared__ float2 cs[128];
  const int b = blockIdx.x / a.T;
  int r;
  long pos, slot;
  if (!rope_row(a, b, blockIdx.x - b * a.T, &r, &pos, &slot)) return;
  const int half = a.rot >> 1;
  if (threadIdx.x < half) {
    float2 x = cos_sin((uint64_t)pos * __ldg(a.turns + threadIdx.x));
    x.x *= a.amp;
    x.y *= a.amp;
    cs[threadIdx.x] = x;
  }
  __syncthreads();
  using P = Pack<T, W>;
  const int units = a.dh / (2 * W), turned = half / W;  // of a head; of them rotated
  const int per = kRT / units;                          // heads at a time
  const int u = threadIdx.x % units, h0 = threadIdx.x / units;
  if (h0 >= per) return;
  const bool rot = u < turned;
  // the unit's two vectors in a head
  const int at_plain = 2 * W * u;
  const int at0 = rot && !PAIRS ? W * u : at_plain;
  const int at1 = rot && !PAIRS ? half + W * u : at_plain + W;
#pragma unroll 1
  for (int g = h0; g < a.end[2]; g += per) {
    const int n = (g >= a.end[0]) + (g >= a.end[1]);
    const RopePart& p = a.part[n];
    const int h = g - (n > 0 ? a.end[n - 1] : 0);
    const bool turn = rot && p.rotate;
    long to = r;
    if (p.slots > 0) {
      if (slot < 0 || slot >= p.slots) continue;
      to = slot;
    }
    const T* x = static_cast<const T*>(p.X) + b * p.x_bld + r * p.x_ld + (long)h * a.dh;
    T* y = static_cast<T*>(p.Y) + b * p.y_bld + to * p.y_ld + (long)h * a.dh;
    if (!turn && x == y) continue;
    const int i0 = p.rotate ? at0 : at_plain, i1 = p.rotate ? at1 : at_plain + W;
    P v0 = *reinterpret_cast<const P*>(x + i0), v1 = *reinterpret_cast<const P*>(x + i1);
    if (turn) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float2 q = cs[W * u + e];
        // PAIRS: the unit's 2 W elements are W neighbouring pairs
        T& px = !PAIRS ? v0.v[e] : 2 * e < W ? v0.v[2 * e % W] : v1.v[2 * e % W];
        T& py = !PAIRS ? v1.v[e] : 2 * e + 1 < W ? v0.v[(2 * e + 1) % W] : v1.v[(2 * e + 1) % W];
        const float fx = to_f32(px), fy = to_f32(py);
        put(px, fx * q.x - fy * q.y);
        put(py, fx * q.y + fy * q.x);
      }
    }
    *reinterpret_cast<P*>(y + i0) = v0;
    *reinterpret_cast<P*>(y + i1) = v1;
  }
}

template <typename T, int W, bool PAIRS>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  return launch_pdl(k_rope<T, W, PAIRS>, dim3((unsigned)((long)a.B * a.T)), dim3(kRT), 0, s, a);
}

template <typename T, int W>
cudaError_t by_layout(const RopeArgs& a, cudaStream_t s) {
  return a.pairs ? launch<T, W, true>(a, s) : launch<T, W, false>(a, s);
}

}  // namespace

cudaError_t rope_run(RopeArgs a, cudaStream_t s) {
  // The widest vectors that rot / 2 is made of (dh, a multiple of 16, then is too).
  const int half = a.rot / 2;
  if (a.dtype == PS_F32) {
    if (half % 4 == 0) return by_layout<float, 4>(a, s);
    return half % 2 == 0 ? by_layout<float, 2>(a, s) : by_layout<float, 1>(a, s);
  }
  using H = __nv_bfloat16;
  if (half % 8 == 0) return by_layout<H, 8>(a, s);
  if (half % 4 == 0) return by_layout<H, 4>(a, s);
  return half % 2 == 0 ? by_layout<H, 2>(a, s) : by_layout<H, 1>(a, s);
}

}  // namespace ps
