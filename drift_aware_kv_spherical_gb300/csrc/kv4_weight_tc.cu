// The weight of many query rows a KV head on the slots of a 4-bit KV cache, on
// the tcgen05 tensor cores:
//   w_out[slot] = w_in[slot] + sum over rows of exp(score(row, slot) - lse[row]).
//
// The product is taken as K Q^T: a slot is a TMEM lane and a row a column, so a
// thread sums its slot's weights over the columns and no sum crosses threads.  A
// CTA takes 256 slots of one KV head (two 128-slot tiles, dequantised once: code
// times scale is exact in bf16, so the queries stay as they are) and passes all
// rows by them, 128 at a time.  19 warps:
//   0-15   four groups of four: a group reads one slot tile's products of every
//          second step, so that one step's exponentials run under the next one's
//          MMAs.  Warps 0-7 dequantise the slots first
//   16, 17 the queries, by cp.async into a ring of four operands, and what the
//          rows bring: their lse, span, position and slope.  With spans, steps
//          whose rows see none of the 256 slots are left out
//   18     issues the MMAs: two 128 x 128 products a step into one half of TMEM
// Where there are few blocks of slots, the rows are split over the CTAs of a
// cluster, whose sums are added in rank order: the result does not depend on
// timing (2048 rows x 4 heads on 1024 slots 16.5 us, unsplit 20.8).
//
// What bounds it: 2048 rows x 32 heads on 4096 slots 82 us, 0.84 PFLOP/s, 43 % of
// a large library product's rate.  The tensor cores and the exponentials are each
// busy 41 % of the time; the rest is the waits between them, 4.5 us a CTA of
// set-up (slots read and dequantised before the first product) and the last of
// four rounds of CTAs.  With 128 slots a CTA and two CTAs an SM it took 130 us:
// 32 KB of queries a step are then all that an SM's share of L2 delivers.
// Every mbarrier wait is bounded (tc::mbar_wait); after a timeout the CTA waits
// for the MMAs it issued, frees TMEM and returns with the status word set.
#include "kv4_tc.cuh"

namespace ps {
namespace {

constexpr int kWThreads = 608;
constexpr int kTile = 128;    // rows a step; slots of a slot tile
constexpr int kSlots = 256;   // slots of a CTA
constexpr int kStages = 4;    // query operands
constexpr int kMaxSplit = 8;  // CTAs of a portable cluster

// What a step's rows bring, by column.
struct StepRows {
  float nlse[kTile];     // -lse; -inf past the last row
  float slope[kTile];    // distance bias, in units of the cap if there is one
  int qpos[kTile];       // the row's position; as float from the block's first slot
                         // where slots are positions
  int lo[kTile];         // positions seen: lo + [0, num)
  uint32_t num[kTile];
  int cols;                            // columns in use, a multiple of 32; 0: the end
  int any_lo, any_hi, all_lo, all_hi;  // slots that some, that every row sees
  int pad[3];
};

template <int DH>
struct WSmem {
  static constexpr uint32_t kOp = (DH / 64) * 16384u;  // 128 rows of DH bf16
  static constexpr uint32_t kQ = 2 * kOp, kRows = kQ + kStages * kOp;
  static constexpr uint32_t kSum = kRows + kStages * sizeof(StepRows);  // float [3][256]
  static constexpr uint32_t kBar = kSum + 3 * kSlots * 4;
  static constexpr size_t kBytes = 1024 + kBar + 256;
};

// The row as bf16 into row r of an operand: 16-byte chunks, eight elements each.
template <int DH>
__device__ __forceinline__ void put_row_bf16(uint8_t* op, int r, const RawRow<DH>& v) {
#pragma unroll
  for (int p = 0; p < DH / 32; ++p) {
    const uint32_t two = ((p < 2 ? v.s.x : v.s.y) >> (16 * (p & 1))) & 0xffffu;
    const uint32_t sc = h2_bits(e4m3x2_f16(two));
    const uint32_t w[4] = {v.c[p].x, v.c[p].y, v.c[p].z, v.c[p].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 s = h2_of(__byte_perm(sc, sc, i < 2 ? 0x1010u : 0x3232u));
      uint32_t h[4], o[4];
      e2m1x8_f16(w[i], h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __float22bfloat162_rn(__half22float2(__hmul2(h2_of(h[e]), s)));
        o[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(op + sw128(r, 4 * p + i)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// The sum of 32 columns' weights: s their raw products, c0 the first column.
// GEN: capped scores, a distance bias or explicit positions.
template <bool GEN, bool MASKED>
__device__ __forceinline__ float weigh32(const Kv4AttnArgs& a, float* s, const StepRows& rows,
                                         int c0, int pos, float dpos) {
  float f = a.scale;  // takes s to natural units
  if constexpr (GEN) {
    if (a.cap > 0.f) {
      const float fy = fminf(fmaxf(a.scale * a.inv_cap, -FLT_MAX), FLT_MAX);
      float top = 0.f;
#pragma unroll
      for (int c = 0; c < 32; c += 2) top = max3(top, fabsf(s[c]), fabsf(s[c + 1]));
      if (__all_sync(0xffffffffu, top * fabsf(fy) <= kTanhTop)) {
        tanh_series<32>(s, fy);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) s[c] = tanhf(s[c] * fy);
      }
      f = a.cap;
    } else if (a.slope != nullptr) {
      const uint64_t ff = f2_pack(f, f);
      f = 1.f;
#pragma unroll
      for (int c = 0; c < 32; c += 2)
        f2_unpack(f2_mul(f2_pack(s[c], s[c + 1]), ff), s[c], s[c + 1]);
    }
    if (a.slope != nullptr) {  // in units of the cap, as s is
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float d = a.kpos != nullptr ? (float)(rows.qpos[c0 + c] - pos)
                                          : __int_as_float(rows.qpos[c0 + c]) - dpos;
        s[c] = fmaf(-rows.slope[c0 + c], fabsf(d), s[c]);
      }
    }
  }
  // natural units up to the exponential: score and lse nearly cancel
  const uint64_t e = f2_pack(kLog2e, kLog2e), ff = f2_pack(f, f);
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(rows.nlse + c0 + c);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = c + 2 * h;
      float x0, x1;
      f2_unpack(f2_mul(f2_fma(f2_pack(s[k], s[k + 1]), ff, h == 0 ? nl.x : nl.y), e), x0, x1);
      if constexpr (MASKED) {
        if ((uint32_t)pos - (uint32_t)rows.lo[c0 + k] >= rows.num[c0 + k]) x0 = -INFINITY;
        if ((uint32_t)pos - (uint32_t)rows.lo[c0 + k + 1] >= rows.num[c0 + k + 1]) x1 = -INFINITY;
      }
      sum[h] = f2_add(sum[h], f2_pack(exp2_approx(x0), exp2_approx(x1)));
    }
  }
  float s0, s1;
  f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
  return s0 + s1;
}

// A step's columns; `free` is arrived at once they have been read.
template <bool GEN, bool MASKED>
__device__ __forceinline__ float weigh_step(const Kv4AttnArgs& a, uint32_t col,
                                            const StepRows& rows, int pos, float dpos,
                                            uint64_t* free) {
  const int cols = rows.cols;
  float sum = 0.f;
#pragma unroll 1
  for (int c0 = 0; c0 < cols; c0 += 32) {
    float s[32];
    tc::tmem_ld32_nowait(col + c0, reinterpret_cast<uint32_t*>(s));
    tc::tmem_wait_ld();
    if (c0 == cols - 32) {
      tc::fence_before_sync();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) tc::mbar_arrive(free);
    }
    sum += weigh32<GEN, MASKED>(a, s, rows, c0, pos, dpos);
  }
  return sum;
}

// The same for 128 columns that every row sees: the next 32 are on their way from
// TMEM (about 280 clocks) while these are summed (82 us for 85).
__device__ __forceinline__ float weigh_all(const Kv4AttnArgs& a, uint32_t col, const StepRows& rows,
                                           uint64_t* free) {
  float s[2][32], sum = 0.f;
  tc::tmem_ld32_nowait(col, reinterpret_cast<uint32_t*>(s[0]));
#pragma unroll
  for (int k = 0; k < kTile / 32; ++k) {
    tc::tmem_wait_ld();
    if (k + 1 < kTile / 32) {
      tc::tmem_ld32_nowait(col + 32 * (k + 1), reinterpret_cast<uint32_t*>(s[(k + 1) & 1]));
    } else {
      tc::fence_before_sync();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) tc::mbar_arrive(free);
    }
    sum += weigh32<false, false>(a, s[k & 1], rows, 32 * k, 0, 0.f);
  }
  return sum;
}

template <int DH, bool GEN>
__global__ void __launch_bounds__(kWThreads, 1)
k_kv4_weight_tc(const __grid_constant__ Kv4AttnArgs a, const int blocks) {
  using SM = WSmem<DH>;
  pdl_prologue();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-tc::smem_u32(smem_raw) & 1023);  // known to be shared memory
  StepRows* steps = reinterpret_cast<StepRows*>(smem + SM::kRows);
  float* sums = reinterpret_cast<float*>(smem + SM::kSum);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBar);
  uint64_t *empty = full + kStages, *s_full = full + 2 * kStages;  // [half][slot tile]
  uint64_t *s_empty = s_full + 4, *k_full = s_full + 8, *drain = s_full + 10;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 11);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform to the compiler too
  const int split = blockIdx.x % a.nsplit, block = blockIdx.x / a.nsplit % blocks;
  const int bh = blockIdx.x / a.nsplit / blocks, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int len = kv4_len(a, b), last = a.Ncache - 1, n0 = block * kSlots;
  const long base = (long)bh * a.Ncache;
  if (n0 >= len) {  // past the sequence: the whole cluster is
    if (split == 0 && tid < kSlots && n0 + tid < a.Ncache)
      a.w_out[base + n0 + tid] = a.w_in != nullptr ? a.w_in[base + n0 + tid] : 0.f;
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(full + i, 2);
      tc::mbar_init(empty + i, 8);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(s_empty + i, 4);
    }
    tc::mbar_init(k_full, 4);
    tc::mbar_init(k_full + 1, 4);
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 18) tc::tmem_alloc(tmem_slot, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp < 16) {
    // ------------------------------------------------------------ weights
    const int g = (warp >> 2) & 1, half = warp >> 3;  // slot tile; odd or even steps
    if (warp < 8) {
      RawRow<DH> k;
      load_row<DH>(a.kcode, a.kscale, base + min(n0 + tid, last), k);
      put_row_bf16<DH>(smem + g * SM::kOp, tid & 127, k);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(k_full + g);
    }
    const int w0 = g * kTile + (warp & 3) * 32;  // the warp's first slot in the block
    const int lo = n0 + w0, hi = min(lo + 32, len);
    const int pos = GEN && a.kpos != nullptr ? __ldg(a.kpos + base + min(lo + lane, last))
                                             : lo + lane;
    const float dpos = (float)(w0 + lane);
    const uint32_t col = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * 256 +
                         g * kTile;
    uint64_t *mine = s_full + half * 2 + g, *free = s_empty + half * 2 + g;
    float sum = 0.f, low = 0.f;  // low: what the sum's rounding has lost
    for (int i = half;; i += 2) {
      const int st = i % kStages;
      const bool ok = tc::mbar_wait(full + st, (i / kStages) & 1, a.status, abort_flag) &&
                      tc::mbar_wait(mine, (i >> 1) & 1, a.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::fence_after_sync();
      const StepRows& rows = steps[st];
      if (rows.cols == 0) break;
      if (lo < rows.any_hi && hi > rows.any_lo) {
        const bool all = lo >= rows.all_lo && hi <= rows.all_hi;
        float x;
        if (!GEN && all && rows.cols == kTile) x = weigh_all(a, col, rows, free);
        else if (all) x = weigh_step<GEN, false>(a, col, rows, pos, dpos, free);
        else x = weigh_step<GEN, true>(a, col, rows, pos, dpos, free);
        const float y = x + low, t = sum + y;
        low = y - (t - sum);
        sum = t;
      } else if (lane == 0) {
        tc::mbar_arrive(free);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty + st);
    }
    sums[half * kSlots + w0 + lane] = sum;
    tc::fence_before_sync();
  } else if (warp < 18) {
    // ------------------------------------------------------------ queries
    const int p = tid - 512;  // of rows p and p + 64
    const bool by_pos = GEN && a.kpos != nullptr;
    const int tiles = (a.M + kTile - 1) / kTile, each = (tiles + a.nsplit - 1) / a.nsplit;
    const int end = min(tiles, (split + 1) * each);
    int i = 0, pending = -1;
    bool ok = true;
    auto publish = [&](int st) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(full + st);
    };
    // What the lane's rows bring, asked for a step ahead: rows lane + 32 k of the
    // step for the spans, p and p + 64 (k = warp, warp + 2) for the rest
    float lse[2], slope[2];
    int2 span[4];
    int qpos[2];
    auto ask = [&](int r) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        span[k] = make_int2(0, INT32_MAX);
        const int m = r * kTile + lane + 32 * k, t = row_token(a, m);
        if (r < end && m < a.M && a.span != nullptr)
          span[k] = row_span(a, (long)b * a.T + t);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int m = r * kTile + p + 64 * k, t = row_token(a, m), h = hkv * a.G + (m - t * a.G);
        const bool in = r < end && m < a.M;
        const long tok = (long)b * a.T + t;
        lse[k] = in ? __ldg(a.lse_in + tok * a.Hq + h) : INFINITY;
        slope[k] = GEN && in && a.slope != nullptr ? __ldg(a.slope + h) : 0.f;
        qpos[k] = GEN && in && a.qpos != nullptr ? __ldg(a.qpos + tok) : 0;
      }
    };
    ask(split * each);
    for (int r = split * each; r < end; ++r) {
      const int m0 = r * kTile;
      int any_lo = 0, any_hi = len, all_lo = 0, all_hi = len;
      if (a.span != nullptr) {
        if (by_pos) {
          all_hi = -1;
        } else {
          int lo = INT32_MAX, hi = INT32_MIN, lo2 = INT32_MIN, hi2 = INT32_MAX;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (m0 + lane + 32 * k >= a.M) continue;
            if (span[k].x < span[k].y) {
              lo = min(lo, span[k].x);
              hi = max(hi, span[k].y);
            }
            lo2 = max(lo2, span[k].x);
            hi2 = min(hi2, span[k].y);
          }
          any_lo = __reduce_min_sync(0xffffffffu, lo);
          any_hi = min(len, __reduce_max_sync(0xffffffffu, hi));
          all_lo = __reduce_max_sync(0xffffffffu, lo2);
          all_hi = min(len, __reduce_min_sync(0xffffffffu, hi2));
          if (any_lo >= n0 + kSlots || any_hi <= n0) {
            ask(r + 1);
            continue;
          }
        }
      }
      const int st = i % kStages;
      const uint32_t ph = ((i / kStages) & 1) ^ 1;
      StepRows& rows = steps[st];
      // no stage free: what is under way is handed over first
      if (pending >= 0 && !__all_sync(0xffffffffu, tc::mbar_test(empty + st, ph))) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        publish(pending);
        pending = -1;
      }
      ok = tc::mbar_wait(empty + st, ph, a.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = p + 64 * k, m = m0 + c;
        const bool in = m < a.M;
        const int t = row_token(a, m), h = hkv * a.G + (m - t * a.G);
        fetch_q<DH>(a.Q, in ? static_cast<const __nv_bfloat16*>(a.Q) + (long)b * a.q_bld +
                             (long)t * a.q_ld + (long)h * DH
                       : nullptr,
                    tc::smem_u32(smem + SM::kQ + st * SM::kOp), c & ~31);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = p + 64 * k;
        const int2 seen = p < 32 ? span[2 * k] : span[2 * k + 1];
        rows.nlse[c] = -lse[k];
        rows.lo[c] = seen.x;
        rows.num[c] = seen.x < seen.y ? (uint32_t)seen.y - (uint32_t)seen.x : 0u;
        if constexpr (GEN) {
          rows.slope[c] = a.cap > 0.f ? slope[k] * a.inv_cap : slope[k];
          rows.qpos[c] = by_pos ? qpos[k] : __float_as_int((float)(qpos[k] - n0));
        }
      }
      if (p == 0) {
        rows.cols = min((a.M - m0 + 31) & ~31, kTile);
        rows.any_lo = any_lo;
        rows.any_hi = any_hi;
        rows.all_lo = all_lo;
        rows.all_hi = all_hi;
      }
      ask(r + 1);
      if (pending >= 0) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        publish(pending);
      }
      pending = st;
      ++i;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ok && pending >= 0) publish(pending);
    for (int e = 0; ok && e < 2; ++e, ++i) {  // the end, for odd and for even steps
      const int st = i % kStages;
      ok = tc::mbar_wait(empty + st, ((i / kStages) & 1) ^ 1, a.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (p == 0) steps[st].cols = 0;
      publish(st);
    }
  } else {
    // ------------------------------------------------------------ MMAs
    const uint32_t kb = tc::smem_u32(smem), qb = kb + SM::kQ;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = tc::mbar_wait(bar, parity, a.status, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
    };
    for (int i = 0, ends = 0; ends < 2; ++i) {
      const int st = i % kStages, half = i & 1;
      wait(full + st, (i / kStages) & 1);
      const int cols = ok ? *static_cast<volatile int*>(&steps[st].cols) : 0;
      const uint32_t id = tc::idesc_bf16(128, cols, false);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (i == 0) wait(k_full + g, 0);
        wait(s_empty + half * 2 + g, ((i >> 1) & 1) ^ 1);
        if (ok && elect_one()) {
          if (cols > 0) {
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
              const uint32_t off = (kk / 4) * 16384u + (kk % 4) * 32u;
              tc::mma_bf16(tmem + half * 256 + g * kTile,
                           tc::desc_sw128(kb + g * SM::kOp + off, 16, 1024),
                           tc::desc_sw128(qb + st * SM::kOp + off, 16, 1024), id, kk > 0);
            }
          }
          tc::mma_commit(s_full + half * 2 + g);
        }
        __syncwarp();
      }
      if (!ok) break;
      __syncwarp();
      ends += cols == 0;
    }
    if (!ok) {  // wait for the MMAs issued before TMEM is freed
      if (elect_one()) tc::mma_commit(drain);
      const uint64_t t0 = tc::globaltimer();
      while (!tc::mbar_try_wait(drain, 0) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 18) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  float w = 0.f;
  if (tid < kSlots) {
    w = sums[tid] + sums[kSlots + tid];
    sums[2 * kSlots + tid] = w;
  }
  if (a.nsplit > 1) {
    __syncwarp();
    tc::cluster_sync_all();
    if (split == 0 && tid < kSlots) {
      const uint32_t at = tc::smem_u32(sums + 2 * kSlots + tid);
      for (int q = 1; q < a.nsplit; ++q) w += tc::ld_dsmem_f32(tc::cluster_map(at, q));
    }
    __syncwarp();
    tc::cluster_sync_all();  // no CTA leaves while another still reads its sums
  }
  if (split == 0 && tid < kSlots && n0 + tid < a.Ncache)
    a.w_out[base + n0 + tid] =
        (a.w_in != nullptr ? a.w_in[base + n0 + tid] : 0.f) + (n0 + tid < len ? w : 0.f);
}

template <int DH, bool GEN>
cudaError_t launch_weight_tc(Kv4AttnArgs a, cudaStream_t s) {
  auto kern = k_kv4_weight_tc<DH, GEN>;
  static DeviceOnce once;
  const cudaError_t e = allow_smem(kern, WSmem<DH>::kBytes, once);
  if (e != cudaSuccess) return e;
  // row splits: the fewest steps, the set-up and the join counted as four, of
  // the SM that takes the most CTAs
  const int blocks = ceil_div(a.Ncache, kSlots), tiles = ceil_div(a.M, kTile);
  const long base = (long)a.B * a.Hkv * blocks;
  a.nsplit = 1;
  long best = ceil_div(base, a.num_sms) * (long)(tiles + 4);
  for (int n = 2; n <= kMaxSplit && n <= tiles; ++n) {
    const long cost = ceil_div(base * n, a.num_sms) * (long)(ceil_div(tiles, n) + 4);
    if (cost < best) {
      best = cost;
      a.nsplit = n;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(base * a.nsplit));
  cfg.blockDim = dim3(kWThreads);
  cfg.dynamicSmemBytes = WSmem<DH>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.nsplit;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.nsplit > 1 ? 1 : 0;
  return launch_ex(cfg, kern, a, blocks);
}

}  // namespace

cudaError_t kv4_weight_tc_launch(const Kv4AttnArgs& a, cudaStream_t s) {
  const bool gen = a.cap > 0.f || a.slope != nullptr || a.kpos != nullptr;
  if (a.dh == 64) return gen ? launch_weight_tc<64, true>(a, s) : launch_weight_tc<64, false>(a, s);
  if (a.dh == 128)
    return gen ? launch_weight_tc<128, true>(a, s) : launch_weight_tc<128, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace ps
