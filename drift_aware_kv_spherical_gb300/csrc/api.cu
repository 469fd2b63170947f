// The C ABI of libpolestar: handle management, argument validation,
// workspace sizing and dispatch to the kernels.  Declarations and the
// meaning of every argument are in include/polestar.h.
#include <cmath>
#include <cstdio>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "ops.h"

namespace ps {

struct TraceRec {
  const void* kernel;
  cudaEvent_t a, b;
};
struct TraceSink {
  std::vector<TraceRec> recs;
  cudaEvent_t pending = nullptr;
};

// The calling thread's sink while it runs a ps_* call on a tracing handle.
thread_local TraceSink* g_trace = nullptr;

void trace_begin(cudaStream_t s) {
  if (g_trace == nullptr) return;
  cudaEvent_t a;
  if (cudaEventCreate(&a) != cudaSuccess) return;
  cudaEventRecord(a, s);
  g_trace->pending = a;
}

void trace_end(cudaStream_t s, const void* kernel) {
  if (g_trace == nullptr || g_trace->pending == nullptr) return;
  cudaEvent_t b;
  if (cudaEventCreate(&b) != cudaSuccess) {
    cudaEventDestroy(g_trace->pending);
    g_trace->pending = nullptr;
    return;
  }
  cudaEventRecord(b, s);
  g_trace->recs.push_back({kernel, g_trace->pending, b});
  g_trace->pending = nullptr;
}

}  // namespace ps

using namespace ps;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define PS_REQUIRE(cond) \
  do {                   \
    if (!(cond)) return PS_ERR_ARG; \
  } while (0)

#define PS_PTR(p) PS_REQUIRE((p) != nullptr && aligned16(p))
#define PS_OPT_PTR(p) PS_REQUIRE((p) == nullptr || aligned16(p))
// arrays read or written one element at a time only need to exist
#define PS_NN(p) PS_REQUIRE((p) != nullptr)

thread_local char g_last_cuda_error[192] = "";

ps_status launch_status(cudaError_t e) {
  if (e == cudaSuccess) return PS_OK;
  std::snprintf(g_last_cuda_error, sizeof(g_last_cuda_error), "%s: %s", cudaGetErrorName(e),
                cudaGetErrorString(e));
  return PS_ERR_CUDA;
}

ps_status check_ws(size_t need, const void* ws, size_t ws_bytes) {
  if (need == 0) return PS_OK;
  if (ws == nullptr || ws_bytes < need) return PS_ERR_WORKSPACE;
  if (!aligned16(ws)) return PS_ERR_ARG;
  return PS_OK;
}

bool dtype_ok(int dt) { return dt == PS_F32 || dt == PS_BF16; }

// Sets the calling thread's trace sink for the duration of one ps_* call.
struct TraceScope {
  explicit TraceScope(ps_handle h) { g_trace = h != nullptr ? h->trace : nullptr; }
  ~TraceScope() { g_trace = nullptr; }
};

void trace_clear(TraceSink* t) {
  for (auto& r : t->recs) {
    cudaEventDestroy(r.a);
    cudaEventDestroy(r.b);
  }
  t->recs.clear();
}

constexpr int kMaxC = 256;
constexpr int kMaxD = 8192;
constexpr int kMaxDh = 256;

bool kv4_dh_ok(int dh) { return dh == 64 || dh == 128 || dh == 256; }
// Query rows of a call, without products that leave their type.
bool kv4_rows_ok(int B, int T, int Hq) {
  constexpr long most = INT32_MAX / 64;
  return T <= most && Hq <= most && (long)T * Hq <= most && (long)T * Hq * B <= most;
}
// Slots a head: a few tiles more than these still are an int.
constexpr int kMaxSlots = INT32_MAX - (1 << 16);
// Sizes of an attention over sequences: S of them, Tq rows, max_k slots at most.
bool attn_sizes_ok(int S, int max_k, int Hq, int Hkv, int dh, int Tq, int max_q) {
  return S >= 0 && S <= (1 << 20) && max_q >= 1 && max_k >= 1 && Tq >= 0 && Hkv >= 1 &&
         Hkv <= 512 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= 4096 &&
         (long)Tq * Hq <= (1 << 30) && dh > 0 && dh % 16 == 0 && dh <= kMaxDh;
}

}  // namespace

extern "C" {

ps_status ps_create(int device, ps_handle* out) {
  if (out == nullptr) return PS_ERR_ARG;
  *out = nullptr;
  int n = 0;
  if (cudaGetDeviceCount(&n) != cudaSuccess || device < 0 || device >= n)
    return PS_ERR_ARG;
  cudaDeviceProp prop;
  cudaError_t e = cudaGetDeviceProperties(&prop, device);
  if (e != cudaSuccess) return launch_status(e);
  if (!(prop.major == 10 && prop.minor == 3)) return PS_ERR_UNSUPPORTED;
  e = cudaSetDevice(device);
  if (e != cudaSuccess) return launch_status(e);
  auto* h = new (std::nothrow) ps_handle_s;
  if (h == nullptr) return PS_ERR_CUDA;
  h->device = device;
  h->num_sms = prop.multiProcessorCount;
  h->status = nullptr;
  h->trace = nullptr;
  h->aux = nullptr;
  e = cudaMalloc(&h->status, 16);
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, 16);
  if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&h->aux, cudaStreamNonBlocking);
  if (e != cudaSuccess) {
    if (h->status) cudaFree(h->status);
    if (h->aux) cudaStreamDestroy(h->aux);
    delete h;
    return launch_status(e);
  }
  *out = h;
  return PS_OK;
}

ps_status ps_destroy(ps_handle h) {
  if (h == nullptr) return PS_ERR_ARG;
  if (h->trace != nullptr) {
    trace_clear(h->trace);
    delete h->trace;
  }
  cudaFree(h->status);
  if (h->aux) cudaStreamDestroy(h->aux);
  delete h;
  return PS_OK;
}

ps_status ps_check(ps_handle h, void* stream, int synchronize) {
  if (h == nullptr) return PS_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = synchronize ? cudaStreamSynchronize(s) : cudaSuccess;
  if (e != cudaSuccess) return launch_status(e);
  int word = 0;
  e = cudaMemcpyAsync(&word, h->status, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return launch_status(e);
  if (word != 0) {
    cudaMemsetAsync(h->status, 0, sizeof(int), s);
    cudaStreamSynchronize(s);
    return word == PS_ERR_TIMEOUT ? PS_ERR_TIMEOUT : PS_ERR_CUDA;
  }
  return PS_OK;
}

const char* ps_status_string(ps_status s) {
  switch (s) {
    case PS_OK: return "ok";
    case PS_ERR_ARG: return "invalid argument";
    case PS_ERR_UNSUPPORTED: return "unsupported device (needs sm_103)";
    case PS_ERR_WORKSPACE: return "workspace too small";
    case PS_ERR_CUDA: return "CUDA error";
    case PS_ERR_TIMEOUT: return "device-side wait timed out";
  }
  return "unknown status";
}

const char* ps_last_cuda_error(void) { return g_last_cuda_error; }

ps_status ps_trace_enable(ps_handle h, int enable) {
  if (h == nullptr) return PS_ERR_ARG;
  if (h->trace != nullptr) {
    trace_clear(h->trace);
    delete h->trace;
    h->trace = nullptr;
  }
  if (enable) {
    h->trace = new (std::nothrow) TraceSink;
    if (h->trace == nullptr) return PS_ERR_CUDA;
  }
  return PS_OK;
}

int ps_trace_count(ps_handle h) {
  return h != nullptr && h->trace != nullptr ? static_cast<int>(h->trace->recs.size()) : 0;
}

ps_status ps_trace_get(ps_handle h, int i, const char** name, float* ms) {
  if (h == nullptr || h->trace == nullptr || name == nullptr || ms == nullptr || i < 0 ||
      i >= static_cast<int>(h->trace->recs.size()))
    return PS_ERR_ARG;
  const TraceRec& r = h->trace->recs[i];
  cudaError_t e = cudaEventSynchronize(r.b);
  if (e == cudaSuccess) e = cudaEventElapsedTime(ms, r.a, r.b);
  if (e == cudaSuccess) e = cudaFuncGetName(name, r.kernel);
  return launch_status(e);
}

size_t ps_workspace_bytes(int op, int B, int N, int d, int C, int Hq, int Hkv,
                          int dh, int k, int P, int V) {
  if (B <= 0) return 0;
  switch (op) {
    case PS_OP_KMEANS: return (N > 0 && C > 0) ? kmeans_ws(B, N, d, C) : 0;
    case PS_OP_NVFP4: return (N > 0 && d > 0) ? nvfp4_ws(B, N, d) : 0;
    case PS_OP_PROXY_KL:
      return (N > 0 && C > 0 && Hkv > 0 && dh > 0 && Hq > 0)
                 ? proxy_ws(B, N, d, C, Hq, Hkv, dh) : 0;
    case PS_OP_TOPK: return 0;
    case PS_OP_REFRESH:
      return (N > 0 && d > 0 && Hkv > 0 && dh > 0) ? refresh_ws(B, N, d, Hkv, dh) : 0;
    case PS_OP_COMMIT: return (P > 0 && V > 0) ? commit_ws(B, P, V) : 0;
    case PS_OP_KV4_ATTN:
    case PS_OP_KV4_WEIGHT:
      if (N <= 0 || N > kMaxSlots || Hkv <= 0 || Hq < Hkv || Hq % Hkv != 0 || P <= 0 ||
          !kv4_dh_ok(dh) || !kv4_rows_ok(B, P, Hq))
        return 0;
      return op == PS_OP_KV4_ATTN ? kv4_attn_ws(B, N, Hq, Hkv, dh, P)
                                  : kv4_weight_ws(B, N, Hq, Hkv, dh, P);
    case PS_OP_ATTN:
      return attn_sizes_ok(B, N, Hq, Hkv, dh, P, k) ? attn_ws(B, N, Hq, Hkv, dh, P, k) : 0;
    case PS_OP_KV4_EVICT: return (Hkv > 0 && k > 0) ? kv4_evict_ws(B, Hkv, k) : 0;
  }
  return 0;
}

ps_status ps_kmeans_spherical(ps_handle h, const void* H, int dtype, int B,
                              int N, int d, int C, int iters, int init_mode,
                              const double* init_u, float* mu, int32_t* assign,
                              float* rho, float* chat, int32_t* counts,
                              float* objective, void* ws, size_t ws_bytes,
                              void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && dtype_ok(dtype));
  PS_REQUIRE(B >= 0 && iters >= 0 && (init_mode == 0 || init_mode == 1));
  if (B == 0) return PS_OK;
  PS_REQUIRE(d > 0 && d % 16 == 0 && d <= kMaxD);
  PS_REQUIRE(C >= 1 && C <= kMaxC && C <= N);
  PS_REQUIRE((long)B * N <= (long)INT32_MAX / 2);
  PS_PTR(H); PS_PTR(mu); PS_NN(assign); PS_NN(rho); PS_PTR(chat); PS_NN(counts);
  if (init_mode == 1) PS_NN(init_u);
  PS_REQUIRE(B <= 65535);
  ps_status st = check_ws(kmeans_ws(B, N, d, C), ws, ws_bytes);
  if (st != PS_OK) return st;
  KmeansArgs a{H, dtype, B, N, d, C, iters, init_mode, init_u, mu, assign, rho,
               chat, counts, objective, ws, h->status, h->num_sms, h->aux};
  return launch_status(kmeans_run(a, static_cast<cudaStream_t>(stream)));
}

ps_status ps_nvfp4_residual(ps_handle h, const void* H, int dtype,
                            const float* mu, const int32_t* assign,
                            const float* rho, int B, int N, int d, int C,
                            uint8_t* codes, uint8_t* scales,
                            float* tensor_scale, void* ws, size_t ws_bytes,
                            void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && dtype_ok(dtype));
  PS_REQUIRE(B >= 0);
  if (B == 0) return PS_OK;
  PS_REQUIRE(N >= 1 && d > 0 && d % 16 == 0 && B <= 65535);
  PS_PTR(H); PS_PTR(codes); PS_NN(scales); PS_NN(tensor_scale);
  if (mu != nullptr) {
    PS_PTR(mu); PS_NN(assign); PS_NN(rho);
    PS_REQUIRE(C >= 1);
  } else {
    PS_REQUIRE(dtype == PS_F32 || dtype == PS_BF16);
    C = 1;
  }
  ps_status st = check_ws(nvfp4_ws(B, N, d), ws, ws_bytes);
  if (st != PS_OK) return st;
  Nvfp4Args a{H, dtype, mu, assign, rho, B, N, d, C, codes, scales, tensor_scale,
              ws, h->num_sms};
  return launch_status(nvfp4_run(a, static_cast<cudaStream_t>(stream)));
}

ps_status ps_proxy_attn_kl(ps_handle h, const void* Q, const float* chat,
                           const void* Wk, int dtype, int B, int N, int d,
                           int C, int Hq, int Hkv, int dh, const float* A_prev,
                           float* A_cur, float* D, void* ws, size_t ws_bytes,
                           void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && dtype_ok(dtype));
  PS_REQUIRE(B >= 0);
  if (B == 0) return PS_OK;
  PS_REQUIRE(N >= 1 && d > 0 && d % 16 == 0 && B <= 65535);
  PS_REQUIRE(C >= 1 && C <= kMaxC);
  PS_REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0);
  PS_REQUIRE(dh > 0 && dh % 16 == 0 && dh <= kMaxDh);
  PS_PTR(Q); PS_PTR(chat); PS_PTR(Wk); PS_NN(A_cur); PS_NN(D);
  ps_status st = check_ws(proxy_ws(B, N, d, C, Hq, Hkv, dh), ws, ws_bytes);
  if (st != PS_OK) return st;
  ProxyArgs a{Q, chat, Wk, dtype, B, N, d, C, Hq, Hkv, dh, A_prev, A_cur, D, ws,
              h->num_sms, h->status};
  return launch_status(proxy_run(a, static_cast<cudaStream_t>(stream)));
}

ps_status ps_topk_drift(ps_handle h, const float* D, const int32_t* assign,
                        const int32_t* counts, int B, int N, int C, int k,
                        int32_t* sel, float* sel_score, int32_t* pos,
                        int32_t* npos, uint8_t* posmask, void* ws,
                        size_t ws_bytes, void* stream) {
  TraceScope trace_scope(h);
  (void)ws; (void)ws_bytes;
  PS_REQUIRE(h != nullptr && B >= 0);
  if (B == 0) return PS_OK;
  PS_REQUIRE(N >= 1 && C >= 1 && C <= kMaxC && C <= N && k >= 1 && k <= C);
  PS_REQUIRE(B <= 65535);
  PS_NN(D); PS_NN(assign); PS_NN(counts); PS_NN(sel); PS_NN(sel_score);
  PS_NN(pos); PS_NN(npos);
  TopkArgs a{D, assign, counts, B, N, C, k, sel, sel_score, pos, npos, posmask};
  return launch_status(topk_run(a, static_cast<cudaStream_t>(stream)));
}

ps_status ps_drift_score(ps_handle h, const float* A_cur, const float* A_prev, int B, int N,
                         int C, int scorer, float* D, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && B >= 0);
  if (B == 0) return PS_OK;
  PS_REQUIRE(N >= 1 && C >= 1 && C <= 4096 && (long)B * N <= 2147483647L);
  PS_REQUIRE(scorer >= PS_SCORER_KL && scorer <= PS_SCORER_ENTROPY);
  PS_NN(A_cur); PS_NN(D);
  PS_REQUIRE(D != A_cur && D != A_prev);
  return launch_status(drift_score_run(A_cur, A_prev, B, N, C, scorer, D,
                                       static_cast<cudaStream_t>(stream)));
}

ps_status ps_refresh_kv(ps_handle h, const void* H, int dtype,
                        const int32_t* pos, const int32_t* npos,
                        const void* Wk, const void* Wv, int B, int N, int d,
                        int Hkv, int dh, void* Kcache, void* Vcache,
                        int Ncache, int cache_off, void* ws, size_t ws_bytes,
                        void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && dtype_ok(dtype) && B >= 0);
  if (B == 0) return PS_OK;
  PS_REQUIRE(N >= 1 && d > 0 && d % 16 == 0 && Hkv >= 1 && dh > 0 && dh % 16 == 0);
  PS_REQUIRE(cache_off >= 0 && (long)cache_off + N <= Ncache && B <= 65535);
  PS_REQUIRE(2L * ceil_div((long)Hkv * dh, 64) <= 65535);
  PS_PTR(H); PS_NN(pos); PS_NN(npos); PS_PTR(Wk); PS_PTR(Wv);
  PS_NN(Kcache); PS_NN(Vcache);
  const bool tc = refresh_tc_ok(dtype, Hkv, dh);
  if (tc) {
    PS_PTR(Kcache); PS_PTR(Vcache);
    ps_status st = check_ws(refresh_ws(B, N, d, Hkv, dh), ws, ws_bytes);
    if (st != PS_OK) return st;
  }
  RefreshArgs a{H, dtype, pos, npos, Wk, Wv, B, N, d, Hkv, dh, Kcache, Vcache,
                Ncache, cache_off, h->num_sms, tc ? ws : nullptr, h->status};
  return launch_status(refresh_run(a, static_cast<cudaStream_t>(stream)));
}

ps_status ps_commit(ps_handle h, const void* logits, int dtype, int B, int P, int V,
                    const uint8_t* role, uint8_t* undecided,
                    const float* D_blk, int d_ld, float* d_sum, int32_t* d_cnt,
                    float* d_prev, const uint8_t* suffix_sel, int sel_ld,
                    ps_commit_params params, int32_t* token, float* conf,
                    uint8_t* commit, void* ws, size_t ws_bytes, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && dtype_ok(dtype) && B >= 0 && P >= 0);
  if (B == 0 || P == 0) return PS_OK;
  PS_REQUIRE(P <= 1024 && V >= 4 && V % 4 == 0 && (long)B * P <= 65535);
  PS_REQUIRE(d_ld >= P && (suffix_sel == nullptr || sel_ld >= P));
  PS_REQUIRE(params.mode >= 0 && params.mode <= 2);
  PS_REQUIRE(params.ensure_progress == 0 || params.ensure_progress == 1);
  PS_PTR(logits); PS_NN(role); PS_NN(undecided); PS_NN(D_blk); PS_NN(d_sum);
  PS_NN(d_cnt); PS_NN(d_prev); PS_NN(token); PS_NN(conf); PS_NN(commit);
  ps_status st = check_ws(commit_ws(B, P, V), ws, ws_bytes);
  if (st != PS_OK) return st;
  CommitArgs a{logits, dtype, B, P, V, role, undecided, D_blk, d_ld, d_sum, d_cnt, d_prev,
               suffix_sel, sel_ld, params, token, conf, commit, ws};
  return launch_status(commit_run(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

// The same NVFP4 residual quantisation as ps_nvfp4_residual, for callers
// that cannot allocate device memory: no workspace argument, scratch in a
// fixed 64 KiB device array inside the library.  See include/polestar.h.
extern "C" ps_status ps_nvfp4_residual_noalloc(
    ps_handle h, const void* H, int dtype, const float* mu, const int32_t* assign,
    const float* rho, int B, int N, int d, int C, uint8_t* codes, uint8_t* scales,
    float* tensor_scale, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && dtype_ok(dtype));
  PS_REQUIRE(B >= 0);
  if (B == 0) return PS_OK;
  PS_REQUIRE(N >= 1 && d > 0 && d % 16 == 0 && B <= 65535);
  PS_PTR(H); PS_PTR(codes); PS_NN(scales); PS_NN(tensor_scale);
  if (mu != nullptr) {
    PS_PTR(mu); PS_NN(assign); PS_NN(rho);
    PS_REQUIRE(C >= 1);
  } else {
    C = 1;
  }
  if (!nvfp4_static_fits(B, N, d)) return PS_ERR_WORKSPACE;
  // the array's address is per device: the kernels must run on the device
  // whose address is used, so the caller's current device must be the
  // handle's
  int cur = -1;
  cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return launch_status(e);
  if (cur != h->device) return PS_ERR_ARG;
  float* scratch = nullptr;
  e = nvfp4_static_scratch(h->device, &scratch);
  if (e != cudaSuccess) return launch_status(e);
  Nvfp4Args a{H, dtype, mu, assign, rho, B, N, d, C, codes, scales, tensor_scale,
              scratch, h->num_sms};
  return launch_status(nvfp4_run(a, static_cast<cudaStream_t>(stream)));
}

// ---- offload of the quantised clusters; see include/polestar.h
namespace {
// device memory, or host memory mapped into this device's address space
bool device_accessible(const void* p) {
  cudaPointerAttributes at{};
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged ||
         (at.type == cudaMemoryTypeHost && at.devicePointer == p);
}
}  // namespace

extern "C" ps_status ps_block_progress(ps_handle h, const uint8_t* commit,
                                       const uint8_t* undecided, const uint8_t* role, int B,
                                       int P, int32_t* out, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && B >= 0 && P >= 0);
  PS_NN(out);
  PS_REQUIRE((reinterpret_cast<uintptr_t>(out) & 7u) == 0);
  PS_REQUIRE(device_accessible(out));
  if (B > 0 && P > 0) {
    PS_REQUIRE((long)B * P <= INT32_MAX);
    PS_NN(commit); PS_NN(undecided); PS_NN(role);
  }
  return launch_status(block_progress_run(commit, undecided, role, B, P, out,
                                          static_cast<cudaStream_t>(stream)));
}

extern "C" size_t ps_store_record_bytes(int d) {
  return d > 0 && d % 32 == 0 ? ps::store_record_bytes(d) : 0;
}

extern "C" ps_status ps_host_alloc(size_t bytes, void** ptr) {
  if (ptr == nullptr || bytes == 0) return PS_ERR_ARG;
  *ptr = nullptr;
  void* p = nullptr;
  cudaError_t e = cudaHostAlloc(&p, bytes, cudaHostAllocMapped | cudaHostAllocPortable);
  if (e != cudaSuccess) return launch_status(e);
  void* dp = nullptr;
  e = cudaHostGetDevicePointer(&dp, p, 0);
  if (e != cudaSuccess || dp != p) {  // one address for host and device (unified addressing)
    cudaFreeHost(p);
    return e != cudaSuccess ? launch_status(e) : PS_ERR_CUDA;
  }
  *ptr = p;
  return PS_OK;
}

extern "C" ps_status ps_host_free(void* ptr) {
  if (ptr == nullptr) return PS_OK;
  return launch_status(cudaFreeHost(ptr));
}

extern "C" ps_status ps_nvfp4_pack_clusters(ps_handle h, const uint8_t* codes,
                                            const uint8_t* scales, const int32_t* assign, int B,
                                            int N, int d, int C, void* store, int32_t* order,
                                            int32_t* cl_off, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && B >= 0);
  if (B == 0) return PS_OK;
  PS_REQUIRE(N >= 1 && N <= 16384 && d > 0 && d % 32 == 0 && C >= 1 && C <= 65535 &&
             B <= 65535);
  PS_PTR(codes); PS_NN(scales); PS_NN(assign); PS_PTR(store); PS_NN(order); PS_NN(cl_off);
  PS_REQUIRE(device_accessible(store));
  return launch_status(pack_clusters_run(codes, scales, assign, B, N, d, C,
                                         static_cast<uint8_t*>(store), order, cl_off,
                                         static_cast<cudaStream_t>(stream)));
}

extern "C" ps_status ps_nvfp4_fetch_dequant(ps_handle h, const void* store, const int32_t* order,
                                            const int32_t* cl_off, const int32_t* sel, int k,
                                            const float* mu, const float* rho,
                                            const float* tensor_scale, int B, int N, int d, int C,
                                            void* Ht, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && B >= 0);
  if (B == 0 || k == 0) return PS_OK;
  PS_REQUIRE(N >= 1 && N <= 65535 && d > 0 && d % 32 == 0 && C >= 1 && k >= 1 && k <= C &&
             B <= 65535);
  PS_PTR(store); PS_NN(order); PS_NN(cl_off); PS_NN(sel); PS_PTR(mu); PS_NN(rho);
  PS_NN(tensor_scale); PS_PTR(Ht);
  PS_REQUIRE(device_accessible(store));
  return launch_status(fetch_dequant_run(static_cast<const uint8_t*>(store), order, cl_off, sel,
                                         k, mu, rho, tensor_scale, B, N, d, C,
                                         static_cast<__nv_bfloat16*>(Ht),
                                         static_cast<cudaStream_t>(stream)));
}

// ---- the 4-bit KV cache; see include/polestar.h
namespace {

// The shape, pointers and tensor scales of a cache.
ps_status check_kv4(const ps_kv4_cache* c) {
  PS_REQUIRE(c != nullptr && c->B >= 0 && c->Hkv >= 1 && c->Hkv <= 512 && c->Ncache >= 1 &&
             c->Ncache <= kMaxSlots && kv4_dh_ok(c->dh));
  PS_REQUIRE(c->B <= 65535 && (long)c->B * c->Hkv <= 65535);
  PS_REQUIRE(std::isnormal(c->kmul) && c->kmul > 0.f && std::isnormal(c->vmul) && c->vmul > 0.f);
  if (c->B > 0) {
    PS_PTR(c->kcode); PS_PTR(c->kscale); PS_PTR(c->vcode); PS_PTR(c->vscale);
  }
  return PS_OK;
}

bool ld_ok(int64_t ld, long least, int dtype) {
  return ld >= least && ld % (dtype == PS_F32 ? 4 : 8) == 0;
}

ps_status kv4_rows(ps_handle h, const ps_kv4_cache* c, const void* K, const void* V, int dtype,
                   int R, int64_t b_ld, int64_t ld, const int32_t* off, const int32_t* rows,
                   const int32_t* cnt, const int32_t* kpos, bool load, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && dtype_ok(dtype) && R >= 0);
  ps_status st = check_kv4(c);
  if (st != PS_OK) return st;
  if (c->B == 0 || R == 0) return PS_OK;
  PS_REQUIRE(ld_ok(ld, (long)c->Hkv * c->dh, dtype) && ld_ok(b_ld, 0, dtype));
  PS_REQUIRE((long)R * c->Hkv <= (1 << 30));
  PS_REQUIRE(!load || c->B == 1 || b_ld > 0);  // sequences read back over one another
  PS_PTR(K); PS_PTR(V);
  Kv4RowsArgs a{K, V, dtype, c->B, R, c->Hkv, c->Ncache, c->dh, (long)b_ld, (long)ld, off, rows,
                cnt, kpos, c->kcode, c->kscale, c->vcode, c->vscale, c->kmul, c->vmul, {}};
  return launch_status(kv4_rows_run(a, load, static_cast<cudaStream_t>(stream)));
}

// Checks a cache and a query and lays out the kernels' arguments; *none is set
// where there is nothing to do.
ps_status kv4_query(ps_handle h, const ps_kv4_cache* c, const ps_kv4_query* q, Kv4AttnArgs* a,
                    bool* none) {
  PS_REQUIRE(h != nullptr && q != nullptr && dtype_ok(q->dtype) && q->T >= 0);
  ps_status st = check_kv4(c);
  if (st != PS_OK) return st;
  PS_REQUIRE(q->Hq >= c->Hkv && q->Hq % c->Hkv == 0);
  PS_REQUIRE(std::isfinite(q->scale) && std::isfinite(q->cap) && q->cap >= 0.f);
  PS_REQUIRE((q->slope == nullptr) || (q->qpos != nullptr));
  *none = c->B == 0 || q->T == 0;
  if (*none) return PS_OK;
  PS_REQUIRE(kv4_rows_ok(c->B, q->T, q->Hq) && q->Hq / c->Hkv <= 4096);
  PS_REQUIRE(ld_ok(q->q_ld, (long)q->Hq * c->dh, q->dtype) && ld_ok(q->q_bld, 0, q->dtype));
  PS_PTR(q->Q);
  *a = Kv4AttnArgs{};
  a->kcode = c->kcode; a->kscale = c->kscale; a->vcode = c->vcode; a->vscale = c->vscale;
  a->Q = q->Q; a->dtype = q->dtype;
  a->B = c->B; a->T = q->T; a->Hq = q->Hq; a->Hkv = c->Hkv;
  a->G = q->Hq / c->Hkv; a->M = q->T * a->G;
  a->by_g = row_quotient(a->G);
  a->Ncache = c->Ncache; a->dh = c->dh;
  a->q_bld = (long)q->q_bld; a->q_ld = (long)q->q_ld;
  a->len = q->len; a->span = q->span; a->kpos = q->kpos; a->qpos = q->qpos; a->slope = q->slope;
  a->scale = q->scale * c->kmul; a->vmul = c->vmul;
  // within [1e-18, 1e30], past which a cap leaves nothing of fp32 scores, or all
  // of those below 1e26: score / cap stays in range
  a->cap = q->cap > 0.f ? std::fmin(std::fmax(q->cap, 1e-18f), 1e30f) : 0.f;
  a->inv_cap = q->cap > 0.f ? 1.f / a->cap : 0.f;
  a->num_sms = h->num_sms; a->status = h->status;
  return PS_OK;
}

}  // namespace

extern "C" ps_status ps_kv4_store(ps_handle h, const ps_kv4_cache* c, const void* K,
                                  const void* V, int dtype, int R, int64_t b_ld, int64_t ld,
                                  const int32_t* off, const int32_t* rows, const int32_t* cnt,
                                  void* stream) {
  return kv4_rows(h, c, K, V, dtype, R, b_ld, ld, off, rows, cnt, nullptr, false, stream);
}

extern "C" ps_status ps_kv4_store_pos(ps_handle h, const ps_kv4_cache* c, const void* K,
                                      const void* V, int dtype, int R, int64_t b_ld, int64_t ld,
                                      const int32_t* off, const int32_t* rows, const int32_t* cnt,
                                      const int32_t* kpos, void* stream) {
  return kv4_rows(h, c, K, V, dtype, R, b_ld, ld, off, rows, cnt, kpos, false, stream);
}

extern "C" ps_status ps_kv4_load(ps_handle h, const ps_kv4_cache* c, void* K, void* V, int dtype,
                                 int R, int64_t b_ld, int64_t ld, const int32_t* off,
                                 const int32_t* rows, const int32_t* cnt, void* stream) {
  return kv4_rows(h, c, K, V, dtype, R, b_ld, ld, off, rows, cnt, nullptr, true, stream);
}

extern "C" ps_status ps_kv4_attn(ps_handle h, const ps_kv4_cache* c, const ps_kv4_query* q,
                                 void* O, float* lse, void* ws, size_t ws_bytes, void* stream) {
  TraceScope trace_scope(h);
  Kv4AttnArgs a;
  bool none;
  ps_status st = kv4_query(h, c, q, &a, &none);
  if (st != PS_OK || none) return st;
  PS_PTR(O);
  st = check_ws(kv4_attn_ws(a.B, a.Ncache, a.Hq, a.Hkv, a.dh, a.T), ws, ws_bytes);
  if (st != PS_OK) return st;
  a.O = O; a.lse = lse; a.ws = ws;
  return launch_status(kv4_attn_run(a, static_cast<cudaStream_t>(stream)));
}

extern "C" ps_status ps_kv4_weight(ps_handle h, const ps_kv4_cache* c, const ps_kv4_query* q,
                                   const float* lse, const float* w_in, float* w_out, void* ws,
                                   size_t ws_bytes, void* stream) {
  TraceScope trace_scope(h);
  Kv4AttnArgs a;
  bool none;
  ps_status st = kv4_query(h, c, q, &a, &none);
  if (st != PS_OK || none) return st;
  PS_NN(lse); PS_NN(w_out);
  st = check_ws(kv4_weight_ws(a.B, a.Ncache, a.Hq, a.Hkv, a.dh, a.T), ws, ws_bytes);
  if (st != PS_OK) return st;
  a.lse_in = lse; a.w_in = w_in; a.w_out = w_out; a.ws = ws;
  return launch_status(kv4_weight_run(a, static_cast<cudaStream_t>(stream)));
}

namespace {

// `on`: ps_kv4_evict_on's part too.
ps_status kv4_evict(ps_handle h, const ps_kv4_cache* src, const ps_kv4_cache* dst, const float* w,
                    const int32_t* len, const int32_t* kpos, int keep, int sink, int recent,
                    float* w_dst, int32_t* kpos_dst, int32_t* len_dst, bool on,
                    const int32_t* shift, int32_t* shift_dst, void* ws, size_t ws_bytes,
                    void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr);
  ps_status st = check_kv4(src);
  if (st == PS_OK) st = check_kv4(dst);
  if (st != PS_OK) return st;
  PS_REQUIRE(src->B == dst->B && src->Hkv == dst->Hkv && src->dh == dst->dh &&
             src->kmul == dst->kmul && src->vmul == dst->vmul);
  PS_REQUIRE(keep >= 1 && sink >= 0 && recent >= 0 && (long)sink + recent <= keep &&
             keep <= dst->Ncache);
  if (src->B == 0) return PS_OK;
  PS_NN(w); PS_NN(w_dst); PS_NN(len_dst);
  PS_REQUIRE(w != w_dst && (kpos == nullptr || kpos != kpos_dst) && len != len_dst);
  PS_REQUIRE(!on || (kpos_dst != nullptr && shift_dst != nullptr && shift != shift_dst));
  PS_REQUIRE(src->kcode != dst->kcode && src->vcode != dst->vcode &&
             src->kscale != dst->kscale && src->vscale != dst->vscale);
  st = check_ws(kv4_evict_ws(src->B, src->Hkv, keep), ws, ws_bytes);
  if (st != PS_OK) return st;
  Kv4EvictArgs a{src->kcode, src->kscale, src->vcode, src->vscale,
                 dst->kcode, dst->kscale, dst->vcode, dst->vscale,
                 src->B, src->Hkv, src->Ncache, dst->Ncache, src->dh, keep, sink, recent,
                 w, len, kpos, w_dst, kpos_dst, len_dst, on ? shift : nullptr,
                 on ? shift_dst : nullptr, ws};
  return launch_status(kv4_evict_run(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" ps_status ps_kv4_evict(ps_handle h, const ps_kv4_cache* src, const ps_kv4_cache* dst,
                                  const float* w, const int32_t* len, const int32_t* kpos,
                                  int keep, int sink, int recent, float* w_dst,
                                  int32_t* kpos_dst, int32_t* len_dst, void* ws,
                                  size_t ws_bytes, void* stream) {
  return kv4_evict(h, src, dst, w, len, kpos, keep, sink, recent, w_dst, kpos_dst, len_dst, false,
                   nullptr, nullptr, ws, ws_bytes, stream);
}

extern "C" ps_status ps_kv4_evict_on(ps_handle h, const ps_kv4_cache* src,
                                     const ps_kv4_cache* dst, const float* w, const int32_t* len,
                                     const int32_t* kpos, int keep, int sink, int recent,
                                     float* w_dst, int32_t* kpos_dst, int32_t* len_dst,
                                     const int32_t* shift, int32_t* shift_dst, void* ws,
                                     size_t ws_bytes, void* stream) {
  return kv4_evict(h, src, dst, w, len, kpos, keep, sink, recent, w_dst, kpos_dst, len_dst, true,
                   shift, shift_dst, ws, ws_bytes, stream);
}

// ---- rotary positions, drawn tokens

namespace {

// Makes the handle's device current for a call (a caller may have another one).
struct DeviceScope {
  int before = -1;
  cudaError_t err;
  explicit DeviceScope(int device) {
    int now = -1;
    err = cudaGetDevice(&now);
    if (err == cudaSuccess && now != device) {
      err = cudaSetDevice(device);
      if (err == cudaSuccess) before = now;
    }
  }
  ~DeviceScope() {
    if (before >= 0) cudaSetDevice(before);
  }
};

}  // namespace

extern "C" ps_status ps_rope(ps_handle h, const ps_rope_rows* r, const ps_rope_part* parts,
                             int nparts, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && r != nullptr && parts != nullptr && nparts >= 1 && nparts <= 3);
  PS_REQUIRE(dtype_ok(r->dtype) && r->B >= 0 && r->T >= 0 && (r->pairs == 0 || r->pairs == 1));
  PS_REQUIRE(r->dh > 0 && r->dh % 16 == 0 && r->dh <= kMaxDh);
  PS_REQUIRE(r->rot >= 2 && r->rot % 2 == 0 && r->rot <= r->dh && std::isfinite(r->amp));
  if (r->B == 0 || r->T == 0) return PS_OK;
  PS_REQUIRE((long)r->B * r->T <= INT32_MAX);
  PS_REQUIRE(r->turns != nullptr && (reinterpret_cast<uintptr_t>(r->turns) & 7u) == 0);
  RopeArgs a{r->turns, r->pos, r->off, r->rows, r->cnt, r->dst, r->B, r->T, r->dh, r->rot,
             r->pairs != 0, r->dtype, r->amp, {}, {}};
  int heads = 0;
  for (int i = 0; i < 3; ++i) {
    if (i < nparts) {
      const ps_rope_part& p = parts[i];
      PS_REQUIRE(p.H >= 1 && p.H <= 4096 && p.slots >= 0 && (p.rotate == 0 || p.rotate == 1));
      PS_PTR(p.X); PS_PTR(p.Y);
      PS_REQUIRE(ld_ok(p.x_ld, (long)p.H * r->dh, r->dtype) && ld_ok(p.x_bld, 0, r->dtype));
      PS_REQUIRE(ld_ok(p.y_ld, (long)p.H * r->dh, r->dtype) && ld_ok(p.y_bld, 0, r->dtype));
      PS_REQUIRE(r->B == 1 || p.y_bld > 0);  // sequences written over one another
      if (p.X == p.Y)
        PS_REQUIRE(p.slots == 0 && p.x_ld == p.y_ld && (r->B == 1 || p.x_bld == p.y_bld));
      a.part[i] = RopePart{p.X, p.Y, (long)p.x_bld, (long)p.x_ld, (long)p.y_bld, (long)p.y_ld,
                           p.slots, p.rotate};
      heads += p.H;
    }
    a.end[i] = heads;
  }
  DeviceScope dev(h->device);
  if (dev.err != cudaSuccess) return launch_status(dev.err);
  return launch_status(rope_run(a, static_cast<cudaStream_t>(stream)));
}

extern "C" ps_status ps_attn(ps_handle h, const ps_attn_rows* q, void* O, float* lse, void* ws,
                             size_t ws_bytes, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && q != nullptr && dtype_ok(q->dtype));
  PS_REQUIRE(attn_sizes_ok(q->S, q->max_k, q->Hq, q->Hkv, q->dh, q->Tq, q->max_q));
  PS_REQUIRE(q->Tk >= 0 && q->Tk <= kMaxSlots && (q->causal == 0 || q->causal == 1) &&
             std::isfinite(q->scale));
  if (q->S == 0 || q->Tq == 0) return PS_OK;
  PS_PTR(q->Q); PS_PTR(O); PS_NN(q->q_off); PS_NN(q->k_off);
  if (q->Tk > 0) {
    PS_PTR(q->K); PS_PTR(q->V);
  }
  PS_REQUIRE(ld_ok(q->q_ld, (long)q->Hq * q->dh, q->dtype) &&
             ld_ok(q->o_ld, (long)q->Hq * q->dh, q->dtype) &&
             ld_ok(q->k_ld, (long)q->Hkv * q->dh, q->dtype) &&
             ld_ok(q->v_ld, (long)q->Hkv * q->dh, q->dtype));
  PS_REQUIRE(O != q->Q && O != q->K && O != q->V);
  ps_status st = check_ws(attn_ws(q->S, q->max_k, q->Hq, q->Hkv, q->dh, q->Tq, q->max_q), ws,
                          ws_bytes);
  if (st != PS_OK) return st;
  AttnArgs a{};
  a.Q = q->Q; a.K = q->K; a.V = q->V;
  a.q_ld = (long)q->q_ld; a.k_ld = (long)q->k_ld; a.v_ld = (long)q->v_ld; a.o_ld = (long)q->o_ld;
  a.q_off = q->q_off; a.k_off = q->k_off; a.k_len = q->k_len; a.span = q->span;
  a.dtype = q->dtype; a.S = q->S; a.Tq = q->Tq; a.Tk = q->Tk;
  a.Hq = q->Hq; a.Hkv = q->Hkv; a.G = q->Hq / q->Hkv; a.dh = q->dh;
  a.causal = q->causal != 0; a.max_q = q->max_q; a.max_k = q->max_k; a.scale = q->scale;
  a.O = O; a.lse = lse; a.ws = ws; a.status = h->status;
  DeviceScope dev(h->device);
  if (dev.err != cudaSuccess) return launch_status(dev.err);
  return launch_status(attn_run(a, static_cast<cudaStream_t>(stream)));
}

extern "C" ps_status ps_sample(ps_handle h, const ps_sample_rows* s, int32_t* token, float* prob,
                               int32_t* n, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && s != nullptr && dtype_ok(s->dtype) && s->R >= 0);
  PS_REQUIRE(s->V >= 1 && s->V <= 1000000 && s->R <= (1 << 27));
  if (s->R == 0) return PS_OK;
  const uintptr_t esz = s->dtype == PS_F32 ? 4 : 2;
  PS_NN(s->logits); PS_NN(s->u); PS_NN(token);
  PS_REQUIRE(reinterpret_cast<uintptr_t>(s->logits) % esz == 0 &&
             reinterpret_cast<uintptr_t>(s->u) % 8 == 0);
  PS_REQUIRE(s->ld >= s->V && s->ld <= INT64_MAX / 8 / s->R);
  SampleArgs a{s->logits, s->u, s->temperature, s->top_k, s->top_p, s->min_p, (long)s->ld,
               s->dtype, s->R, s->V, token, prob, n, 0, 0, false};
  DeviceScope dev(h->device);
  if (dev.err != cudaSuccess) return launch_status(dev.err);
  return launch_status(sample_run(a, static_cast<cudaStream_t>(stream)));
}

extern "C" ps_status ps_commit_drawn(ps_handle h, const float* conf, int B, int P,
                                     const uint8_t* role, uint8_t* undecided, const float* D_blk,
                                     int d_ld, float* d_sum, int32_t* d_cnt, float* d_prev,
                                     const uint8_t* suffix_sel, int sel_ld,
                                     ps_commit_params params, uint8_t* commit, void* stream) {
  TraceScope trace_scope(h);
  PS_REQUIRE(h != nullptr && B >= 0 && P >= 0);
  if (B == 0 || P == 0) return PS_OK;
  PS_REQUIRE(P <= 1024 && (long)B * P <= 65535);
  PS_REQUIRE(d_ld >= P && (suffix_sel == nullptr || sel_ld >= P));
  PS_REQUIRE(params.mode >= 0 && params.mode <= 2);
  PS_REQUIRE(params.ensure_progress == 0 || params.ensure_progress == 1);
  PS_NN(conf); PS_NN(role); PS_NN(undecided); PS_NN(D_blk); PS_NN(d_sum);
  PS_NN(d_cnt); PS_NN(d_prev); PS_NN(commit);
  CommitArgs a{nullptr, 0, B, P, 0, role, undecided, D_blk, d_ld, d_sum, d_cnt, d_prev,
               suffix_sel, sel_ld, params, nullptr, const_cast<float*>(conf), commit, nullptr};
  DeviceScope dev(h->device);
  if (dev.err != cudaSuccess) return launch_status(dev.err);
  return launch_status(commit_drawn_run(a, static_cast<cudaStream_t>(stream)));
}
