/*
 * libpolestar -- the per-step drift-scoring and sparse-refresh path of
 * Polestar-Cache / Polestar-Commit on one NVIDIA GB300 (sm_103a).
 *
 * Method source: "Polestar: Drift-Aware Cache Calibration and Token
 * Commitment for Efficient Inference of Diffusion LLMs" (gist.science
 * explainer of arXiv 2607.14107), technical summary, cited below as
 * [Polestar §x, <paragraph>].
 *
 * Conventions shared by every call
 * --------------------------------
 * Memory   Every array argument is a DEVICE pointer to caller-owned memory,
 *          row-major, contiguous, last index fastest, 16-byte aligned.
 *          The library allocates nothing inside an op: scratch comes from the
 *          caller's workspace `ws` of at least ps_workspace_bytes(op, ...)
 *          bytes (NULL is fine when that size is 0).  Outputs must not alias
 *          inputs unless the argument says "in/out".
 * Streams  `stream` is a cudaStream_t passed as void* (NULL = the legacy
 *          default stream).  Calls only enqueue work and return; the results
 *          are valid once the stream reaches that point.
 * Errors   Argument errors are detected on the host before anything is
 *          enqueued and return PS_ERR_ARG (nothing is launched, no output is
 *          touched).  A launch failure returns PS_ERR_CUDA.  A device-side
 *          failure (a bounded wait that gave up) sets the handle's status word;
 *          ps_check() reports it as PS_ERR_TIMEOUT.
 * Sizes    B >= 0 (B == 0 is a no-op), d % 16 == 0, dh % 16 == 0,
 *          Hq % Hkv == 0, 1 <= k <= C <= min(N, 256), d <= 8192,
 *          dh <= 256, V % 4 == 0, P <= 1024, B * P <= 65535.
 * Threads  One handle per concurrently used stream; no C++ exception
 *          crosses this interface.
 * State    Step-to-step state (centroids, previous distributions, drift
 *          history, undecided flags, the KV cache) lives in caller buffers.
 */
#ifndef POLESTAR_H
#define POLESTAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PS_OK = 0,
  PS_ERR_ARG = 1,          /* bad pointer, size, alignment or dtype       */
  PS_ERR_UNSUPPORTED = 2,  /* device is not sm_103                         */
  PS_ERR_WORKSPACE = 3,    /* ws smaller than ps_workspace_bytes()         */
  PS_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed         */
  PS_ERR_TIMEOUT = 5       /* a device-side bounded wait gave up           */
} ps_status;

typedef enum { PS_F32 = 0, PS_BF16 = 1 } ps_dtype;

typedef enum {
  PS_OP_KMEANS = 0, PS_OP_NVFP4 = 1, PS_OP_PROXY_KL = 2,
  PS_OP_TOPK = 3, PS_OP_REFRESH = 4, PS_OP_COMMIT = 5,
  PS_OP_KV4_ATTN = 6, PS_OP_KV4_WEIGHT = 7, PS_OP_KV4_EVICT = 8,
  PS_OP_ATTN = 9
} ps_op;

typedef struct ps_handle_s* ps_handle;

/* Create a handle on `device` (made current).  Allocates the handle's
 * 16-byte device status word -- the only allocation the library makes.
 * PS_ERR_UNSUPPORTED unless the device has compute capability 10.3. */
ps_status ps_create(int device, ps_handle* out);
ps_status ps_destroy(ps_handle h);

/* Status of device-side work enqueued so far on `stream`: reads the
 * handle's status word after the work on `stream` has finished (the read is
 * ordered on `stream` and waited for; synchronize != 0 additionally
 * synchronises the stream first and reports a failed synchronisation).
 * Clears the word.  Returns PS_OK, PS_ERR_TIMEOUT or PS_ERR_CUDA. */
ps_status ps_check(ps_handle h, void* stream, int synchronize);

const char* ps_status_string(ps_status s);

/* The CUDA runtime error behind the calling thread's most recent
 * PS_ERR_CUDA ("cudaErrorName: description"), or "" if there was none.  The
 * text lives in thread-local storage owned by the library and stays valid
 * until the thread's next call that fails with PS_ERR_CUDA. */
const char* ps_last_cuda_error(void);

/* Kernel trace, for diagnostics (no counterpart in the paper).  While it is
 * enabled on a handle, every kernel a ps_* call on that handle launches is
 * bracketed by two CUDA events on the call's stream, kept in host memory the
 * handle owns.  Enabling (enable != 0) or disabling discards earlier
 * records.  Not for calls made while the stream is captured into a CUDA
 * graph.  PS_ERR_ARG for a NULL handle. */
ps_status ps_trace_enable(ps_handle h, int enable);
/* Number of kernels recorded since tracing was enabled (0 when it is off). */
int ps_trace_count(ps_handle h);
/* Record i (0-based, in launch order): the kernel's name and its duration in
 * milliseconds; waits for the kernel to finish.  The name is owned by the
 * CUDA runtime and stays valid while the library is loaded.  PS_ERR_ARG for
 * an index out of range or NULL outputs, PS_ERR_CUDA if an event query
 * fails. */
ps_status ps_trace_get(ps_handle h, int i, const char** name, float* ms);

/* ---------------------------------------------------------------------------
 * Offload of the quantised clusters.
 * [Polestar §2.C, CPU offloading] -- "quantised hidden-state clusters are
 * offloaded to pinned CPU memory while only the centroids stay on the GPU;
 * the top-k clusters are fetched asynchronously".
 *
 * Store of a window: one record per row, grouped by cluster (ascending id)
 * and by ascending position inside a cluster.  A record holds the row's E2M1
 * codes (d/2 bytes) then its E4M3 block scales (d/16 bytes), each part
 * zero-padded to a multiple of 16 bytes: ps_store_record_bytes(d) bytes
 * (0 unless d is a positive multiple of 32).  Layout [B][N][record].
 *
 * ps_host_alloc: `bytes` of pinned host memory mapped into the device's
 * address space, one pointer valid on host and device (the GPU reaches it
 * over NVLink-C2C or PCIe).  PS_ERR_ARG for ptr == NULL or bytes == 0;
 * PS_ERR_CUDA if the allocation fails.  Release with ps_host_free.
 * ------------------------------------------------------------------------- */
size_t ps_store_record_bytes(int d);
ps_status ps_host_alloc(size_t bytes, void** ptr);
ps_status ps_host_free(void* ptr);

/* Writes the store of every window (the offload: the GPU stores straight
 * into it when it lies in host memory).
 * codes [B][N][d/2] u8, scales [B][N][d/16] u8, assign [B][N] i32 in [0, C)
 * (ps_nvfp4_residual's and ps_kmeans_spherical's outputs)
 * store [B][N][record] u8 out: device memory or ps_host_alloc memory,
 *       16-byte aligned
 * order [B][N] i32 out: position of record r;  cl_off [B][C+1] i32 out:
 *       first record of cluster c (cl_off[C] = rows with a label in [0, C))
 * PS_ERR_ARG for NULL or misaligned pointers, a store the device cannot
 * reach, N > 16384, or d not a multiple of 32. */
ps_status ps_nvfp4_pack_clusters(ps_handle h, const uint8_t* codes,
                                 const uint8_t* scales, const int32_t* assign,
                                 int B, int N, int d, int C, void* store,
                                 int32_t* order, int32_t* cl_off, void* stream);

/* Reads the records of the selected clusters from the store (the fetch) and
 * writes each row's reconstruction into Ht:
 *   g = fl(s_b S), deq = fl(v g), t = fl(rho_i mu_c), h~ = fl(t + deq)
 * (fp32, one rounding each, no fused multiply-add; v the element's E2M1
 * value, s_b its block's E4M3 value, S the window's tensor scale), rounded
 * to bf16 (nearest-even).  Rows of unselected clusters are left untouched,
 * so ps_refresh_kv can take Ht with the same pos / npos.
 * sel [B][k] i32 (ps_topk_drift's; entries < 0 ignored), mu [B][C][d] f32,
 * rho [B][N] f32, tensor_scale [B] f32, Ht [B][N][d] bf16 out.
 * PS_ERR_ARG as for ps_nvfp4_pack_clusters, or k outside [1, C]. */
ps_status ps_nvfp4_fetch_dequant(ps_handle h, const void* store,
                                 const int32_t* order, const int32_t* cl_off,
                                 const int32_t* sel, int k, const float* mu,
                                 const float* rho, const float* tensor_scale,
                                 int B, int N, int d, int C, void* Ht,
                                 void* stream);

/* Workspace bytes `op` needs for these sizes (arguments an op does not use
 * are ignored).  0 means ws may be NULL. */
size_t ps_workspace_bytes(int op, int B, int N, int d, int C, int Hq, int Hkv,
                          int dh, int k, int P, int V);

/* ---------------------------------------------------------------------------
 * a1  Spherical k-means of each window's hidden states.
 * [Polestar §2.A, local window & clustering] -- "clusters the hidden states
 * in the window with spherical k-means".
 *
 * H        [B][N][d]  f32 or bf16 (dtype)      hidden states of the window
 * mu       [B][C][d]  f32, in/out              centroids: input = warm start
 *          (init_mode 0, e.g. the previous step's result) or ignored
 *          (init_mode 1); output = final unit-norm centroids
 * init_u   [B][C]     f64 in [0,1)             k-means++ draws (init_mode 1;
 *          NULL for init_mode 0).  First centre = row floor(u0*N); centre r =
 *          first row whose running sum of w_i = 1 - max cos to the chosen
 *          centres exceeds u_r * sum(w).
 * iters    number of centroid updates I >= 0; I+1 assignment passes run.
 * assign   [B][N] i32 out  final cluster of each row (ties -> lower index)
 * rho      [B][N] f32 out  <h_i, mu_{assign_i}>
 * chat     [B][C][d] f32 in/out  mean(rho of members) * mu_c; clusters left
 *          empty keep the caller's values
 * counts   [B][C] i32 out  cluster sizes
 * objective[B][I+1] f32 out (nullable)  sum_i cos(h_i, mu_{a_i}) per pass;
 *          with the faster passes (bf16 windows, at least one 128-row tile per
 *          SM) the passes before the last sum their bf16-centroid scores, each
 *          within 2^-9 * N of the exact sum; the last pass's is exact up to
 *          fp32 rounding
 * Empty clusters keep their centroid.  Rows of zero norm join cluster 0.
 *
 * Two forms compute the same passes.  bf16 windows of N <= 1024 rows with
 * C <= 256, d <= 16384 and iters >= 2 run them on the window's cosine Gram
 * matrix (24-bit fixed point, exact integer cluster sums) inside one
 * thread-block cluster; a row whose two best cosines lie within about 1e-6
 * may take the other label than an fp64 pass would.  Other shapes, and any
 * call made while PS_KMEANS_LLOYD is set in the environment (read once per
 * process), form every centroid and assign on the tensor cores per pass.
 * ------------------------------------------------------------------------- */
ps_status ps_kmeans_spherical(ps_handle h, const void* H, int dtype, int B,
                              int N, int d, int C, int iters, int init_mode,
                              const double* init_u, float* mu, int32_t* assign,
                              float* rho, float* chat, int32_t* counts,
                              float* objective, void* ws, size_t ws_bytes,
                              void* stream);

/* ---------------------------------------------------------------------------
 * a2  NVFP4 quantisation of the k-means residuals.
 * [Polestar §2.A, local window & clustering] -- "quantises residuals with
 * NVFP4 to create compact proxy representations".
 *
 * r = fl(h - fl(rho_i * mu_{a_i}))  (fp32, two roundings); mu == NULL
 * quantises H itself (then assign/rho are ignored).
 * S_b = max(fl(amax_b / 2688), FLT_MIN) for 0 < amax_b < inf, else 1.
 * Block scale (16 elements along d): E4M3(fl(amax_blk / fl(6 S_b))), RNE,
 * saturating; element: E2M1(fl(r / fl(s_blk * S_b))), RNE, saturating, or
 * 0 when s_blk == 0.  Negative values rounding to zero keep their sign.
 *
 * codes  [B][N][d/2]  u8 out  element 2j in the low nibble of byte j
 * scales [B][N][d/16] u8 out  E4M3 block scales
 * tensor_scale [B]    f32 out S_b
 * Outputs are bit-exact functions of the inputs.
 * ------------------------------------------------------------------------- */
ps_status ps_nvfp4_residual(ps_handle h, const void* H, int dtype,
                            const float* mu, const int32_t* assign,
                            const float* rho, int B, int N, int d, int C,
                            uint8_t* codes, uint8_t* scales,
                            float* tensor_scale, void* ws, size_t ws_bytes,
                            void* stream);

/* ---------------------------------------------------------------------------
 * a3+a4  Proxy attention on centroid keys and the per-position KL drift.
 * [Polestar §2.A, sparse updates] -- proxy attention with cluster centroids;
 * [Polestar §2.A, drift measurement] -- D_i = KL(A_i^(t) || A_i^(t-1)).
 *
 * K~[b][c][g] = chat[b][c] . Wk[:, g*dh:(g+1)*dh]            (fp32)
 * s = q[b][i][h] . K~[b][c][h / (Hq/Hkv)] / sqrt(dh); p = softmax_c(s)
 * A_cur[b][i][c] = mean over the Hq heads of p
 * D[b][i] = max(0, sum_c A_cur (ln A_cur - ln max(A_prev, 1e-30))), terms
 *           with A_cur == 0 skipped; D = 0 when A_prev == NULL.
 *
 * Q      [B][N][Hq][dh]  f32 or bf16 (dtype)
 * chat   [B][C][d]       f32   (from ps_kmeans_spherical)
 * Wk     [d][Hkv*dh]     dtype
 * A_prev [B][N][C] f32 or NULL;  A_cur [B][N][C] f32 out;  D [B][N] f32 out
 * Deterministic: identical inputs give identical bits, so A_prev == A_cur
 * from an identical call gives D == 0 exactly.
 * ------------------------------------------------------------------------- */
ps_status ps_proxy_attn_kl(ps_handle h, const void* Q, const float* chat,
                           const void* Wk, int dtype, int B, int N, int d,
                           int C, int Hq, int Hkv, int dh, const float* A_prev,
                           float* A_cur, float* D, void* ws, size_t ws_bytes,
                           void* stream);

/* ---------------------------------------------------------------------------
 * a5  Top-k most-drifting clusters and the positions they cover.
 * [Polestar §2.A, sparse updates] -- "identifies the top-k drifting
 * clusters and runs a sparse forward pass on only these positions".
 *
 * score_c = (sum of D_i over members, fp64, ascending i) / n_c, for n_c > 0.
 * sel       [B][k] i32 out  clusters by score descending, ties -> lower c,
 *                           padded with -1
 * sel_score [B][k] f32 out  their scores (fp32 of the fp64 mean), pad -inf
 * pos       [B][N] i32 out  ascending positions whose cluster is selected,
 *                           then -1
 * npos      [B]    i32 out  number of such positions (stays on the device)
 * posmask   [B][N] u8  out  (nullable) 1 where the position is selected
 * Bit-exact.
 * ------------------------------------------------------------------------- */
ps_status ps_topk_drift(ps_handle h, const float* D, const int32_t* assign,
                        const int32_t* counts, int B, int N, int C, int k,
                        int32_t* sel, float* sel_score, int32_t* pos,
                        int32_t* npos, uint8_t* posmask, void* ws,
                        size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * a6  Sparse K/V refresh of the selected positions.
 * [Polestar §2.A, sparse updates] -- "a sparse forward pass on only these
 * positions ... refreshes the corresponding KV-cache entries".
 *
 * For j < npos[b], p = pos[b][j]:
 *   Kcache[b][cache_off + p] = round(H[b][p] . Wk), same for V with Wv,
 *   accumulated in fp32, rounded to the cache dtype (bf16 RNE or f32).
 * Rows not listed are untouched.  npos is read on the device.
 * H [B][N][d], Wk/Wv [d][Hkv*dh], Kcache/Vcache [B][Ncache][Hkv][dh], all
 * of `dtype`.  Requires cache_off + N <= Ncache.  bf16 with Hkv*dh a
 * multiple of 64 runs on the tensor cores and needs the workspace
 * (ps_workspace_bytes(PS_OP_REFRESH, ...): the gathered rows, B*N*d bf16
 * at most); the caches must then be 16-byte aligned.
 * ------------------------------------------------------------------------- */
ps_status ps_refresh_kv(ps_handle h, const void* H, int dtype,
                        const int32_t* pos, const int32_t* npos,
                        const void* Wk, const void* Wv, int B, int N, int d,
                        int Hkv, int dh, void* Kcache, void* Vcache,
                        int Ncache, int cache_off, void* ws, size_t ws_bytes,
                        void* stream);

/* ---------------------------------------------------------------------------
 * a7  Confidence and drift-aware commitment of a block.
 * [Polestar §2.B, current block commitment] -- commit when the drift delta
 * exceeds alpha (tau_s - c)^2;  [Polestar §2.B, suffix block commitment] --
 * suffix tokens commit only with c >= tau_s.
 *
 * Per row: token = first arg-max of the logits, conf = 1 / sum exp(l - max).
 * role[j]: 0 current block, 1 suffix block, 2 inactive.
 * Current, undecided j:  commit if conf >= tau_s, or (d_cnt >= 1 and)
 *   mode 0 DELTA_DROP:  d_sum/d_cnt - D > alpha (tau_s - conf)^2
 *   mode 1 DELTA_RISE:  D - d_sum/d_cnt > alpha (tau_s - conf)^2
 *   mode 2 RATIO:       D < ratio * d_prev
 * Suffix, undecided j: commit if suffix_sel[b][j] and conf >= tau_s.
 * ensure_progress: if no current token commits while some are undecided,
 *   the undecided current token with the largest conf commits (ties: lower j).
 * Then every undecided current token sets d_sum = fl32(d_sum + D),
 *   d_cnt += 1, d_prev = D; committed tokens get undecided = 0.
 *
 * logits [B][P][V] of `dtype` (PS_F32, or PS_BF16 as an LM head emits them;
 *   bf16 values are exact in fp32, and the bf16 scan differs from the fp32 one
 *   only in how its fp32 partial sums are grouped, so on the same values the
 *   tokens are equal and the confidences agree to rounding);
 *   role [P] u8; undecided [B][P] u8 in/out;
 * D_blk: element (b, j) at D_blk[b*d_ld + j] (e.g. the last layer's D with
 *   d_ld = N, offset to the block); d_sum/d_prev [B][P] f32 in/out,
 *   d_cnt [B][P] i32 in/out; suffix_sel: element (b, j) at
 *   suffix_sel[b*sel_ld + j] or NULL (no suffix commits);
 * token [B][P] i32, conf [B][P] f32, commit [B][P] u8 out.
 * ------------------------------------------------------------------------- */
typedef struct {
  float tau_s;
  float alpha;
  float ratio;
  int mode;            /* 0 DELTA_DROP, 1 DELTA_RISE, 2 RATIO */
  int ensure_progress; /* 0 or 1 */
} ps_commit_params;

ps_status ps_commit(ps_handle h, const void* logits, int dtype, int B, int P, int V,
                    const uint8_t* role, uint8_t* undecided,
                    const float* D_blk, int d_ld, float* d_sum, int32_t* d_cnt,
                    float* d_prev, const uint8_t* suffix_sel, int sel_ld,
                    ps_commit_params params, int32_t* token, float* conf,
                    uint8_t* commit, void* ws, size_t ws_bytes, void* stream);


/* ---------------------------------------------------------------------------
 * NVFP4 residual quantisation without a workspace.
 * The paper has no counterpart to this call: it exists for callers that
 * cannot allocate device memory -- e.g. a host application that gives the
 * library only preallocated inputs and outputs, or code running where a
 * cudaMalloc is not allowed because it may synchronise the device or break
 * a fixed memory budget.
 *
 * Computes exactly what ps_nvfp4_residual computes (same arguments, same
 * bit-exact outputs) but takes no `ws`: its scratch (per-CTA partial maxima)
 * lives in one fixed 64 KiB file-scope device array inside the library,
 * which every GPU that loads the library keeps until the process exits.
 * It calls no cudaMalloc, cudaFree or allocating library routine.
 *
 * Limit: B <= 16384 (the array holds 16384 partials; a window takes at
 * most 16384 / B of them);
 * larger B returns PS_ERR_WORKSPACE and launches nothing.
 * Device: the handle's device must be the calling thread's current device
 * (PS_ERR_ARG otherwise), since the array's address differs per device.
 * Set-up: the first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) and keeps it; make that first call before any
 * stream capture.  The kept address belongs to the device's context, so the
 * library must not be used across a reset of that device (cudaDeviceReset).
 * A failed look-up returns PS_ERR_CUDA with ps_last_cuda_error() set.
 * Sharing: every call on a device uses the same array and leaves the last
 * call's values in it.  Nothing in it has to start at zero (each call writes
 * every slot it later reads), but calls that overlap on the GPU -- on
 * different streams, or from different threads -- race on it and must be
 * serialised by the caller.
 * ------------------------------------------------------------------------- */
ps_status ps_nvfp4_residual_noalloc(ps_handle h, const void* H, int dtype,
                                    const float* mu, const int32_t* assign,
                                    const float* rho, int B, int N, int d,
                                    int C, uint8_t* codes, uint8_t* scales,
                                    float* tensor_scale, void* stream);

/* ---------------------------------------------------------------------------
 * Alternative drift signals for the ablation.
 * [Polestar §2.A, drift measurement]: KL drift tracks contextual shifts more
 * closely than cosine dissimilarity on subsets; [Polestar §4, ablation
 * studies]: it beats cosine similarity and uncertainty-based selection.
 *
 * One signal per position from the proxy distributions that
 * ps_proxy_attn_kl wrote (call it with A_prev = NULL to skip its fused KL,
 * then this on its A_cur and the previous step's distribution):
 *   PS_SCORER_KL       D = max(0, sum_c a ln(a / max(a', 1e-30))), a > 0
 *   PS_SCORER_COSINE   D = max(0, 1 - <a, a'> / (|a| |a'|)); 0 if a norm is 0
 *   PS_SCORER_ENTROPY  D = -sum_c a ln a over a > 0 (uncertainty of the
 *                      current distribution; A_prev is not read)
 * With A_prev == NULL, KL and COSINE write D = 0.
 *
 * A_cur, A_prev [B][N][C] f32 (rows of any non-negative weights; the proxy
 * writes distributions); D [B][N] f32 out, must not alias either input.
 * Sizes: B >= 0 (0: no-op), N >= 1, 1 <= C <= 4096, B * N <= 2^31 - 1.
 * Errors: a NULL handle, A_cur or D, a bad size or an unknown scorer return
 * PS_ERR_ARG before anything is enqueued.
 * ------------------------------------------------------------------------- */
typedef enum {
  PS_SCORER_KL = 0, PS_SCORER_COSINE = 1, PS_SCORER_ENTROPY = 2
} ps_scorer;

ps_status ps_drift_score(ps_handle h, const float* A_cur, const float* A_prev,
                         int B, int N, int C, int scorer, float* D,
                         void* stream);

/* ---------------------------------------------------------------------------
 * The outcome of a decode step that the refresh schedule below consumes.
 * [Polestar §2.A, schedule]: refreshes are triggered by the number of
 * decoded tokens; the window moves on when the current block is decided.
 *
 * One small kernel writes out[0] = the largest number of positions any of
 * the B sequences committed in this step (commit [B][P] u8, every role) and
 * out[1] = 1 when no sequence has an undecided current-block position left
 * (undecided [B][P] u8, role [P] u8 with 0 = current block), else 0 -- the
 * (committed, block_done) pair of ps_schedule_step, computed where the
 * flags are, so the host reads one 8-byte pair.
 * out: int32[2], 8-byte aligned, in device memory or in ps_host_alloc
 * memory (then readable on the host once the stream has reached it).
 * B == 0 or P == 0 writes (0, 1).  Errors: a NULL handle or out, an
 * unreachable or misaligned out, or NULL flags with B, P > 0 return
 * PS_ERR_ARG before anything is enqueued.
 * ------------------------------------------------------------------------- */
ps_status ps_block_progress(ps_handle h, const uint8_t* commit,
                            const uint8_t* undecided, const uint8_t* role,
                            int B, int P, int32_t* out, void* stream);

/* ---------------------------------------------------------------------------
 * Refresh schedule of the decode loop (host only; no handle, no GPU work).
 * [Polestar §2.A, schedule]: the drift refresh is triggered once the decoded
 * context has moved enough -- after tau_upd tokens were decoded -- and
 * periodic full passes refresh positions outside the top-k clusters too.
 *
 * Called after every decode step with the number of tokens that step
 * committed and whether the current block is now decided; returns the
 * actions of the NEXT step (an OR of the flags below, 0 = reuse the cache):
 *   block_done:        REFRESH | FULL | SLIDE | REINIT -- the window slides
 *                      by block_len, the next step clusters it from scratch
 *                      (k-means++), refreshes every position, and the
 *                      counts restart (since = refreshes = 0);
 *   else since += committed; if since >= tau_upd (tau_upd = 0: every step):
 *                      REFRESH, since = 0, refreshes += 1, and FULL too when
 *                      full_period > 0 and refreshes % full_period == 0.
 * The state is caller-owned; zero it for the first window (whose first step
 * the caller runs as block_done would: clustered and refreshed in full).
 * Errors: NULL pointers, tau_upd < 0, full_period < 0, block_len < 1,
 * committed < 0 or a negative state field return -PS_ERR_ARG and leave the
 * state unchanged.  The token count saturates at INT_MAX.
 * ------------------------------------------------------------------------- */
enum {
  PS_SCHED_REFRESH = 1, /* run the drift path and the top-k refresh         */
  PS_SCHED_FULL = 2,    /* refresh every window position, not only top-k    */
  PS_SCHED_SLIDE = 4,   /* a new block: reset the commit state              */
  PS_SCHED_REINIT = 8   /* re-seed k-means (k-means++), no previous A       */
};

typedef struct {
  int tau_upd;      /* tokens between refreshes, >= 0                        */
  int full_period;  /* every full_period-th refresh is full; 0 = never       */
  int block_len;    /* positions the window slides by, >= 1                  */
} ps_schedule_params;

typedef struct {
  int since;        /* tokens committed since the last refresh              */
  int refreshes;    /* refreshes since the window was built                 */
  int block_start;  /* sequence position of the current block               */
} ps_schedule_state;

int ps_schedule_step(const ps_schedule_params* p, ps_schedule_state* s,
                     int committed, int block_done);

/* ---------------------------------------------------------------------------
 * The 4-bit KV cache: rows in and out, the attention that reads it, the
 * weight that attention puts on its slots, and eviction by that weight.
 * [Polestar §2.A, sparse updates] keeps a KV cache that the refresh writes;
 * holding it in NVFP4 and dropping rows of it are this library's own.
 *
 * A layer's cache holds a K and a V row for every (sequence, KV head, slot):
 *   codes  [B][Hkv][Ncache][dh/2]  u8  E2M1, element 2j in byte j's low nibble
 *   scales [B][Hkv][Ncache][dh/16] u8  E4M3, one per 16 elements along dh
 * and two tensor scales (host values, positive and normal): an element is
 * code * scale * kmul (vmul).  dh is 64, 128 or 256.  144 bytes a slot and
 * head for dh = 128, against 512 in bf16.  A slot that was never stored may
 * hold any bytes; calls never let it reach a result.
 *
 * Every call needs B >= 0 (0: no-op), 1 <= Hkv <= 512, B * Hkv <= 65535,
 * 1 <= Ncache < 2^31 - 2^16 and 16-byte aligned codes, scales, K, V, Q and O;
 * the other arrays may start at any element.
 * ------------------------------------------------------------------------- */
typedef struct {
  uint8_t* kcode;
  uint8_t* kscale;
  uint8_t* vcode;
  uint8_t* vscale;
  int B, Hkv, Ncache, dh;
  float kmul, vmul;
} ps_kv4_cache;

/* Stores rows of K and V.  For every list entry j < min(cnt[b], R) (R where
 * cnt is NULL), r = rows[b*R + j] (j where rows is NULL) names row r of
 * sequence b, which goes to slot off[b] + r (off NULL: 0); entries with r
 * outside [0, R) or a slot outside the cache are skipped, other slots are
 * untouched.  ps_topk_drift's pos / npos are such a list.
 * Per 16 elements x: s = E4M3(fl(amax / fl(6 S))), code = E2M1(fl(x / fl(s S))),
 * RNE, saturating, 0 where s == 0 (S = kmul or vmul): ps_nvfp4_residual's
 * rounding with a given tensor scale.  Bit-exact.  Infinities saturate, a NaN
 * becomes 6 s S.
 * K, V: element (b, r, h, i) at [b*b_ld + r*ld + h*dh + i], f32 or bf16 (dtype);
 *   ld >= Hkv*dh and b_ld >= 0, multiples of 16 bytes (K and V may be parts of
 *   one projection's output);  off [B], rows [B][R], cnt [B] i32 or NULL.
 * A slot named twice in one call holds either row. */
ps_status ps_kv4_store(ps_handle h, const ps_kv4_cache* c, const void* K,
                       const void* V, int dtype, int R, int64_t b_ld,
                       int64_t ld, const int32_t* off, const int32_t* rows,
                       const int32_t* cnt, void* stream);

/* The same into a cache whose slots hold the positions kpos [B][Hkv][Ncache]
 * (ascending in every head; NULL: the slots themselves), as an eviction leaves it:
 * row r goes, in every KV head, to the slot that holds position off[b] + r, and is
 * skipped where none does. */
ps_status ps_kv4_store_pos(ps_handle h, const ps_kv4_cache* c, const void* K,
                           const void* V, int dtype, int R, int64_t b_ld,
                           int64_t ld, const int32_t* off, const int32_t* rows,
                           const int32_t* cnt, const int32_t* kpos, void* stream);

/* The reverse, with the same list: element = fl(code * s * S) rounded to
 * dtype (bf16: RNE) into K and V, whose rows must not overlap (b_ld > 0 for
 * B > 1); rows not listed are untouched. */
ps_status ps_kv4_load(ps_handle h, const ps_kv4_cache* c, void* K, void* V,
                      int dtype, int R, int64_t b_ld, int64_t ld,
                      const int32_t* off, const int32_t* rows,
                      const int32_t* cnt, void* stream);

/* Queries of T tokens a sequence and what they see of the cache.
 *   s   = scale * <q, k>                       k as the cache holds it
 *   s   = cap * tanh(s / cap)                  if cap > 0
 *   s  -= slope[h] * |qpos[b][t] - pos|        if slope (and qpos) given; at
 *                                              most 2^31 - 1 apart
 * Slot n of head g holds position kpos[b][g][n] (kpos NULL: n).  Row (b, t)
 * sees slot n iff n < len[b] (len NULL: Ncache) and span[b][t][0] <= pos <
 * span[b][t][1] (span NULL: all): causal is [0, qpos + 1), a prefix mask
 * [0, max(prefix, qpos + 1)), a document mask the document's bounds.
 * Q: element (b, t, h, i) at [b*q_bld + t*q_ld + h*dh + i]; query head h reads
 * KV head h / (Hq / Hkv).  B * T * Hq <= 2^25 - 1, Hq / Hkv <= 4096. */
typedef struct {
  const void* Q;
  const int32_t* len;   /* [B] or NULL                                      */
  const int32_t* span;  /* [B][T][2] or NULL                                */
  const int32_t* kpos;  /* [B][Hkv][Ncache] or NULL                         */
  const int32_t* qpos;  /* [B][T], needed with slope                        */
  const float* slope;   /* [Hq] or NULL                                     */
  int64_t q_bld, q_ld;  /* >= 0 and >= Hq*dh, multiples of 16 bytes         */
  int dtype, T, Hq;     /* PS_F32 or PS_BF16; T >= 0 (0: no-op)             */
  float scale, cap;     /* finite; cap >= 0, 0 for none                     */
} ps_kv4_query;

/* O [B][T][Hq][dh] (dtype) = softmax over the seen slots of s, times V;
 * lse [B][T][Hq] f32 (nullable) = ln sum exp s.  A row that sees nothing gives
 * O = 0 and lse = -inf.  Sums and statistics in fp32; the products' operands
 * are f16: the cache's values and bf16 queries exact, fp32 queries and their
 * weights in two f16 terms, the weights of bf16 queries rounded to 11 bits.
 * The cap's tanh to 2^-20 of the score; of bf16 queries under a cap of up to 64
 * to 2.5e-7 of the cap, where that is more (ps_kv4_weight: fp32's precision).
 * Deterministic.  Workspace: ps_workspace_bytes(PS_OP_KV4_ATTN, B, N = Ncache,
 * Hq, Hkv, dh, P = T). */
ps_status ps_kv4_attn(ps_handle h, const ps_kv4_cache* c, const ps_kv4_query* q,
                      void* O, float* lse, void* ws, size_t ws_bytes,
                      void* stream);

/* w_out[b][g][n] = w_in[b][g][n] + the sum over the T tokens and the query
 * heads of group g of exp(s - lse), lse [B][T][Hq] as ps_kv4_attn wrote it for
 * the same query; slots that no row sees get w_in (w_in NULL: 0).  w_in may be
 * w_out.  [B][Hkv][Ncache] f32.  A term is as good as the difference of an fp32 s
 * and an fp32 lse: to some 2^-22 of their size.  Deterministic.  Workspace: PS_OP_KV4_WEIGHT,
 * same sizes. */
ps_status ps_kv4_weight(ps_handle h, const ps_kv4_cache* c, const ps_kv4_query* q,
                        const float* lse, const float* w_in, float* w_out,
                        void* ws, size_t ws_bytes, void* stream);

/* Evicts: copies the kept slots of every (sequence, KV head) of src, in
 * ascending order, to the first slots of dst (another cache of the same B,
 * Hkv, dh and tensor scales, dst->Ncache >= keep, no memory in common).
 * len[b] <= keep: all len[b] slots.  Else `keep` of them: the first `sink`, the
 * last `recent`, and of the others the ones of largest w, ties to the lower
 * slot, NaN below every number.  w_dst and kpos_dst [B][Hkv][dst->Ncache] take
 * the kept slots' weights and positions (kpos NULL: the slot itself; kpos_dst
 * nullable), len_dst[b] = min(len[b], keep).  What lies past that is untouched.
 * 0 <= sink, recent; sink + recent <= keep; keep >= 1.  Bit-exact.
 * Workspace: PS_OP_KV4_EVICT with B, N = Ncache, Hkv, k = keep. */
ps_status ps_kv4_evict(ps_handle h, const ps_kv4_cache* src, const ps_kv4_cache* dst,
                       const float* w, const int32_t* len, const int32_t* kpos,
                       int keep, int sink, int recent, float* w_dst,
                       int32_t* kpos_dst, int32_t* len_dst, void* ws,
                       size_t ws_bytes, void* stream);

/* The same, and leaves dst ready to go on: the slots behind the kept ones, up to
 * dst->Ncache, get weight 0 and the positions that come next.  A slot n behind the
 * filled ones stands for position n + shift[b] (shift [B], NULL: 0), in dst for
 * n + shift_dst[b], shift_dst[b] = shift[b] + len[b] - len_dst[b].  kpos_dst and
 * shift_dst are needed, shift_dst is not shift. */
ps_status ps_kv4_evict_on(ps_handle h, const ps_kv4_cache* src, const ps_kv4_cache* dst,
                          const float* w, const int32_t* len, const int32_t* kpos,
                          int keep, int sink, int recent, float* w_dst,
                          int32_t* kpos_dst, int32_t* len_dst, const int32_t* shift,
                          int32_t* shift_dst, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Rotary positions, on the way into the cache.
 * [Polestar §2.A, sparse updates] refreshes K and V rows; the layers it was
 * measured on give queries and keys their positions by rotation, which
 * ps_refresh_kv leaves to this call.
 *
 * Pair i < rot/2 of a head -- elements (i, i + rot/2), or (2i, 2i + 1) with
 * `pairs` -- is turned by the angle a = position * freq_i:
 *   (x, y) -> amp (x cos a - y sin a, x sin a + y cos a)
 * in fp32, rounded to dtype; elements from rot on stay as they are.
 * freq_i = base^(-2i/rot) radians a position, and for contexts that are
 * stretched `factor` times past a trained length of orig_len:
 *   PS_ROPE_LINEAR  freq_i / factor
 *   PS_ROPE_NTK     base * factor^(rot/(rot-2)) in place of base
 *   PS_ROPE_PARTS   freq_i (w + (1 - w) / factor), w = (orig_len freq_i / 2 pi - low)
 *                   / (high - low) within [0, 1]: frequencies that turned more than
 *                   `high` times in the trained length keep their speed
 * ------------------------------------------------------------------------- */
enum { PS_ROPE_PLAIN = 0, PS_ROPE_LINEAR = 1, PS_ROPE_NTK = 2, PS_ROPE_PARTS = 3 };

typedef struct {
  int rot;                      /* elements that are rotated, even, >= 2        */
  int scaling;                  /* PS_ROPE_*                                    */
  double base;                  /* >= 1                                         */
  double factor;                /* > 0; not read by PS_ROPE_PLAIN               */
  double low, high, orig_len;   /* PS_ROPE_PARTS: 0 <= low < high, orig_len > 0 */
} ps_rope_params;

/* turns[i] = the turns that pair i makes a position, modulo 1, in units of
 * 2^-64 (so that position * turns modulo 2^64 is the angle, exact at any
 * position).  Host only: rot/2 values in host memory, which the caller copies to
 * the device once.  PS_ERR_ARG for NULL pointers or parameters out of range. */
ps_status ps_rope_turns(const ps_rope_params* p, uint64_t* turns);

/* Rows of one tensor: element (b, r, h, i) of X at [b*x_bld + r*x_ld + h*dh + i],
 * Y likewise.  Strides are >= 0, x_ld and y_ld >= H*dh, multiples of 16 bytes.
 * slots == 0: row r of X goes to row r of Y, and Y may be X (with X's strides).
 * slots > 0: row r goes to the slot that the call gives it, if that is one of the
 * `slots` rows that a sequence has in Y; Y and X have no memory in common. */
typedef struct {
  const void* X;
  void* Y;
  int64_t x_bld, x_ld, y_bld, y_ld;
  int H;          /* heads, >= 1                                              */
  int rotate;     /* 0: the rows are moved as they are (V); 1: rotated        */
  int slots;
} ps_rope_part;

/* For every list entry j < min(cnt[b], T) (T where cnt is NULL), r = rows[b*T + j]
 * (j where rows is NULL; entries outside [0, T) are skipped) names row r of
 * sequence b: its position is pos[b*T + r] (pos NULL: off[b] + r), its slot
 * dst[b*T + r] (dst NULL: off[b] + r; off NULL: r).  Other rows are untouched.
 * An entry that is there twice writes the same twice, but with Y == X, where the
 * entries of a list must differ.  Of a slot that two rows name every element is one of
 * the two rows', not all of them the same one's, and another call's may be others. */
typedef struct {
  const uint64_t* turns;  /* [rot/2], device memory                           */
  const int32_t* pos;     /* [B][T] or NULL; negative positions turn back     */
  const int32_t* off;     /* [B] or NULL                                      */
  const int32_t* rows;    /* [B][T] or NULL                                   */
  const int32_t* cnt;     /* [B] or NULL                                      */
  const int32_t* dst;     /* [B][T] or NULL                                   */
  int B, T, dh, rot;      /* B, T >= 0 (0: no-op); dh % 16 == 0, dh <= 256    */
  int pairs, dtype;       /* 0 or 1; PS_F32 or PS_BF16                        */
  float amp;              /* finite                                           */
} ps_rope_rows;

/* One to three parts (a layer's Q, K and V) in one launch.  B * T < 2^31,
 * H <= 4096.  The angle is position * turns to 2^-25 radians at any position of 32
 * bits (ps_rope_turns works in fp64: some 2^-50 of a frequency).  Bit-exact from
 * call to call, slots named twice apart. */
ps_status ps_rope(ps_handle h, const ps_rope_rows* r, const ps_rope_part* parts,
                  int nparts, void* stream);

/* ---------------------------------------------------------------------------
 * Attention over packed sequences, or over rows of the cache.
 * [Polestar §2.A, sparse updates] keeps a KV cache that the refresh writes; this is
 * the attention that reads it in the type it was written in: a prompt's rows, a
 * block's, or single tokens', for any number of sequences of unequal lengths.
 *
 * Sequence s has the rows q_off[s] .. q_off[s+1] - 1 of Q, and of K and V the rows
 * k_off[s] .. k_off[s] + k_len[s] - 1 (its slots 0, 1, ...; k_len NULL: up to
 * k_off[s+1], and k_off has S + 1 entries).  In a cache [B][Ncache][Hkv][dh],
 * k_off[s] = s * Ncache.  Row t of n (from 0), of a sequence with m slots, sees slot j iff
 *   j < m,
 *   j <= m - n + t           if causal (its rows are the last ones of the slots),
 *   span[0] <= j < span[1]   if span is given (for the row of Q).
 * s = scale * <q, k>;  O = softmax over the seen slots of s, times V;  lse = ln sum
 * exp s.  A row that sees nothing, or no score above -inf, gives O = 0, lse = -inf.  Query head h reads KV head
 * h / (Hq / Hkv).  What a row does not see never reaches it, NaN or not.  Rows of
 * O and lse that belong to no sequence are left as they are.  Offsets outside the
 * tensors are cut to them; q_off must ascend.
 *
 * Q: element (r, h, i) at [r*q_ld + h*dh + i], K and V likewise with Hkv heads; O
 *   [Tq][Hq][dh] at o_ld; strides >= a row, multiples of 16 bytes, all of dtype
 * lse [Tq][Hq] f32 (nullable)
 * max_q, max_k: the most rows and slots of a sequence, as well as the caller knows
 *   them: they choose a launch and its workspace, never a result's rows or slots.
 * Sums and statistics in fp32.  bf16: products exact, the weights rounded to bf16 on
 * their way into the product with V (lse and the weights' sum are of the unrounded ones).  f32: to some 2^-21 of the terms.  Deterministic.
 * Sizes: S, Tq >= 0 (0: no-op), S <= 2^20, Tq * Hq <= 2^30, Tk < 2^31 - 2^16,
 *   Hkv <= 512, Hq / Hkv <= 4096, dh % 16 == 0, dh <= 256, max_q, max_k >= 1.
 * Workspace: ps_workspace_bytes(PS_OP_ATTN, B = S, N = max_k, Hq, Hkv, dh, P = Tq,
 * k = max_q), of the numbers that the call gets: others, larger ones too, may give less,
 * since they choose how the slots are shared out.  A caller whose lengths grow passes one
 * max_k throughout. */
typedef struct {
  const void* Q;
  const void* K;
  const void* V;
  int64_t q_ld, k_ld, v_ld, o_ld;
  const int32_t* q_off;  /* [S + 1]                    */
  const int32_t* k_off;  /* [S], or [S + 1] without k_len */
  const int32_t* k_len;  /* [S] or NULL                */
  const int32_t* span;   /* [Tq][2] or NULL            */
  int dtype, S, Tq, Tk, Hq, Hkv, dh;
  int causal;            /* 0 or 1                     */
  int max_q, max_k;
  float scale;           /* finite                     */
} ps_attn_rows;

ps_status ps_attn(ps_handle h, const ps_attn_rows* a, void* O, float* lse, void* ws,
                  size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Tokens drawn from the logits, and the commit rule on drawn tokens.
 * [Polestar §2.B] rates tokens by a confidence that it does not define;
 * ps_commit takes the arg-max and its probability, these calls a drawn token and
 * the probability it was drawn with.
 *
 * Per row r, of V logits l (a NaN counts as -inf):
 *   w_i = exp((l_i - max l) / T)     T = temperature[r] (1e-30 at least); T <= 0 or NaN: 1,
 *                                    and the token is the first arg-max in place of a draw
 * in descending order of l, ties to the lower index, what is left is
 *   the first top_k                  (top_k <= 0: all),
 *   of those the shortest prefix whose sum of w is at least top_p times theirs
 *                                    (top_p >= 1 or NaN: all), one at least,
 *   of those the ones with w_i >= min_p   (min_p <= 0 or NaN: all; above 1: as 1).
 * token = the first i in ascending order whose running sum of the w left exceeds
 * u[r] times their sum; prob = w_token / their sum; n = how many are left, -inf not
 * counted.  An infinite maximum counts as 0 and all below it as -inf.  A row with
 * nothing above -inf gives token -1, prob 0, n 0.
 * The w are fixed point of 43 bits, good to 2^-29 of themselves and 2^-43 (a smaller one
 * is 0, and such a token not drawn); sums are exact.  So a result differs from that of
 * exact w only where a sum lies that close to a border.
 * Bit-exact from call to call.
 *
 * logits: element (r, i) at [r*ld + i], f32 or bf16 (dtype), ld >= V; any alignment of
 *   rows (16-byte aligned ones are read faster)
 * u [R] f64 in [0, 1) (outside: the nearest); temperature, top_p, min_p [R] f32,
 * top_k [R] i32, each NULL for none
 * token [R] i32, prob [R] f32 (nullable), n [R] i32 (nullable) out
 * R >= 0 (0: no-op), R <= 2^27, 1 <= V <= 10^6. */
typedef struct {
  const void* logits;
  const double* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int64_t ld;
  int dtype, R, V;
} ps_sample_rows;

ps_status ps_sample(ps_handle h, const ps_sample_rows* s, int32_t* token, float* prob,
                    int32_t* n, void* stream);

/* ps_commit's rule with the tokens' confidences given (conf [B][P] f32, e.g. the prob
 * of ps_sample; any numbers, a NaN counts as -inf): everything as there, no logits, no
 * workspace. */
ps_status ps_commit_drawn(ps_handle h, const float* conf, int B, int P,
                          const uint8_t* role, uint8_t* undecided, const float* D_blk,
                          int d_ld, float* d_sum, int32_t* d_cnt, float* d_prev,
                          const uint8_t* suffix_sel, int sel_ld,
                          ps_commit_params params, uint8_t* commit, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* POLESTAR_H */
