/*
 * hsa.h - C ABI of the Heterogeneous Step Allocation (HSA) denoising step on
 * NVIDIA B200 (sm_100a).  Implemented by libhsa.so.
 *
 * The method ("Not All Tokens Need 40 Steps: Heterogeneous Step Allocation in
 * Diffusion Transformers for Efficient Video Generation"; its steps are laid
 * out in "Technical Summary: Heterogeneous Step Allocation (HSA) for
 * Efficient Video Generation", sections 2.1-2.4, cited below as [TS]) splits
 * the N tokens of a video latent into K groups with step budgets s_k | T.
 * Only the tokens active at a global iteration run through the transformer;
 * their fresh K/V rows overwrite a per-layer KV cache that every active query
 * attends to in full; and one cached Euler update advances all N tokens.
 *
 * Conventions for every call:
 *  - Pointers marked (device) are caller-owned device memory on the device
 *    that was current at hsa_create; (host) pointers are host memory.  All
 *    device pointers must be 16-byte aligned.  Tensors are dense row-major
 *    with exactly the strides given.
 *  - bf16 buffers are passed as void* and hold IEEE bfloat16 values.
 *  - Every call enqueues its kernels on the context's stream and returns
 *    without waiting for them; the caller orders other work on that stream.
 *    A context is not re-entrant: calls on one context must not overlap.
 *  - Calls return a status and never abort.  A status other than HSA_OK comes
 *    with a message from hsa_last_error().  Argument errors are detected on
 *    the host before anything is launched.  Errors found by kernels (an index
 *    out of range, a wait that timed out) set a device flag that
 *    hsa_sync_check() reads.
 *  - Shapes: C = 16 latent channels; head_dim d = D / H is 64 or 128;
 *    D % 128 == 0; F % 64 == 0; 1 <= N < 2^31; 1 <= K <= 8.
 */
#ifndef HSA_H_
#define HSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  HSA_OK = 0,
  HSA_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, n out of range, ... */
  HSA_ERR_BUDGET = 2,       /* s_k does not divide T, s_1 != T, counts do not sum to N */
  HSA_ERR_SHAPE = 3,        /* model shape outside the supported set above */
  HSA_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed */
  HSA_ERR_OOM = 5,          /* scratch allocation failed in hsa_create */
  HSA_ERR_TIMEOUT = 6,      /* a kernel's bounded wait expired (read by hsa_sync_check) */
  HSA_ERR_DEVICE_CHECK = 7, /* a kernel found a bad index or a NaN score (hsa_sync_check) */
  HSA_ERR_SCRATCH_LIMIT = 8 /* a size beyond the fixed scratch of hsa_select_groups_static */
} hsa_status;

/* Model shape.  N tokens, C latent channels, D hidden, H heads, F MLP width, L layers. */
typedef struct {
  int N, C, D, H, F, L;
} hsa_model_cfg;

/* One transformer block's weights, bf16, Linear layout [out, in], row-major (device). */
typedef struct {
  const void* w_qkv; /* [3D, D]: rows 0..D-1 -> Q, D..2D-1 -> K, 2D..3D-1 -> V */
  const void* w_o;   /* [D, D] */
  const void* w_1;   /* [F, D] */
  const void* w_2;   /* [D, F] */
} hsa_layer_weights;

/* Whole-model weights for hsa_step. */
typedef struct {
  const float* w_in;               /* fp32 [D, C] latent -> hidden embed (device) */
  const float* w_head;             /* fp32 [C, D] hidden -> velocity head (device) */
  const hsa_layer_weights* layers; /* host array of L blocks */
} hsa_model_weights;

/* Per-loop state for hsa_step (all device buffers, caller-owned). */
typedef struct {
  float* x;            /* fp32 [N, C] latent, advanced in place */
  float* v_hat;        /* fp32 [N, C] velocity of each token's latest active step */
  float* v_hat_prev;   /* fp32 [N, C] the velocity before that */
  float* v_fresh;      /* fp32 [N, C] this step's head output (rows of A_i written) */
  float* score;        /* fp32 [N] last selector scores */
  uint8_t* g;          /* uint8 [N] group id per token */
  uint8_t* mask;       /* uint8 [N] active mask of the current iteration */
  int32_t* active_idx; /* int32 [N] ascending active tokens (first |A_i| valid) */
  float* h;            /* fp32 [N, D] hidden rows */
  void* const* k_cache;/* host array of L device pointers, bf16 [N, D] each */
  void* const* v_cache;/* host array of L device pointers, bf16 [N, D] each */
} hsa_state;

typedef struct hsa_ctx hsa_ctx;

/*
 * Create a context for one model shape and group layout ([TS] 2.1).
 *   cfg      (host) model shape.
 *   T        total steps.
 *   budgets  (host) s_1..s_K: s_1 == T, strictly decreasing, each divides T.
 *   counts   (host) n_1..n_K tokens per group, sum == N.
 *   K        number of groups, 1..8.
 *   m        phase-aware window ([TS] 2.4): the first m and last m iterations
 *            are full passes for all tokens; 0 disables it; 2m <= T.
 *   stream   cudaStream_t to launch on (NULL = legacy default stream).
 *   out      (host) receives the context.
 * Allocates the context's scratch (compact activations sized for |A| = N,
 * selector histograms, the device error flag) with cudaMalloc.  On failure
 * *out is NULL and nothing is leaked.
 */
hsa_status hsa_create(const hsa_model_cfg* cfg, int T, const int* budgets, const int* counts,
                      int K, int m, void* stream, hsa_ctx** out);

/* Free the context and its scratch.  Synchronises its stream first.  NULL is a no-op. */
void hsa_destroy(hsa_ctx* ctx);

/* Message for the last failing call on ctx (never NULL).  ctx may be NULL for hsa_create errors. */
const char* hsa_last_error(const hsa_ctx* ctx);

/* Replace the stream used by later calls. */
hsa_status hsa_set_stream(hsa_ctx* ctx, void* stream);

/* Synchronise the stream, then read and clear the device error flag. */
hsa_status hsa_sync_check(hsa_ctx* ctx);

/*
 * Failure-detection self-test.  Launches one kernel whose mbarrier wait is
 * never satisfied; the same bounded wait the pipelined kernels use gives up
 * after timeout_us microseconds (1..2000000) and records a timeout in the
 * device flag.  The next hsa_sync_check then returns HSA_ERR_TIMEOUT and
 * clears the flag; the context stays usable.  Nothing faults or hangs.
 */
hsa_status hsa_selftest_timeout(hsa_ctx* ctx, int timeout_us);

/* Number of kernels this context has launched so far (host counter, no sync). */
uint64_t hsa_kernel_launches(const hsa_ctx* ctx);

/*
 * Per-launch timing of the calls above, for measuring the kernels inside a
 * running step (no counterpart on the pages: instrumentation).  While on, every
 * kernel launch of the context is bracketed by two CUDA events on its stream
 * and its algorithmic work is added up per class:
 *   0 attention   (hsa_attention, hsa_attention_kv, hsa_cross_attention; work = 4 n n_kv D
 *                  FLOP, n_kv the padded count where lengths are on the device)
 *   1 GEMM        (QKV, out-projection, MLP, linear, 8-bit products; work = 2 M Ncols K
 *                  operations)
 *   2 row kernels (LN gather, KV scatter, embed, head, quantisation, rotary positions;
 *                  work = bytes moved)
 *   3 per-token   (schedule, score, selection, Euler; work = 0)
 * hsa_kernel_times synchronises the stream, writes the first n_classes
 * classes' totals (launch calls, summed event milliseconds, work) to out, and
 * clears them.  Events are taken from a pool the context owns.  Off by
 * default; not meant for use under stream capture.
 */
typedef struct {
  uint64_t calls;
  double ms;
  double work;
} hsa_kernel_class_time;

hsa_status hsa_time_kernels(hsa_ctx* ctx, int on);
hsa_status hsa_kernel_times(hsa_ctx* ctx, hsa_kernel_class_time* out, int n_classes);

/*
 * |A_i| computed on the host from the group counts ([TS] 2.1): the sum of n_k
 * over the groups active at iteration i.  Valid when g holds exactly counts[k]
 * tokens of group k, which the initial split and hsa_select_groups guarantee.
 * Returns -1 if i is outside [0, T).
 */
int hsa_n_active(const hsa_ctx* ctx, int i);

/*
 * Group schedule ([TS] 2.1, 2.4).  Token n is active at iteration i iff
 * i mod (T / s_{g[n]}) == 0, or i is inside the phase window.
 *   g           (device) uint8 [N] group ids, each < K.
 *   mask        (device) uint8 [N] out: 1 if active.
 *   active_idx  (device) int32 [N] out: active tokens in ascending order.
 *   n_active_dev(device) int32 [1] out, may be NULL: |A_i| as counted on the GPU.
 *   n_active    (host)   out, may be NULL: |A_i| from hsa_n_active (no sync).
 * A group id >= K counts as inactive and sets the device check flag.
 */
hsa_status hsa_schedule(hsa_ctx* ctx, int i, const uint8_t* g, uint8_t* mask, int32_t* active_idx,
                        int32_t* n_active_dev, int* n_active);

/*
 * Per-token L1 relative change of the velocity ([TS] 2.1, Dynamic Selection):
 *   score[n] = sum_c |v_cur[n,c] - v_prev[n,c]| / (sum_c |v_prev[n,c]| + 1e-6)
 * in float32, each sum in channel order 0..C-1, one IEEE division.
 *   v_prev, v_cur (device) fp32 [N, C];  score (device) fp32 [N] out.
 */
hsa_status hsa_score(hsa_ctx* ctx, const float* v_prev, const float* v_cur, float* score);

/*
 * Group assignment from a score buffer ([TS] 2.1): tokens ranked by (score
 * descending, index ascending); the first n_1 get group 0 (budget T), the
 * next n_2 group 1, and so on.  Exact and deterministic (integer radix select).
 *   score (device) fp32 [N], finite and >= 0 (a NaN sets the device check flag).
 *   g     (device) uint8 [N] out.
 */
hsa_status hsa_select_from_score(hsa_ctx* ctx, const float* score, uint8_t* g);

/* hsa_score followed by hsa_select_from_score; score may not be NULL. */
hsa_status hsa_select_groups(hsa_ctx* ctx, const float* v_prev, const float* v_cur, float* score,
                             uint8_t* g);

/*
 * Gather + LayerNorm of the active rows (the first stage of the active-only
 * forward, [TS] 2.2 step 1): u[m] = LN(x[idx[m]]) without affine, eps 1e-5.
 *   x   (device) fp32 [N, D];  idx (device) int32 [n];  u (device) bf16 [n, D] out.
 */
hsa_status hsa_ln_gather(hsa_ctx* ctx, const float* x, const int32_t* idx, int n, void* u);

/*
 * QKV projection of the active rows and KV-cache write ([TS] 2.2 steps 1-2):
 * [Q|K|V] = u W_qkv^T; Q goes to the compact buffer q, the fresh K and V rows
 * overwrite rows idx[m] of this layer's caches.
 *   w_qkv (device) bf16 [3D, D];  u (device) bf16 [n, D];  idx (device) int32 [n]
 *   q (device) bf16 [n, D] out;  k_cache, v_cache (device) bf16 [N, D] in/out.
 */
hsa_status hsa_qkv_project(hsa_ctx* ctx, const void* w_qkv, const void* u, const int32_t* idx,
                           int n, void* q, void* k_cache, void* v_cache);

/*
 * The same QKV projection for a sequence-sharded step, with the exchange of
 * the fresh K/V rows folded into the GEMM's epilogue ([TS] 2.2 steps 1-2:
 * every active token's fresh K/V rows must reach every copy of the cache
 * before attention reads it).  Q goes to q as in hsa_qkv_project; every fresh
 * K and V row is stored to row idx[m] of each of the n_caches cache pairs,
 * so that one launch writes this rank's rows into its own cache and, through
 * peer-mapped pointers, into every other rank's copy over NVLink.
 *   w_qkv, u, idx, q as hsa_qkv_project;
 *   k_caches, v_caches (HOST arrays of n_caches pointers, borrowed for the
 *   call): device bf16 [N, D] caches, each on this GPU or a peer GPU's memory
 *   mapped into this process (CUDA IPC or peer access); 1 <= n_caches <= 8.
 * The launch only stores to peer memory (no load reads another GPU).  The
 * caller orders it against the peers' readers: no peer may read the rows
 * before this launch completes (a device-side barrier on the stream after
 * it), and no peer may still be reading a previous step's rows of these
 * caches when it starts.  HSA_ERR_INVALID_ARG for n_caches out of range or a
 * NULL / misaligned pointer; an index outside [0, N) is skipped and reported
 * by hsa_sync_check (HSA_ERR_DEVICE_CHECK).
 */
hsa_status hsa_qkv_project_peers(hsa_ctx* ctx, const void* w_qkv, const void* u,
                                 const int32_t* idx, int n, void* q, void* const* k_caches,
                                 void* const* v_caches, int n_caches);

/*
 * Active-row linear map, the tensor-core building block of the QKV,
 * out-projection and MLP products ([TS] 2.2): out = a w^T, fp32 accumulation.
 *   a (device) bf16 [M, Kd];  w (device) bf16 [Ncols, Kd];  out (device) bf16 [M, Ncols].
 *   Kd % 64 == 0, Ncols % 32 == 0, M >= 0.
 */
hsa_status hsa_linear(hsa_ctx* ctx, const void* a, int M, int Kd, const void* w, int Ncols,
                      void* out);

/*
 * KV-cache write alone ([TS] 2.2 step 2): k_cache[idx[m]] = k_rows[m],
 * v_cache[idx[m]] = v_rows[m].
 *   k_rows, v_rows (device) bf16 [n, D];  k_cache, v_cache (device) bf16 [N, D].
 */
hsa_status hsa_kv_scatter(hsa_ctx* ctx, const void* k_rows, const void* v_rows,
                          const int32_t* idx, int n, void* k_cache, void* v_cache);

/*
 * The same KV-cache write from packed rows, as a sequence-sharded step
 * receives them after gathering every rank's fresh rows ([TS] 2.2 step 2):
 * k_cache[idx[m]] = kv_rows[m][0 .. D), v_cache[idx[m]] = kv_rows[m][D .. 2D).
 *   kv_rows (device) bf16 [n, 2D];  idx (device) int32 [n], each < N;
 *   k_cache, v_cache (device) bf16 [N, D].  An index outside [0, N) is skipped
 *   and reported by hsa_sync_check (HSA_ERR_DEVICE_CHECK).
 */
hsa_status hsa_kv_scatter_packed(hsa_ctx* ctx, const void* kv_rows, const int32_t* idx, int n,
                                 void* k_cache, void* v_cache);

/*
 * Full-context attention of the active queries ([TS] 2.2 steps 3-4):
 * per head, o[m] = softmax(q[m] K^T / sqrt(d)) V over all N cached rows,
 * fp32 accumulation, online softmax.  Cost O(n * N).
 *   q (device) bf16 [n, D];  k_cache, v_cache (device) bf16 [N, D];  o (device) bf16 [n, D] out.
 */
hsa_status hsa_attention(hsa_ctx* ctx, const void* q, int n, const void* k_cache,
                         const void* v_cache, void* o);

/*
 * The same attention against an explicit set of n_kv key/value rows, e.g. the
 * text tokens of cross-attention ([TS] 2.2 step 4 names cross-attention as
 * work that skipped tokens do not incur): o[m] = softmax(q[m] K^T / sqrt(d)) V
 * per head over the n_kv rows.
 *   q (device) bf16 [n, D];  k, v (device) bf16 [n_kv, D];  o (device) bf16 [n, D] out.
 * HSA_ERR_SHAPE if n_kv < 1.
 */
hsa_status hsa_attention_kv(hsa_ctx* ctx, const void* q, int n, const void* k, const void* v,
                            int n_kv, void* o);

/*
 * Out-projection on the active rows, added into the residual rows
 * ([TS] 2.2 step 4): x[idx[m]] += o[m] W_o^T.
 *   w_o (device) bf16 [D, D];  o (device) bf16 [n, D];  x (device) fp32 [N, D] in/out.
 */
hsa_status hsa_out_proj_residual(hsa_ctx* ctx, const void* w_o, const void* o,
                                 const int32_t* idx, int n, float* x);

/*
 * MLP on the active rows ([TS] 2.2 step 4):
 * x[idx[m]] += GELU(LN(x[idx[m]]) W_1^T) W_2^T (exact erf GELU, no biases).
 *   w_1 (device) bf16 [F, D];  w_2 (device) bf16 [D, F];  x (device) fp32 [N, D] in/out.
 * Uses the context's scratch for the LN output and the [n, F] hidden.
 */
hsa_status hsa_mlp_residual(hsa_ctx* ctx, const void* w_1, const void* w_2, float* x,
                            const int32_t* idx, int n);

/*
 * The stages above with the timestep modulation of a conditioned block (the
 * reading of hsa_layer_forward_cond below; [TS] 2.2 step 4 names conditioning
 * only as work skipped tokens do not incur), for callers that run a
 * conditioned block stage by stage, such as a sequence-sharded step:
 *   hsa_ln_gather_mod:            u[m] = LN(x[idx[m]]) * (1 + scale) + shift
 *   hsa_out_proj_residual_gated:  x[idx[m]] += gate * (o[m] W_o^T)
 *   hsa_mlp_residual_mod:         x[idx[m]] += gate * GELU(u2 W_1^T) W_2^T with
 *                                 u2 = LN(x[idx[m]]) * (1 + scale) + shift
 * shift, scale, gate (device) fp32 [D], 16-byte aligned; shift and scale are
 * both given or both NULL (no modulation), gate NULL means 1.  Other
 * arguments, layouts and errors as the unmodulated calls.
 */
hsa_status hsa_ln_gather_mod(hsa_ctx* ctx, const float* x, const int32_t* idx, int n, void* u,
                             const float* shift, const float* scale);
hsa_status hsa_out_proj_residual_gated(hsa_ctx* ctx, const void* w_o, const void* o,
                                       const int32_t* idx, int n, float* x, const float* gate);
hsa_status hsa_mlp_residual_mod(hsa_ctx* ctx, const void* w_1, const void* w_2, float* x,
                                const int32_t* idx, int n, const float* shift,
                                const float* scale, const float* gate);

/*
 * One transformer block on the active set ([TS] 2.2): LN -> QKV (K/V written
 * into the caches) -> attention of the n queries against all N cached rows
 * -> out-projection + residual -> LN -> MLP + residual.  Only rows idx of x
 * and of the caches change.
 *   w (host) weights;  x (device) fp32 [N, D];  idx (device) int32 [n], ascending,
 *   each < N;  k_cache, v_cache (device) bf16 [N, D].
 */
hsa_status hsa_layer_forward(hsa_ctx* ctx, const hsa_layer_weights* w, float* x,
                             const int32_t* idx, int n, void* k_cache, void* v_cache);

/* Text cross-attention of a conditioned block: its weights and the text
 * tokens' keys and values, fixed for the whole sampling run. */
typedef struct {
  const void* w_q;    /* (device) bf16 [D, D] query projection */
  const void* w_o;    /* (device) bf16 [D, D] output projection */
  const void* k_txt;  /* (device) bf16 [n_txt, D] */
  const void* v_txt;  /* (device) bf16 [n_txt, D] */
  int n_txt;          /* >= 1 */
} hsa_cross_attn;

/*
 * A conditioned block on the active set.  The pages name timestep conditioning
 * and text cross-attention only as work skipped tokens do not incur ([TS] 2.2
 * step 4) and give no architecture, so this follows the usual video-DiT form:
 *   u   = LN(x) * (1 + scale_a) + shift_a;  QKV, K/V into the caches, attention
 *         over all N cached rows;  x += gate_a * (o W_o^T)
 *   x  += W_oc Attn(LN(x) W_qc^T, k_txt, v_txt)            (if xa != NULL)
 *   u2  = LN(x) * (1 + scale_m) + shift_m;  x += gate_m * (GELU(u2 W_1^T) W_2^T)
 * with mod (device, fp32 [6, D], 16-byte aligned) holding the rows
 * shift_a, scale_a, gate_a, shift_m, scale_m, gate_m of this iteration.
 * mod == NULL and xa == NULL is hsa_layer_forward.  Only rows idx of x and of
 * the caches change.  Errors as hsa_layer_forward; HSA_ERR_SHAPE if
 * xa->n_txt < 1, HSA_ERR_INVALID_ARG for a NULL or misaligned pointer.
 */
hsa_status hsa_layer_forward_cond(hsa_ctx* ctx, const hsa_layer_weights* w, const float* mod,
                                  const hsa_cross_attn* xa, float* x, const int32_t* idx, int n,
                                  void* k_cache, void* v_cache);

/*
 * Embed the active latent rows: h[idx[m]] = x_lat[idx[m]] W_in^T.
 *   w_in (device) fp32 [D, C];  x_lat (device) fp32 [N, C];  h (device) fp32 [N, D].
 */
hsa_status hsa_embed(hsa_ctx* ctx, const float* w_in, const float* x_lat, const int32_t* idx,
                     int n, float* h);

/*
 * Velocity head on the active rows: v_fresh[idx[m]] = LN(h[idx[m]]) W_head^T.
 *   w_head (device) fp32 [C, D];  h (device) fp32 [N, D];  v_fresh (device) fp32 [N, C].
 */
hsa_status hsa_head(hsa_ctx* ctx, const float* w_head, const float* h, const int32_t* idx,
                    int n, float* v_fresh);

/*
 * Cached Euler update over all N tokens in one pass ([TS] 2.3):
 *   v_hat_prev[n] = mask[n] ? v_hat[n]   : v_hat_prev[n]
 *   v_hat[n]      = mask[n] ? v_fresh[n] : v_hat[n]
 *   x[n]          = x[n] + (sigma_next - sigma_i) * v_hat[n]
 * in float32 with one rounding per operation (no fused multiply-add).
 *   x, v_hat, v_hat_prev (device) fp32 [N, C] in/out;  v_fresh (device) fp32 [N, C];
 *   mask (device) uint8 [N].
 */
hsa_status hsa_euler_step(hsa_ctx* ctx, float* x, float* v_hat, float* v_hat_prev,
                          const float* v_fresh, const uint8_t* mask, float sigma_i,
                          float sigma_next);

/*
 * The same cached Euler update, and in the same pass the score of the
 * re-grouping that follows it ([TS] 2.1, Dynamic Selection; [TS] 2.3): after
 * the update above,
 *   score[n] = sum_c |v_hat[n,c] - v_hat_prev[n,c]| / (sum_c |v_hat_prev[n,c]| + 1e-6)
 * in float32, sums in channel order, bit for bit what hsa_score writes for
 * (v_hat_prev, v_hat).  A re-grouping step thus reads the velocity caches
 * once; hsa_select_from_score then assigns the groups.
 *   score (device) fp32 [N] out; the other arguments as hsa_euler_step.
 *   A NaN, negative or infinite score is reported by hsa_sync_check
 *   (HSA_ERR_DEVICE_CHECK).
 */
hsa_status hsa_euler_step_score(hsa_ctx* ctx, float* x, float* v_hat, float* v_hat_prev,
                                const float* v_fresh, const uint8_t* mask, float sigma_i,
                                float sigma_next, float* score);

/*
 * One global iteration i of the HSA loop ([TS] 2.1-2.3): schedule -> embed
 * the active latent rows -> every layer on A_i -> head -> cached Euler over
 * all N -> (when ``regroup`` is non-zero and T/s_K <= i < T-1) re-select the
 * groups from v_hat_prev and v_hat (the Euler pass writes the scores, as
 * hsa_euler_step_score).  No host synchronisation.
 *   w (host) model weights;  s (host) state;  sigma_i, sigma_next the noise
 *   levels of iterations i and i+1.
 */
hsa_status hsa_step(hsa_ctx* ctx, const hsa_model_weights* w, const hsa_state* s, int i,
                    float sigma_i, float sigma_next, int regroup);

/*
 * Conditioning of one iteration for hsa_step_cond: per layer, the modulation
 * vectors of this iteration (they follow the timestep, so the caller passes
 * new ones each iteration) and the text cross-attention (fixed for the run).
 * See hsa_layer_forward_cond for what they do; the pages give no
 * architecture for either ([TS] 2.2 step 4 only says skipped tokens incur no
 * cross-attention).
 */
typedef struct {
  const float* const* mod;  /* host array of L device pointers, fp32 [6, D] each (a NULL
                               entry: that layer unmodulated), or NULL for none */
  const hsa_cross_attn* xa; /* host array of L entries, or NULL for no cross-attention */
} hsa_cond;

/*
 * hsa_step with conditioned blocks: every layer runs hsa_layer_forward_cond
 * with cond->mod[l] and cond->xa[l].  cond == NULL is hsa_step.  Arrays are
 * read during the call only.  Errors as hsa_step and hsa_layer_forward_cond.
 */
hsa_status hsa_step_cond(hsa_ctx* ctx, const hsa_model_weights* w, const hsa_state* s,
                         const hsa_cond* cond, int i, float sigma_i, float sigma_next,
                         int regroup);

/* ------------------------------------------------------------------------
 * Operators around the block for models that need them: 8-bit integer
 * products, rotary positions, query/key norms, and cross-attention of ragged
 * sequences.  The pages describe none of these; the formulas are given at each
 * call.  Besides the conventions above:
 *  - The calls below make the context's device current while they launch, so
 *    they work from a thread whose current device is another one.
 *  - They read no tensor on the host and never wait, so they can be captured
 *    into a CUDA graph.  hsa_cross_attention uses the context's scratch: like
 *    calls, replays of graphs captured from one context must not overlap.
 *  - `ld_*` arguments are distances between rows in elements.
 *  - n == 0 rows launch nothing.
 * ------------------------------------------------------------------------ */

/* Element types of the calls that take more than one. */
typedef enum { HSA_BF16 = 0, HSA_F32 = 1 } hsa_type;

/*
 * Quantise n rows to signed 8 bits, one scale per row:
 *   top = max_k |a[m,k]|;  scale[m] = top / 127;  q[m,k] = rint(a[m,k] * (127 / top))
 * in fp32, halves to even, so |q| <= 127 and a ~ scale q.  A row with
 * top < 2^-100 gives q = 0, scale = 0; a row that holds an infinity or a NaN
 * gives q = 0, scale = NaN.
 *   a     (device) HSA_BF16 or HSA_F32 [n, Kd], rows ld_a >= Kd apart (any alignment of rows);
 *   q     (device) int8 [n, Kd] out, rows ld_q apart, a multiple of 16, >= Kd (bytes past Kd
 *         are left as they are);
 *   scale (device) fp32 [n] out.   1 <= Kd <= 131071.
 * Weights kept in 8 bits are made by the same call (a row per output channel).
 */
hsa_status hsa_quant_rows(hsa_ctx* ctx, const void* a, int a_type, int n, int Kd, int64_t ld_a,
                          int8_t* q, int64_t ld_q, float* scale);

/*
 * Linear map of 8-bit rows with scales per row and per output channel:
 *   out[m,j] = a_scale[m] * w_scale[j] * sum_k a[m,k] w[j,k]
 * The sum is exact (32-bit integers); the products are fp32, rounded once to bf16.
 *   a (device) int8 [M, ld_a];  a_scale (device) fp32 [M];
 *   w (device) int8 [Ncols, ld_w];  w_scale (device) fp32 [Ncols];
 *   out (device) bf16 [M, Ncols].
 *   ld_a, ld_w multiples of 16, >= Kd; bytes past Kd are ignored.
 *   M >= 0, Ncols >= 1, 1 <= Kd <= 131071.
 */
hsa_status hsa_linear_quant(hsa_ctx* ctx, const int8_t* a, int64_t ld_a, const float* a_scale,
                            int M, int Kd, const int8_t* w, int64_t ld_w, const float* w_scale,
                            int Ncols, void* out);

/*
 * hsa_ln_gather_mod straight to 8 bits: the rows u[m] = LN(x[idx[m]]) (1 + mscale) + shift
 * (fp32, not rounded to bf16 first) quantised as hsa_quant_rows does.
 *   x, idx, n, shift, mscale as hsa_ln_gather_mod;  q (device) int8 [n, D] out;
 *   scale (device) fp32 [n] out.  D <= 5120 (HSA_ERR_SHAPE beyond).
 */
hsa_status hsa_ln_gather_quant(hsa_ctx* ctx, const float* x, const int32_t* idx, int n, int8_t* q,
                               float* scale, const float* shift, const float* mscale);

/* Which places of a head form plane i of a rotation over `rot` places. */
typedef enum {
  HSA_ROPE_INTERLEAVED = 0, /* (2i, 2i + 1) */
  HSA_ROPE_HALF = 1         /* (i, i + rot / 2) */
} hsa_rope_layout;

/* How frequencies are scaled for contexts longer than the model was trained on. */
typedef enum {
  HSA_ROPE_PLAIN = 0,  /* f_i = base^(-2 i / dim) */
  HSA_ROPE_LINEAR = 1, /* f_i / factor (positions interpolated) */
  HSA_ROPE_BASE = 2,   /* base * factor^(dim / (dim - 2)) in place of base (dim > 2) */
  HSA_ROPE_PARTS = 3   /* by the turns r = orig_len f_i / 2 pi of a plane over the trained
                          length: f_i / factor for r <= slow, f_i for r >= fast, and their
                          mean weighted by (r - slow) / (fast - slow) in between */
} hsa_rope_scaling;

/* A rotary table: up to three position axes (e.g. frame, row, column of a
 * video token), axis x turning dims[x] / 2 planes of its own, in axis order.
 * Each axis has frequencies over its own dims[x]. */
typedef struct {
  int n_axes;      /* 1..3 */
  int dims[3];     /* rotated places per axis: even, >= 2; their sum rot is <= 128 */
  double base;     /* > 1 */
  int scaling;     /* hsa_rope_scaling */
  double factor;   /* >= 1; not read by HSA_ROPE_PLAIN */
  double orig_len; /* > 0, HSA_ROPE_PARTS */
  double fast, slow; /* fast > slow >= 0, HSA_ROPE_PARTS */
  double amp;      /* multiplies cosines and sines (1: a pure rotation) */
} hsa_rope_cfg;

/*
 * Table of a rotary position embedding: table[p][i] = amp (cos, sin)(pos[p][axis(i)] f_i).
 * Angles are counted in 64-bit fractions of a turn: an entry is within 2^-21 amp of
 * the exact one at every int32 position (an absolute bound: a small sine keeps fewer bits).
 *   cfg (host);  pos (device) int32 [P, n_axes], or NULL with one axis: row p has position p;
 *   table (device) fp32 [P, rot / 2, 2] out.   P >= 0.
 */
hsa_status hsa_rope_table(hsa_ctx* ctx, const hsa_rope_cfg* cfg, const int32_t* pos, int P,
                          float* table);

/*
 * Rotate the first `rot` places of every head: with (u, v) plane i of a head of
 * row m and (c, s) = table[pos[m]][i],
 *   out = (u c - v s, v c + u s),  or with `inverse` (u c + v s, v c - u s),
 * the other places of the head copied.  The inverse is also the gradient.
 *   x, out (device) type HSA_BF16 or HSA_F32, n rows of `heads` heads of D/H places, rows
 *   ld_x / ld_out apart (multiples of 16 bytes); out may be x;
 *   table (device) fp32 [P, rot / 2, 2];  pos (device) int32 [n] table rows, or NULL: row m
 *   uses table row m;  rot a multiple of 16, 16 <= rot <= D/H;  heads >= 1.
 * A row whose table row is outside [0, P) is left unwritten and reported by
 * hsa_sync_check (HSA_ERR_DEVICE_CHECK).
 */
hsa_status hsa_rope(hsa_ctx* ctx, const void* x, int64_t ld_x, int type, int n, int heads,
                    const float* table, int P, int rot, const int32_t* pos, int layout,
                    int inverse, void* out, int64_t ld_out);

/* What the RMS norm of queries and keys runs over. */
typedef enum { HSA_NORM_NONE = 0, HSA_NORM_HEAD = 1, HSA_NORM_ROW = 2 } hsa_qk_norm;

typedef struct {
  int norm;           /* hsa_qk_norm: each head's D/H places, or the row's D */
  const float* w_q;   /* (device) fp32 [D/H] (HEAD) or [D] (ROW) weights, NULL: 1 */
  const float* w_k;   /* same, keys */
  float eps;          /* x / sqrt(mean(x^2) + eps) * w;  >= 0 */
  const float* table; /* (device) fp32 [P, rot / 2, 2], NULL: no rotation */
  int P;              /* table rows */
  int rot;            /* as hsa_rope */
  int layout;         /* hsa_rope_layout */
} hsa_qk_rope;

/*
 * Norm and rotation of fresh queries and keys, and the cache write, in one pass:
 *   q[m]              = rot(norm(q_in[m]))
 *   k_cache[idx[m]]   = rot(norm(k_in[m]))
 *   v_cache[idx[m]]   = v_in[m]
 * norm then rotation in fp32, rounded once to bf16.
 *   idx (device) int32 [n] distinct cache rows in [0, N), or NULL: row m;
 *   pos (device) int32 [n] table rows, or NULL: the cache row (a token's place in the latent);
 *   q (device) bf16 [n, D] out, NULL: no queries;  q_in (device) bf16, rows ld_q apart, NULL: q in place;
 *   k_cache (device) bf16 [N, D], NULL: no keys;   k_in (device) bf16, rows ld_k apart, NULL: the
 *   cache rows in place (after hsa_qkv_project; idx must then ascend);
 *   v_cache (device) bf16 [N, D] and v_in, rows ld_v apart: both or neither.
 *   ld_* multiples of 8, >= D; 0 <= n <= N; D <= 10240 (HSA_ERR_SHAPE beyond).
 * q may be q_in; no other output may overlap an input.  A row with an index or table row out of range
 * (or, with keys in place, an index not above the one before it) is skipped whole: its cache rows
 * keep their key and value, its q row is zeroed if that was to be written, and
 * hsa_sync_check reports it.  (Order is judged by neighbours alone: in place, a reported
 * list that names a row twice may have turned that row twice.)
 */
hsa_status hsa_qk_norm_rope(hsa_ctx* ctx, const hsa_qk_rope* a, const int32_t* idx,
                            const int32_t* pos, int n, const void* q_in, int64_t ld_q, void* q,
                            const void* k_in, int64_t ld_k, void* k_cache, const void* v_in,
                            int64_t ld_v, void* v_cache);

/* Cross-attention of B sequences of queries to B padded sequences of encoder states. */
typedef struct {
  const void* q;           /* (device) bf16 [n, D]: the sequences' queries one after another */
  const int32_t* q_start;  /* (device) int32 [B + 1], ascending, in [0, n]: sequence b owns rows
                              q_start[b] .. q_start[b + 1] - 1; NULL: n / B rows each, n % B == 0 */
  int n, B;                /* n >= 0, B >= 1 */
  const void* k;           /* (device) bf16 [B, S, kv_heads * D/H], rows ld_k apart, */
  const void* v;           /*   sequences bs_k apart (elements); v likewise */
  int64_t ld_k, bs_k, ld_v, bs_v; /* multiples of 8; ld >= kv_heads * D/H; bs >= 0 (0: shared) */
  int S;                   /* padded key count, 1 .. 2^26 */
  int kv_heads;            /* divides H: query head h reads key head h / (H / kv_heads) */
  const int32_t* kv_len;   /* (device) int32 [B] keys of each sequence, in [0, S]; NULL: S */
  const uint8_t* kv_mask;  /* (device) uint8 [B, S], 0 = key not seen; NULL: all seen */
  float scale;             /* of the scores; 0: 1 / sqrt(D/H) */
  void* o;                 /* (device) bf16 [n, D] out, rows of the sequences only */
} hsa_cross_args;

/*
 * o[m] = sum_j softmax_j(scale q[m] . k[b][j]) v[b][j] per head, over the keys
 * j < kv_len[b] that kv_mask[b] lets through; b is the sequence of row m.  Statistics and sums in
 * fp32; the weights fp32 where sequences have few queries on average (n (H / kv_heads) <= 4 B),
 * else rounded to bf16 for their product with v.  A row without any key gets zeros.  What lies in unseen keys and values (NaN,
 * infinities) never reaches the result.  Rows of no sequence are left as they were.
 * q_start, kv_len and kv_mask are read on the device, so a captured graph
 * serves later prompts of other lengths.  A kv_len outside [0, S] is clamped, a q_start
 * that descends or leaves [0, n] is clamped; both are reported by hsa_sync_check.
 */
hsa_status hsa_cross_attention(hsa_ctx* ctx, const hsa_cross_args* a);

/* One transformer block's weights in signed 8 bits, as hsa_quant_rows makes them
 * from the bf16 weights (a row per output channel, rows dense), with their scales. */
typedef struct {
  const int8_t *w_qkv, *w_o, *w_1, *w_2;         /* (device) int8 [3D, D], [D, D], [F, D], [D, F] */
  const float *s_qkv, *s_o, *s_1, *s_2;          /* (device) fp32 [3D], [D], [F], [D] */
} hsa_layer_weights_quant;

/* What a block may have beyond hsa_layer_forward; zero-initialise and set what is wanted. */
typedef struct {
  const float* mod;                  /* as hsa_layer_forward_cond */
  const hsa_cross_attn* xa;          /* as hsa_layer_forward_cond (weights in bf16) */
  const int32_t* txt_len;            /* (device) int32 [1]: text tokens that count, in [0, n_txt]; NULL: n_txt */
  const uint8_t* txt_mask;           /* (device) uint8 [n_txt], 0 = not seen; NULL: all seen */
  const hsa_qk_rope* qk;             /* norm and rotation of the self-attention's Q and K; a token's
                                        table row is its place in the latent */
  const hsa_layer_weights_quant* wq; /* the four products in 8 bits; NULL: bf16 weights w */
} hsa_block_ext;

/*
 * hsa_layer_forward_cond with the operators above inside the block:
 *  - qk: Q and the fresh K rows are normalised and rotated (hsa_qk_norm_rope, in
 *    place) between the QKV product and the attention, so the cache holds rotated keys;
 *  - txt_len / txt_mask: the text cross-attention is hsa_cross_attention over the tokens
 *    that count, read on the device: a captured step serves prompts of any length up to n_txt;
 *  - wq: LN rows, attention output and MLP hidden rows are quantised per token
 *    (hsa_ln_gather_quant, hsa_quant_rows) and multiplied in 8 bits; w is not read and may be NULL.
 * ext == NULL or all members NULL is hsa_layer_forward.  Errors as
 * hsa_layer_forward_cond and the calls named; with wq also HSA_ERR_SHAPE for
 * D > 5120 or F > 36864.
 */
hsa_status hsa_layer_forward_ext(hsa_ctx* ctx, const hsa_layer_weights* w, const hsa_block_ext* ext,
                                 float* x, const int32_t* idx, int n, void* k_cache, void* v_cache);

/*
 * hsa_step with every layer run by hsa_layer_forward_ext: ext is a host array of L
 * entries, read during the call only, or NULL.  w->layers may be NULL when every
 * entry has wq.
 */
hsa_status hsa_step_ext(hsa_ctx* ctx, const hsa_model_weights* w, const hsa_state* s,
                        const hsa_block_ext* ext, int i, float sigma_i, float sigma_next,
                        int regroup);

/*
 * Group selection without any device allocation.  The paper has no
 * counterpart: this is a service for callers that cannot call cudaMalloc,
 * such as a host framework that owns all device memory through its own pool
 * and forbids a library to allocate, or a latency-critical serving loop
 * where cudaMalloc's implicit device synchronisation would stall other work.
 *
 * Same result as hsa_select_groups (scores, then exact group assignment with
 * ties broken by token index), but it needs no context: the scores and cut
 * keys live in one static device array of the library, sized for at most
 * HSA_SELECT_STATIC_MAX_N tokens (512 KiB of scores + 64 B of cut keys +
 * 256 B for the error flag), which every GPU that loads the library holds
 * until the process exits.
 *   v_prev, v_cur (device) fp32 [N, 16];  counts (host) n_1..n_K, sum == N;
 *   g (device) uint8 [N] out;  stream cudaStream_t (NULL = legacy default).
 * Returns HSA_ERR_SCRATCH_LIMIT when N > HSA_SELECT_STATIC_MAX_N, and the
 * other argument errors of hsa_create / hsa_select_groups; there is no
 * message string.  Calls no cudaMalloc or cudaFree.  The first call on a
 * device looks up the array's device address (cudaGetSymbolAddress) with
 * that device current; make that first call before any stream capture.  The
 * address belongs to the device's primary context: after cudaDeviceReset the
 * next call finds a new context and looks the address up again (make that
 * call, too, outside stream capture).
 * All calls share the array and it keeps the last call's contents; calls
 * that overlap on the GPU race on it.  Device-side checks (a NaN score) are
 * not reported by this call.
 */
#define HSA_SELECT_STATIC_MAX_N 131072
hsa_status hsa_select_groups_static(const float* v_prev, const float* v_cur, int N,
                                    const int* counts, int K, uint8_t* g, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HSA_H_ */
