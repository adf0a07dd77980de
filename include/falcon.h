/*
 * falcon.h — C ABI of the GB300 Falcon fast-weight forward library
 * (libfalcon.so, built for sm_103a).
 *
 * The method: a fixed-size fast-weight state S (d_k x d_v, fp32) is written
 * once per token by one normalised online gradient step on the
 * prefix-aligned pair (x_t, v_t) = (phi(k_{t-1}), v_t), with a shrinkage
 * decay gamma_t = 1 - lambda_t kept >= eps_gamma, and read after the write,
 * o_t = S_t^T q_t.  Sources, cited by page title and section:
 *   [FW]  "Falcon 家族重新对齐 fast-weight 记忆" (zhouql-dev explainer):
 *         本质 (pair alignment), Falcon 家族 (variants, knobs),
 *         三种等价形式 (recurrent / masked-parallel / chunked forms).
 *   [JC]  "给记忆装一个“及时纠错”的开关" (long write-up):
 *         把记忆更新变成一次梯度下降 (gradient step, NLMS step),
 *         Falcon家族六个变体各管一段 (1/2/3 and A variants, batched solve),
 *         数学上的稳定阀门:正衰减钳制 (decay floor eps_gamma),
 *         三种视角看同一个更新 (the three forms, WY representation).
 *
 * Update of one step t (window W(t) = existing pairs among the last W;
 * W = 1 except for Falcon-3/3A; n_t = |W(t)|; e_t = mean ||x_j||^2 over W(t)):
 *   gamma_t = clamp(1 - lambda_t, eps_gamma, 1)
 *   eta_t   = beta_t / (eps + e_t)          (scalar, or per value channel)
 *   Z       = gamma_t S_{t-1}
 *   regression (1, 2, 3):  S_t = Z + (1/n_t) sum_j x_j (eta_t * (v_j - Z^T x_j))^T
 *   additive  (1A, 2A, 3A): S_t = Z + (1/n_t) sum_j x_j (eta_t * v_j)^T
 *   o_t = S_t^T q_t
 * The pair of a token whose global index (carry pos + local index) is < 1
 * does not exist (it would need the key before the sequence) and writes
 * nothing; a step with no existing pair only decays.
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library never allocates device memory.  Scratch memory, where needed,
 *     is the caller's `workspace` of at least the size the matching
 *     *_workspace_size() call returns, 256-byte aligned.
 *   - Layouts are dense row-major: q, k [B, T, H, dk]; v, o [B, T, H, dv];
 *     beta [B, T, H] (Falcon-2/2A: [B, T, H, dv]); lambda [B, T, H].
 *     q, k, v, o, carry k_prev / win_x / win_v use the params' dtype
 *     (bf16 or fp32); beta, lambda and the state S are fp32; pos is int64.
 *     q and k are the features phi(q), phi(k): the caller applies phi.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t passed as
 *     void*; NULL = the legacy default stream).  Errors found on the host
 *     (arguments, shapes) return before anything is enqueued.
 *   - Return value: FALCON_OK (0) or a negative FALCON_ERR_* code; no
 *     exception crosses the ABI.  FALCON_ERR_CUDA reports a launch error
 *     (cudaGetLastError after the launches).
 *   - Inputs must not overlap outputs.  The chunk forward reads carry_in
 *     and writes carry_out; the two must not overlap (use two carries).
 *     The recurrent step updates its carry in place.
 */
#ifndef FALCON_H
#define FALCON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Variants [FW Falcon 家族; JC Falcon家族六个变体各管一段]:
 * 1 scalar step, 2 per-value-channel step, 3 sliding-window mini-batch of the
 * last `window` pairs (window-averaged); "A" = inner-product objective,
 * additive write. */
typedef enum {
  FALCON_1 = 0,
  FALCON_1A = 1,
  FALCON_2 = 2,
  FALCON_2A = 3,
  FALCON_3 = 4,
  FALCON_3A = 5
} falcon_variant_t;

typedef enum { FALCON_BF16 = 0, FALCON_F32 = 1 } falcon_dtype_t;

/* Which key a value is paired with.  PREFIX (the method): pair t is
 * (phi(k_{t-1}), v_t) [FW 本质; JC 一个被忽略的时间差], x_0 the carried k_prev,
 * and a pair with global index < 1 does not exist.  SAME_STEP (the ablation
 * the pages set against it, the usual delta-rule pairing): pair t is
 * (phi(k_t), v_t), every pair with global index >= 0 exists and k_prev is
 * not read (it is still written to a carry).  Window rings hold zeros for
 * pairs that do not exist. */
typedef enum { FALCON_PAIR_PREFIX = 0, FALCON_PAIR_SAME_STEP = 1 } falcon_pairing_t;

/* Steps either side of the path, done by the library when asked
 * [FW 三种等价形式 (phi(Q), phi(K)); JC 把记忆更新变成一次梯度下降]:
 * L2NORM_QK: q and k are raw projections; the feature map phi is the
 *   per-token L2 normalisation x / max(|x|, 1e-12) (fp32, then the dtype).
 *   Carried keys (k_prev, win_x) hold features phi(k).
 * GATE_LOGITS: beta and lambda hold logits: beta = sigmoid(b) and
 *   lambda = sigmoid(a), i.e. gamma = 1 - lambda = sigmoid(-a) before the
 *   eps_gamma floor.
 * The chunk forward applies them in one pass over the inputs into its
 * workspace (falcon_workspace_size counts it), the varlen forward in its
 * gather pass, the recurrent step inside its kernel.  The backward and the
 * masked-parallel reference take features and gates (prologue must be 0). */
typedef enum {
  FALCON_PROLOGUE_L2NORM_QK = 1,
  FALCON_PROLOGUE_GATE_LOGITS = 2
} falcon_prologue_t;

/* Kernel family for the chunk forward.  AUTO picks the tensor-core path
 * (tcgen05 + TMEM + TMA) when it supports the shape, else the window
 * recurrence for Falcon-3 when it does, else the portable CUDA-core chunk
 * path.  GENERIC, TC and SCAN force one (TC and SCAN return
 * FALCON_ERR_UNSUPPORTED for shapes they do not cover).  The tensor-core
 * path covers Falcon-1, 1A, 2 and 2A with bf16 inputs, chunk 64 and
 * d_k = d_v in {64, 128}, Falcon-3A with bf16, chunk 64, d = 64 and
 * 2 <= window <= 16, and Falcon-3 with bf16, chunk 64, d = 64 and
 * 2 <= window <= 9.  SCAN (Falcon-3, 2 <= window <= 8, d_k in {32, 64},
 * d_v a multiple of 16, bf16 or fp32) walks the steps with the state's
 * value columns spread over threads and ignores `chunk`.  TC and SCAN need
 * q, k, v, o and the carried keys / values on 16-byte boundaries: AUTO falls
 * back to the portable path for misaligned tensors, a forced TC or SCAN
 * returns FALCON_ERR_INVALID_ARG. */
typedef enum {
  FALCON_IMPL_AUTO = 0,
  FALCON_IMPL_GENERIC = 1,
  FALCON_IMPL_TC = 2,
  FALCON_IMPL_SCAN = 3
} falcon_impl_t;

enum {
  FALCON_OK = 0,
  FALCON_ERR_INVALID_ARG = -1,   /* null pointer, bad enum, bad size */
  FALCON_ERR_UNSUPPORTED = -2,   /* shape or combination not supported */
  FALCON_ERR_WORKSPACE = -3,     /* workspace missing, too small or misaligned */
  FALCON_ERR_CUDA = -4,          /* a CUDA call or launch failed */
  FALCON_ERR_TIMEOUT = -5        /* a bounded device-side wait expired */
};

typedef struct {
  int32_t B, T, H;      /* batch, tokens in this call, heads (all >= 1; T >= 0 for chunk fwd) */
  int32_t dk, dv;       /* key / value head dims: 16, 32, 64 or 128 */
  int32_t chunk;        /* chunk length of the chunked form: 16, 32 or 64 */
  int32_t window;       /* Falcon-3/3A window W in [1, 64]; ignored otherwise */
  float eps;            /* NLMS regulariser, > 0 (e.g. 1e-6) */
  float eps_gamma;      /* positive-decay floor, in (0, 1] (e.g. 1e-3) */
  int32_t variant;      /* falcon_variant_t */
  int32_t dtype;        /* falcon_dtype_t of q, k, v, o and the carried keys/values */
  int32_t impl;         /* falcon_impl_t (chunk forward only) */
  int32_t pairing;      /* falcon_pairing_t (0 = prefix alignment) */
  int32_t prologue;     /* falcon_prologue_t flags (0 = inputs are features and gates) */
} falcon_params_t;

/* Decode carry: everything the next call needs to continue a sequence.
 * All pointers are device pointers owned by the caller.
 *   S      [B, H, dk, dv] fp32   fast-weight state
 *   k_prev [B, H, dk]     dtype  last key consumed (x of the next pair)
 *   win_x  [B, H, W-1, dk] dtype  window ring of previous pairs' keys  (3/3A, W > 1)
 *   win_v  [B, H, W-1, dv] dtype  window ring of previous pairs' values (3/3A, W > 1)
 *   pos    [B, H]         int64  tokens consumed so far
 * The pair with global index p lives in ring slot p mod (W-1); slots whose
 * pair does not exist (p < 1; with same-step pairing p < 0) hold zeros.  As
 * an input, a NULL carry (or NULL fields) means a fresh sequence: S = 0,
 * k_prev = 0, pos = 0; win_* may be NULL only when no earlier pair exists
 * (pos <= 1, with same-step pairing pos == 0) for every (b, h). */
typedef struct {
  float* S;
  void* k_prev;
  void* win_x;
  void* win_v;
  int64_t* pos;
} falcon_carry_t;

/* Bytes of workspace falcon_chunk_fwd needs for these params (0 if none). */
size_t falcon_workspace_size(const falcon_params_t* p);

/* Chunk-parallel (SSD-style) forward [FW 三种等价形式; JC 三种视角看同一个更新]:
 * the sequence is cut into chunks of `chunk` tokens; inside a chunk the
 * rank-one updates are gathered in the WY representation (Gram matrix of
 * the shifted keys, unit lower-triangular solve), and the state S is carried
 * across chunks with the cumulative log-decay.  Computes o [B, T, H, dv] for
 * the T tokens and, when carry_out is non-NULL, the carry after them
 * (carry_out->S holds the final state S_T; every non-NULL carry_out field
 * is written).  carry_in == NULL starts a fresh sequence.
 * Errors: FALCON_ERR_INVALID_ARG (null q/k/v/beta/lambda/o with T > 0, bad
 * params, carry_in/carry_out overlap), FALCON_ERR_UNSUPPORTED (dims outside
 * {16,32,64,128}, window outside [1,64], forced TC on an unsupported shape),
 * FALCON_ERR_WORKSPACE, FALCON_ERR_CUDA. */
int falcon_chunk_fwd(const falcon_params_t* p, const void* q, const void* k, const void* v,
                     const float* beta, const float* lambda, const falcon_carry_t* carry_in,
                     void* o, falcon_carry_t* carry_out, void* workspace, size_t workspace_bytes,
                     void* stream);

/* falcon_chunk_fwd, plus timing hooks: records the caller's CUDA events
 * (cudaEvent_t handles passed as void*) on `stream`, events[0] before the
 * first kernel of the call and events[i] right after kernel i.  n_events must
 * equal the launch count falcon_chunk_fwd_plan reports plus one.  The work
 * done is exactly that of falcon_chunk_fwd.  Errors: those of
 * falcon_chunk_fwd, and FALCON_ERR_INVALID_ARG for a bad event list. */
int falcon_chunk_fwd_timed(const falcon_params_t* p, const void* q, const void* k, const void* v,
                           const float* beta, const float* lambda, const falcon_carry_t* carry_in,
                           void* o, falcon_carry_t* carry_out, void* workspace,
                           size_t workspace_bytes, void* stream, void* const* events,
                           int32_t n_events);

/* falcon_chunk_fwd for callers that cannot allocate device memory.  The
 * pages have no counterpart to this entry point; it exists for hosts that
 * pass a kernel library only tensors and a stream (plugin interfaces without
 * an allocator, services whose memory budget is fixed once they start
 * serving), which therefore cannot supply falcon_chunk_fwd's workspace.
 *
 * The scratch lives in a fixed 32 MiB array inside the library's device
 * image, held by every device that loads the library until the process
 * exits.  The call itself allocates nothing (no cudaMalloc/cudaFree).
 * Covered: Falcon-1 and Falcon-1A with prologue 0 on the tensor-core path (bf16,
 * d_k = d_v in {64, 128}, chunk 64; see falcon_chunk_fwd_plan) whose
 * falcon_workspace_size is at most 32 MiB: B * H * ceil(T / 64) <= 1927 at
 * d = 64 (17 KB of scratch per chunk) and <= 992 at d = 128 (33 KB per
 * chunk).  Larger problems return FALCON_ERR_WORKSPACE, other variants and
 * shapes FALCON_ERR_UNSUPPORTED (falcon_chunk_fwd serves them; its
 * falcon_workspace_size says whether they need a workspace, 0 for the
 * portable CUDA-core path).  Both are found on the host before anything is
 * enqueued.
 * Every call looks up the array's device address (the first call on a
 * device may also load the library's device code there); make that first
 * call before any stream capture.  All calls share the one array: calls that
 * overlap on the GPU (other streams, other host threads) race and must be
 * serialised by the caller.  The status of the last call is read with
 * falcon_workspace_status(NULL, stream).  Arguments, outputs and other
 * errors as falcon_chunk_fwd. */
int falcon_chunk_fwd_noalloc(const falcon_params_t* p, const void* q, const void* k,
                             const void* v, const float* beta, const float* lambda,
                             const falcon_carry_t* carry_in, void* o, falcon_carry_t* carry_out,
                             void* stream);

/* Bytes of workspace falcon_chunk_fwd_varlen needs for these params
 * (p->B = number of sequences, p->T = their maximum length). */
size_t falcon_varlen_workspace_size(const falcon_params_t* p);

/* Chunk forward over packed sequences of different lengths (varlen), as
 * the chunked framework is used for training [FW 三种等价形式; JC
 * 三种视角看同一个更新].  cu_seqlens (device int32 [B + 1], non-decreasing,
 * cu_seqlens[0] = 0, cu_seqlens[B] = total_tokens) delimits sequence b's
 * tokens [cu_seqlens[b], cu_seqlens[b+1]); every length must be <= p->T.
 * q, k [total_tokens, H, dk], v, o [total_tokens, H, dv], beta
 * [total_tokens, H] (or [total_tokens, H, dv]), lambda [total_tokens, H];
 * carry_in / carry_out are per sequence ([B, H, ...], as for
 * falcon_chunk_fwd; NULL carry_in = every sequence fresh).  On the
 * Falcon-1 / 1A d = 64 tensor-core path (bf16, rows on 16-byte boundaries)
 * the kernels read and write the packed rows in place and take only the
 * chunks that hold tokens (p->prologue applied inside them).  Otherwise the
 * tokens are laid out as a [B, p->T] batch in the workspace (applying
 * p->prologue on the way); positions past a sequence's end get beta = 0 and
 * lambda = 0, steps that neither write nor decay, so each sequence's state
 * after p->T steps is its state after its own length; the same kernel
 * family as falcon_chunk_fwd then runs, and the outputs go back to the
 * packed layout.  carry_out's k_prev, pos and window ring are those after
 * each sequence's own last token.  Errors as falcon_chunk_fwd. */
int falcon_chunk_fwd_varlen(const falcon_params_t* p, const int32_t* cu_seqlens, int64_t total_tokens,
                            const void* q, const void* k, const void* v, const float* beta,
                            const float* lambda, const falcon_carry_t* carry_in, void* o,
                            falcon_carry_t* carry_out, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Which kernel family falcon_chunk_fwd uses for these params
 * (FALCON_IMPL_GENERIC, FALCON_IMPL_TC or FALCON_IMPL_SCAN, written to *impl_out) and how many
 * kernels one call enqueues (*launches_out).  Host-only; either output
 * pointer may be NULL.  Returns FALCON_OK or the error the call would give
 * for these params. */
int falcon_chunk_fwd_plan(const falcon_params_t* p, int32_t* impl_out, int32_t* launches_out);

/* Recurrent form, one token per sequence [FW 三种等价形式 (inference form,
 * O(1) state per step); JC 三种视角看同一个更新]: p->T must be 1.  q, k, v
 * are [B, 1, H, d], beta / lambda [B, 1, H] (or [B, 1, H, dv]).  Updates the
 * carry in place (S, k_prev <- k, window ring push, pos += 1) and writes
 * o [B, 1, H, dv].  carry, carry->S, carry->k_prev and carry->pos are
 * required; win_x / win_v are required for Falcon-3/3A with window > 1.
 * Errors: FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED, FALCON_ERR_CUDA. */
int falcon_recurrent_step(const falcon_params_t* p, const void* q, const void* k, const void* v,
                          const float* beta, const float* lambda, falcon_carry_t* carry, void* o,
                          void* stream);

/* Bytes of workspace falcon_masked_parallel_ref_gpu needs. */
size_t falcon_masked_parallel_workspace_size(const falcon_params_t* p);

/* Masked-parallel form of a fresh sequence [FW 三种等价形式 (linear attention
 * (phi(Q) phi(K)^T (.) M) V without denominator); JC 三种视角看同一个更新]:
 * the whole T x T decay mask from the global cumulative log-decay and, for
 * the regression variants, one unit lower-triangular solve over all T
 * steps (T*W unknowns for Falcon-3).  fp32 arithmetic, quadratic cost: a
 * reference for tests, limited to T <= 1024 (T*window <= 2048).  Writes
 * o [B, T, H, dv] and S_final [B, H, dk, dv] (fp32).
 * Errors: FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED (T too large),
 * FALCON_ERR_WORKSPACE, FALCON_ERR_CUDA. */
int falcon_masked_parallel_ref_gpu(const falcon_params_t* p, const void* q, const void* k,
                                   const void* v, const float* beta, const float* lambda, void* o,
                                   float* S_final, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Bytes of workspace falcon_backward needs for these params (0 when the
 * params are invalid or not covered). */
size_t falcon_backward_workspace_size(const falcon_params_t* p);

/* Gradient of the chunk forward, for training in the chunked framework
 * [FW 三种等价形式; JC 三种视角看同一个更新] (the pages give the forward
 * only; the backward is the chain rule through the update written at the
 * top of this header, Falcon-3/3A's window of pairs included).  For the loss
 * L = <o, dO> + <S_T, dS_final> of falcon_chunk_fwd(p, q, k, v, beta,
 * lambda, carry_in) it writes
 *   dq, dk [B, T, H, dk], dv [B, T, H, dv] (the params' dtype),
 *   dbeta (the shape of beta), dlambda [B, T, H] (fp32),
 * and, through the fields of dcarry (NULL, or any field NULL, skips them):
 *   dcarry->S      [B, H, dk, dv] fp32  gradient of carry_in->S,
 *   dcarry->k_prev [B, H, dk] dtype      gradient of carry_in->k_prev,
 *   dcarry->win_x  [B, H, W-1, dk], dcarry->win_v [B, H, W-1, dv] dtype
 *                  gradients of the carried window ring (Falcon-3/3A, W > 1;
 *                  both or neither; slot layout as in the carry);
 * dcarry->pos is ignored.  dO has the shape and dtype of o; dS_final (fp32
 * [B, H, dk, dv]) may be NULL (zero).  carry_in supplies S, k_prev, the
 * window ring and pos as for the forward (NULL = fresh sequence); a key or
 * ring entry that no existing pair reads gets a zero gradient.  The decay
 * clamp passes the gradient where eps_gamma <= 1 - lambda <= 1.  The forward
 * is recomputed inside (states kept at every 64th step in the workspace), so
 * o need not be saved.  Covered: every variant, both pairings, bf16 or fp32,
 * d_k = d_v in {32, 64, 128}; Falcon-3/3A with W up to 64 (up to 34 at
 * d = 128, the window kernel's shared memory); any T >= 0 (chunk and impl
 * are ignored).  Falcon-1/1A at d = 64 run a chunked kernel, Falcon-3/3A
 * and d = 128 a step-by-step kernel that carries the window's key and value
 * gradients in a ring, the rest a step-by-step one-pair kernel.  Gradients
 * must not overlap inputs or one another.  The chunked kernel with bf16
 * inputs runs its products on the tensor cores with bounded waits: a wait
 * that runs out is recorded in the workspace's status word and read with
 * falcon_workspace_status, as for the chunk forward.
 * Errors: FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED (other dims, the
 * prologue, a window past the limit), FALCON_ERR_WORKSPACE, FALCON_ERR_CUDA. */
int falcon_backward_carry(const falcon_params_t* p, const void* q, const void* k, const void* v,
                          const float* beta, const float* lambda, const falcon_carry_t* carry_in,
                          const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                          float* dbeta, float* dlambda, const falcon_carry_t* dcarry, void* workspace,
                          size_t workspace_bytes, void* stream);

/* falcon_backward_carry with dcarry = {dS_in, dk_prev} (no ring gradients):
 * dS_in [B, H, dk, dv] fp32 and dk_prev [B, H, dk] dtype may each be NULL. */
int falcon_backward(const falcon_params_t* p, const void* q, const void* k, const void* v,
                    const float* beta, const float* lambda, const falcon_carry_t* carry_in,
                    const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                    float* dbeta, float* dlambda, float* dS_in, void* dk_prev, void* workspace,
                    size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Softmax-attention layers (the full-attention layers a stack of Falcon
 * layers is interleaved with; the pages have no counterpart).  Four
 * operators forward: falcon_qk_norm_rope over a token's
 * queries and keys, falcon_attn_prompt over whole packed prompts,
 * falcon_kv_append into a paged cache held in 8 bits, falcon_attn_decode of
 * one token per sequence over that cache.  Two for training, the gradients of
 * the first two: falcon_attn_prompt_backward and falcon_qk_norm_rope_backward.
 *
 * Layouts: q [tokens, Hq, d], k and v [tokens, Hkv, d] in the params' dtype,
 * tokens of all sequences packed one after the other, heads and dims dense,
 * q_stride / k_stride / v_stride / o_stride elements from one token to the
 * next (0 = dense; larger for slices of a fused projection).  Results and
 * workspaces must not lie over one another or over what a call reads (the cache
 * among it).  Query head h
 * reads key / value head h / (Hq / Hkv).  FALCON_ERR_UNSUPPORTED past 2^31 - 1024
 * rows or keys of one sequence, k_tokens above that, or (Hq + Hkv) d above
 * 2^31 - 1; for attn_decode also past 2^31 units of 64 keys in the batch. */

/* Which dims of a head form the rotated pairs: HALF (i, i + rot/2),
 * INTERLEAVED (2i, 2i + 1), i < rot/2. */
typedef enum { FALCON_ROPE_HALF = 0, FALCON_ROPE_INTERLEAVED = 1 } falcon_rope_layout_t;

typedef struct {
  int32_t B;            /* sequences (kv_append, attn_decode, attn_prompt) */
  int32_t Hq, Hkv;      /* query heads, key / value heads (Hkv divides Hq) */
  int32_t d;            /* head dim: 16, 32, 64 or 128 */
  int32_t dtype;        /* falcon_dtype_t of q, k, v, o */
  int32_t qk_norm;      /* nonzero: RMS norm of each head row (qk_norm_rope, kv_append) */
  int32_t rot;          /* leading dims of a head that are rotated: even, 0 .. d */
  int32_t rope_layout;  /* falcon_rope_layout_t */
  int32_t rope_rows;    /* positions the rotary table holds */
  int32_t page;         /* tokens per cache page: 16, 32, 64 or 128 */
  int32_t num_pages;    /* pages in the cache */
  int32_t max_pages;    /* columns of block_table */
  int32_t max_q;        /* no sequence brings more tokens than this to the call; any larger bound will do */
  int32_t max_k;        /* no sequence has more keys than this (attn_decode); any larger bound will do */
  float norm_eps;       /* > 0 where qk_norm is set */
  float scale;          /* of the scores; 0 = 1 / sqrt(d) */
  int64_t tokens;       /* rows of q (qk_norm_rope, attn_prompt) or of the new k, v (kv_append) */
  int64_t k_tokens;     /* rows of k, v (attn_prompt) */
  int64_t q_stride, k_stride, v_stride, o_stride;
} falcon_attn_params_t;

/* The paged cache.  Page p, head h, slot s of K is the row
 * k[((p Hkv + h) page + s) d ..] of e4m3 codes; its value is code times the
 * power of two of the scale byte k_scale[p Hkv + h] (e8m0: 2^(byte - 127)).
 * V the same.  k and v 16-byte aligned.  Sequence b's token t sits in page
 * block_table[b max_pages + t / page], slot t % page. */
typedef struct {
  uint8_t* k;        /* [num_pages, Hkv, page, d] */
  uint8_t* v;        /* [num_pages, Hkv, page, d] */
  uint8_t* k_scale;  /* [num_pages, Hkv] */
  uint8_t* v_scale;  /* [num_pages, Hkv] */
} falcon_kv_cache_t;

/* Rotary table [rows, rot/2, 2] fp32: (cos, sin) of position times
 * inv_freq[i] (device fp64 [rot/2]), times mscale; angles in 64 bits.  Long
 * contexts are scaled through inv_freq and mscale. */
int falcon_rope_table(const double* inv_freq, int32_t rot, int32_t rows, float mscale, float* table,
                      void* stream);

/* Norm of queries and keys for each head and rotation, one pass:
 *   y = x / sqrt(mean(x^2) + norm_eps) * w     (qk_norm; w_q, w_k fp32 [d], NULL = ones)
 *   (a, b) -> (a c - b s, b c + a s)           on the rot/2 pairs, (c, s) = table[position, i]
 * fp32 arithmetic, rounded once to the dtype (a row whose sum of squares passes
 * fp32's range gives 0).  q -> q_out (row stride
 * o_stride, 0 = dense), k -> k_out (dense); q or k may be NULL (skipped).  An
 * output may be its own input when their strides agree (in place, also inside
 * a fused projection), and its rows must not share a byte with another
 * operand's otherwise.  (Operands of one stride may lie between one another's
 * rows, here and in falcon_attn_prompt and falcon_attn_decode.)  positions: int64 [tokens], needed with
 * rot > 0, as is table; the rotated dims of a token whose position is not
 * in [0, rope_rows) are NaN.  Errors: FALCON_ERR_INVALID_ARG,
 * FALCON_ERR_UNSUPPORTED, FALCON_ERR_CUDA. */
int falcon_qk_norm_rope(const falcon_attn_params_t* p, const void* q, const void* k, const float* w_q,
                        const float* w_k, const int64_t* positions, const float* table, void* q_out,
                        void* k_out, void* stream);

/* Append new keys and values to the cache, with the norm (qk_norm, w_k) and
 * the rotation (rot, table) of falcon_qk_norm_rope applied to the keys on
 * the way.  cu_new (int32 [B + 1], as cu_seqlens) delimits each sequence's
 * rows of k and v, ctx_lens (int32 [B]) holds its tokens cached before; new
 * token i has position ctx_lens[b] + i.  Each page that receives tokens:
 *   e_new = smallest e in [-126, 127] with amax <= 448 * 2^e over its new
 *           tokens' finite values, for K and for V, for each head
 *   e     = e_new if its slot 0 is written now, else max(e_old, e_new)
 *   codes already there -> rounded again to 2^e where e > e_old
 *   new code = e4m3(x * 2^-e), rounded to nearest even; infinities
 *   saturate to 448, NaN stays NaN
 * The slots past the new tokens keep their bytes.  One page must not belong
 * to two sequences that append in the same call.  Tokens whose block_table
 * entry is outside [0, num_pages), whose column is past max_pages, or that
 * are past max_q tokens of their sequence are not stored.  Slot 0 of a page
 * that starts within the call never depends on what the page held.  Errors:
 * FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED, FALCON_ERR_CUDA. */
int falcon_kv_append(const falcon_attn_params_t* p, const void* k, const void* v, const float* w_k,
                     const float* table, const int32_t* cu_new, const int32_t* ctx_lens,
                     const int32_t* block_table, const falcon_kv_cache_t* cache, void* stream);

/* Bytes of workspace falcon_attn_decode needs (0 when the params are invalid). */
size_t falcon_attn_decode_workspace_size(const falcon_attn_params_t* p);

/* Attention of one token per sequence over the cache: q [B, Hq, d],
 *   s_j = scale <q, K_j>, j < lens[b];  o = sum_j exp(s_j) V_j / sum_j exp(s_j)
 *   lse = log sum_j exp(s_j)   (fp32 [B, Hq], NULL = not wanted)
 * lens: int32 [B], at most max_k (and max_pages * page) of them are read;
 * lens[b] <= 0 gives o = 0 and lse = -inf.  Whatever lies in the slots past
 * lens[b] is not used.  Keys of a page whose block_table entry is outside
 * [0, num_pages) are masked.  o [B, Hq, d] with row stride o_stride.  One
 * kernel where max_k <= 512, or <= 1024 at d < 128 with at least three rows of
 * work (sequence, key head, group of 8 query heads) an SM; else two.  Waits on
 * copies are bounded and reported through falcon_workspace_status(workspace,
 * stream).  Any scale byte of a page will do: each weight is rounded relative
 * to its own tile's largest (11 bits for bf16, 22 for fp32).
 * Errors: FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED (dims, page sizes, a
 * cache of 2^38 bytes or more), FALCON_ERR_WORKSPACE, FALCON_ERR_CUDA. */
int falcon_attn_decode(const falcon_attn_params_t* p, const void* q, const falcon_kv_cache_t* cache,
                       const int32_t* block_table, const int32_t* lens, void* o, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace falcon_attn_prompt needs (0 when the params are invalid). */
size_t falcon_attn_prompt_workspace_size(const falcon_attn_params_t* p);

/* Causal attention over packed prompts.  cu_q / cu_k (int32 [B + 1]) delimit
 * each sequence's lq rows of q and lk rows of k, v (lq <= max_q;
 * lq != lk for a prompt that continues earlier tokens).  The causal mask is
 * aligned at the end: query i sees the keys j <= i + lk - lq.  A row that
 * sees no key gives o = 0 and lse = -inf.  o [tokens, Hq, d] with row stride
 * o_stride, lse fp32 [tokens, Hq] (NULL = not wanted).  Rows of q past max_q
 * of their sequence are not computed.  Any max_q will do; the exact bound is the quickest (the
 * tokens of all sequences as the bound: 1.1 to 1.5 times the time for 16 prompts
 * of 1024 tokens and 256 of 128).  bf16 rows on 16-byte boundaries run
 * their products on the tensor cores with bounded waits, reported through
 * falcon_workspace_status(workspace, stream) as for the chunk forward; fp32,
 * other alignments and calls of a few short prompts take a warp-level kernel
 * (bf16 rows off the 16-byte boundaries 4 to 11 times as long as on them).  The
 * bf16 weights are rounded to 8 bits on the tensor cores, to 11 there.
 * Errors: FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED,
 * FALCON_ERR_WORKSPACE, FALCON_ERR_CUDA. */
int falcon_attn_prompt(const falcon_attn_params_t* p, const void* q, const void* k, const void* v,
                       const int32_t* cu_q, const int32_t* cu_k, void* o, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Where a layer's gradients go, and how they and dO lie: elements from one token
 * to the next, 0 = dense.  dq, dk and dv may be slices of one fused gradient,
 * as q, k and v of a fused projection. */
typedef struct {
  void* dq;  /* [tokens, Hq, d] */
  void* dk;  /* [k_tokens, Hkv, d] (qk_norm_rope_backward: [tokens, Hkv, d]) */
  void* dv;  /* [k_tokens, Hkv, d]; attn_prompt_backward only */
  int64_t dq_stride, dk_stride, dv_stride;
  int64_t do_stride; /* of dO; attn_prompt_backward only */
} falcon_attn_grads_t;

/* Bytes of workspace falcon_attn_prompt_backward needs (0 when the params are invalid).  In fp32 it holds q, dO, k and
 * v once more, each sequence rounded up to 64 rows and rows of 16 and 32 dims to 64. */
size_t falcon_attn_prompt_backward_workspace_size(const falcon_attn_params_t* p);

/* Gradient of falcon_attn_prompt(p, q, k, v, cu_q, cu_k) with results o and lse,
 * for the loss L = <o, dO> + <lse, dlse>:
 *   P_ij = exp(scale <q_i, k_j> - lse_i) for the keys j that query i sees
 *   D_i  = <dO_i, o_i> - dlse_i,   dS_ij = P_ij (<dO_i, v_j> - D_i)
 *   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i
 * the sums of dk and dv also over the query heads that share the key head.  The
 * weights are formed again, nothing of their size is kept.  o (row stride
 * o_stride) and lse are what the forward returned for the same params; dO
 * [tokens, Hq, d] in the params' dtype, dlse fp32 [tokens, Hq] or NULL (zero).
 * g->dq may be NULL (skipped), or g->dk and g->dv.  Rows that see no key give
 * dq = 0 and add nothing; keys that no query sees get dk = dv = 0.  Rows of q past
 * max_q of their sequence have no gradient: their dq is left as it is and they
 * add nothing.  So are rows of dq, dk and dv behind the last sequence.  What
 * lies in rows that a row does not see (infinities, NaN) does not reach it.
 * Every sum has one order: the same call gives the same bits.  Sums are
 * fp32.  bf16: P and dS are rounded to 8 bits (rows off the 16-byte boundaries and
 * scales below 2^-100: 11);
 * fp32: operands, P and dS keep 22 bits, down to 2^-40 of the largest magnitude of
 * their row.  Bounded waits that run out are reported through
 * falcon_workspace_status(workspace, stream) (in the bf16 kernel of dq, where a
 * block has rows that are computed again, up to 2 us a key and such row later: they
 * hold up the next block).
 * Errors: FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED,
 * FALCON_ERR_WORKSPACE, FALCON_ERR_CUDA. */
int falcon_attn_prompt_backward(const falcon_attn_params_t* p, const void* q, const void* k, const void* v,
                                const int32_t* cu_q, const int32_t* cu_k, const void* o, const float* lse,
                                const void* d_o, const float* dlse, const falcon_attn_grads_t* g, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Bytes of workspace falcon_qk_norm_rope_backward needs (0 when the params are invalid). */
size_t falcon_qk_norm_rope_backward_workspace_size(const falcon_attn_params_t* p);

/* Gradient of falcon_qk_norm_rope(p, q, k, w_q, w_k, positions, table): from
 * dq_out (row stride o_stride) and dk_out (dense), the gradients of its
 * results, to g->dq and g->dk (row strides g->dq_stride, g->dk_stride) and, with
 * qk_norm, dw_q and dw_k (fp32 [d], NULL = not wanted):
 *   n = dy rotated back,  r = 1 / sqrt(mean(x^2) + norm_eps),  u = n w
 *   dx = r (u - x r mean(u x r)),   dw = sum over tokens and heads of n x r
 * (without the norm dx = n, and q and k are not read).  fp32 arithmetic and sums,
 * dx rounded once to the dtype; every sum has one order.  dq_out or dk_out may
 * be NULL (skipped, their dw untouched).  g->dq may be dq_out itself when
 * their strides agree, g->dk the same; other overlaps are refused.  A row whose sum
 * of squares passes fp32's range gives 0.  Rotated dims of a token whose
 * position is not in [0, rope_rows) are NaN, and with the norm so are its whole
 * rows and dw of the rotated dims.  tokens = 0 gives dw = 0.  The workspace is needed where a dw is
 * wanted.  Errors: FALCON_ERR_INVALID_ARG, FALCON_ERR_UNSUPPORTED,
 * FALCON_ERR_WORKSPACE, FALCON_ERR_CUDA. */
int falcon_qk_norm_rope_backward(const falcon_attn_params_t* p, const void* q, const void* k, const float* w_q,
                                 const float* w_k, const int64_t* positions, const float* table, const void* dq_out,
                                 const void* dk_out, const falcon_attn_grads_t* g, float* dw_q, float* dw_k,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Status of the last tensor-core chunk forward that used `workspace`
 * (falcon_chunk_fwd_plan reports FALCON_IMPL_TC for it; falcon_chunk_fwd,
 * _timed, _varlen), or, with workspace == NULL, of the last
 * falcon_chunk_fwd_noalloc call on the current device.  The pages have no
 * counterpart: this is the library's failure detection.  Every wait of
 * those kernels on another warp, a copy or a product is bounded in time
 * (2 s); a wait that runs out makes its kernel record a timeout in the
 * status word (the first 4 bytes of the workspace), skip its remaining
 * chunks, wait for its own copies in flight, free its tensor memory and
 * return, and the kernels after it in the call compute nothing.  The call
 * itself returned FALCON_OK before the kernels ran, so this is how the
 * caller learns of it.  Each such call clears the word when it starts.
 * The function synchronises `stream` (the call's stream), reads the word
 * and clears it.  Returns FALCON_OK, FALCON_ERR_TIMEOUT (the outputs and
 * carry of that call are incomplete), FALCON_ERR_WORKSPACE (workspace not
 * 256-byte aligned) or FALCON_ERR_CUDA.  The chunked backward (Falcon-1 /
 * 1A, d = 64) and falcon_attn_decode / _prompt / _prompt_backward keep their
 * words in the same place (a call without rows to write launches nothing and
 * leaves the word alone).
 * Other kernel families have no device-side waits and do not write the word. */
int falcon_workspace_status(const void* workspace, void* stream);

/* Test hook of the failure-detection path (no counterpart on the pages; not
 * for production use).  wait_limit_ns > 0 sets the limit of the bounded
 * device-side waits of the Falcon-1 / 1A, 3 and 3A tensor-core kernels
 * and of the chunked backward and the softmax-attention operators launched
 * from now on in this process (0 restores 2 s; the Falcon-2 kernel keeps 2 s).
 * stall != 0 makes the next forward call's per-chunk kernel (or the next
 * falcon_attn_decode, or tensor-core falcon_attn_prompt, or the first tensor-core kernel of
 * products of falcon_attn_prompt_backward) wait once, before it loads anything, on a barrier
 * that nothing completes: that wait runs out after the limit, the timeout is
 * recorded as described at falcon_workspace_status and the call's later
 * kernels skip their work.  No fault, trap or unbounded wait is involved;
 * the CUDA context stays usable.  Process-wide; not thread-safe against
 * concurrent calls that should not see it. */
void falcon_test_hooks(uint64_t wait_limit_ns, int32_t stall);

/* Static description of an error code (never NULL). */
const char* falcon_strerror(int code);

/* Library version string, e.g. "falcon-gb300 0.1 sm_103a". */
const char* falcon_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FALCON_H */
