/*
 * kvpop.h -- C ABI of the KVpop fixed-budget KV cache, decode-time hot path.
 *
 * Method: "KVpop -- Key-Value Cache Compression with Predictive Online
 * Pruning" (summary page of arXiv 2607.05061v2).  Every KV head keeps a
 * bounded cache of budget B = S + W + K tokens, the same for every head:
 * S attention-sink tokens, a protected window of the W most recent tokens,
 * and K long-range slots holding the running top-k of the tokens that have
 * left the window, ranked by a small headwise scorer on [k; v]
 * (page §3 "Fixed-budget pruning", §C.1 "Mask Definition", §E.1-§E.2,
 * §I "KVpop Pseudocode").  Optional delayed scoring (page §3 "Stateful
 * scorers", §E.4 "Delayed Readout") is a D-slot staging ring between the
 * window and the long-range slots: a token is scored D steps after it leaves
 * the window.  Staged tokens stay cached and are attended.
 *
 * Conventions for every call:
 *  - Return value: KVPOP_OK (0) or a negative KVPOP_ERR_* code.  Nothing
 *    throws or aborts across the ABI.  Arguments are validated before any
 *    work is enqueued; a call that fails validation enqueues nothing.
 *  - Device pointers point to memory on the device the handle was created on.
 *    The library never allocates or frees device memory: the caller owns all
 *    of it and lends it for the duration of the call (inputs) or the handle's
 *    lifetime (the cache buffer).
 *  - Work is asynchronous on the caller's CUDA stream (`stream`, a
 *    cudaStream_t; NULL = legacy default stream).  Only kvpop_create,
 *    kvpop_inspect, kvpop_get_error, kvpop_paged_create and
 *    kvpop_paged_get_error synchronise.
 *  - Calls on one handle must be ordered on one stream (or by the caller's
 *    events): the handle's split-K scratch is shared by its layers.
 *  - All batch rows share one sequence length.  Layers are independent and
 *    each keeps its own position counter (on the device).
 *  - Element type of q, k, v, the cache and the output: config.dtype.
 *    Scores are fp32 (the page, §F, ranks and selects in float32).
 */
#ifndef KVPOP_H
#define KVPOP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define KVPOP_OK 0
#define KVPOP_ERR_INVALID_ARG -1      /* null pointer, out-of-range layer, bad flag */
#define KVPOP_ERR_BAD_SHAPE -2        /* shape combination not valid / not built */
#define KVPOP_ERR_ORDER -3            /* call out of order (e.g. prefill after decode) */
#define KVPOP_ERR_CONTEXT_OVERFLOW -4 /* position counter would pass max_context */
#define KVPOP_ERR_CUDA -5             /* a CUDA runtime call failed */
#define KVPOP_ERR_DEVICE -6           /* a kernel recorded an error (see kvpop_get_error) */
#define KVPOP_ERR_TIMEOUT -7          /* a bounded device-side wait gave up */
#define KVPOP_ERR_SCRATCH_LIMIT -8    /* needs more scratch than kvpop_decode_step_noalloc's static buffer */

/* Size of the static split-K scratch buffer behind kvpop_decode_step_noalloc
 * (16 MiB on every GPU that loads the library, held until the process exits). */
#define KVPOP_NOALLOC_SCRATCH_BYTES (16u << 20)

/* Element types. */
#define KVPOP_DTYPE_F32 0
#define KVPOP_DTYPE_BF16 1

/* Scorer kinds (kvpop_config.scorer_kind). */
#define KVPOP_SCORER_MLP 0    /* stateless MLP, or the linear scorer when scorer_hidden = 0 (page §E.2) */
#define KVPOP_SCORER_MLSTM 1  /* stateful mLSTM scorer with delayed readout (page §A, §E.3, §E.4) */

/* Floats of one (layer, KV head) block of kvpop_config.mlstm_w: rows of 2d
 * weights W_q (p rows), W_k (p), W_v (dv), w_i, w_f, then w_o (dv), b_i, b_f,
 * b_o, padded to a multiple of 4. */
#define KVPOP_MLSTM_HEAD_FLOATS(p, dv, d) ((2 * (p) + (dv) + 2) * 2 * (d) + (((dv) + 3 + 3) / 4) * 4)

/* Flags. */
#define KVPOP_FLAG_EXTERNAL_SCORES 1u /* caller supplies every token's score instead of the MLP */
#define KVPOP_FLAG_DEBUG_CHECKS 2u    /* kernels check slot bookkeeping and NaN scores */

/* Device error bits reported by kvpop_get_error. */
#define KVPOP_DEVERR_CONTEXT_OVERFLOW 1
#define KVPOP_DEVERR_TIMEOUT 2
#define KVPOP_DEVERR_BAD_INDEX 4
#define KVPOP_DEVERR_NAN_SCORE 8
#define KVPOP_DEVERR_STATE_MISMATCH 16

typedef struct kvpop_config {
  int32_t batch;        /* batch rows b >= 1 */
  int32_t n_layers;     /* layers L >= 1 */
  int32_t n_q_heads;    /* query heads Hq, a multiple of n_kv_heads (GQA) */
  int32_t n_kv_heads;   /* KV heads Hkv >= 1 */
  int32_t head_dim;     /* d: 64 or 128 (bf16), 64 (fp32) */
  int32_t sinks;        /* S >= 0 */
  int32_t window;       /* W >= 1 */
  int32_t topk;         /* K >= 0 long-range slots; budget B = S + W + K */
  int32_t delay;        /* D >= 0 staging slots for delayed scoring (outside B) */
  int32_t ref_context;  /* prompt length the compression ratio is quoted against; 0 = no check */
  float compression_ratio; /* redundant, checked: |(1 - CR) * ref_context - B| <= 0.5 */
  int32_t max_context;  /* positions must stay below this (int32 positions) */
  int32_t max_prefill_chunk; /* largest n_tokens of one kvpop_prefill call */
  int32_t dtype;        /* KVPOP_DTYPE_F32 or KVPOP_DTYPE_BF16 */
  int32_t scorer_hidden; /* MLP 2d -> hidden -> 1 with hidden in {32, 64, 128}, or 0 = linear scorer */
  /* Scorer weights, device fp32, borrowed for the handle's lifetime
   * (may be NULL with KVPOP_FLAG_EXTERNAL_SCORES):
   *   w1 [L][Hkv][hidden][2d]  (input x = [k; v], page §E.1)
   *   b1 [L][Hkv][hidden], w2 [L][Hkv][hidden], b2 [L][Hkv]
   * score = w2 . relu(W1 x + b1) + b2 (page §E.2, stateless MLP scorer).
   * With scorer_hidden = 0 (page §E.2, stateless headwise linear scorer):
   * w1 [L][Hkv][2d] and b2 [L][Hkv], score = w1 . x + b2; b1, w2 may be NULL. */
  const float* w1;
  const float* b1;
  const float* w2;
  const float* b2;
  uint32_t flags;       /* KVPOP_FLAG_* */
  /* Optional temporal decay (page §B.3 "Temporal Decay and Static
   * Priorities"): device fp32 [L][Hkv] holding ln(gamma_h), each finite and
   * <= 0 (0 < gamma_h <= 1), borrowed for the handle's lifetime; NULL = no
   * decay.  Token j becomes eligible at step e_j = j + W + D; its effective
   * score at step q is s_j + (q - e_j) ln gamma_h, which ranks like the
   * static priority p_j = s_j - e_j ln gamma_h.  The library ranks by p_j,
   * formed once in fp32 (one rounding, like fmaf), and stores p_j as the
   * long-range slots' scores.  Requires max_context <= 2^24. */
  const float* log_decay;
  /* Scorer kind: KVPOP_SCORER_MLP (w1/b1/w2/b2 above) or KVPOP_SCORER_MLSTM
   * (the fields below; w1/b1/w2/b2 and scorer_hidden are then unused).  The
   * mLSTM scorer (page §A "Background: Linear Attention and mLSTM", §E.3
   * "mLSTM Scorer", §E.4 "Delayed Readout"): per KV head a recurrent state
   * (matrix memory C [2p][dv], normaliser n [2p], stabiliser m) in fp64 in
   * the cache buffer, updated by every token t with x_t = [k_t; v_t]:
   *   phi_t = [softmax(W_k x_t); softmax(-W_k x_t)] (Hedgehog feature map),
   *   i~ = w_i . x_t + b_i, log f = log sigmoid(w_f . x_t + b_f),
   *   m' = max(log f + m, i~), C' = e^(log f + m - m') C + e^(i~ - m') phi_t (W_v x_t)^T,
   *   n' = e^(log f + m - m') n + e^(i~ - m') phi_t;
   * the token u that becomes eligible at step q = u + W + D is read out from
   * the state after token q with r = Hedgehog(W_q x_u):
   *   h = C^T r / max(|n . r|, e^-m),  score = w_o . SiLU(h) + b_o,
   * rounded once to fp32.  Each decode step updates the state with the new
   * token before deciding the boundary token, so the decision is taken in
   * the step itself (one extra small launch per layer and step).  The
   * prefill attention calls do not take this scorer (KVPOP_ERR_BAD_SHAPE). */
  int32_t scorer_kind;
  int32_t mlstm_p;        /* Hedgehog projection size p, 1..16 (2p features) */
  int32_t mlstm_dv;       /* value size dv, 1..32 */
  const float* mlstm_w;   /* device fp32 [L][Hkv][KVPOP_MLSTM_HEAD_FLOATS(p, dv, d)], 16-byte aligned,
                             borrowed for the handle's lifetime (may be NULL with KVPOP_FLAG_EXTERNAL_SCORES) */
} kvpop_config;

typedef struct kvpop_handle kvpop_handle;

/* Offsets (bytes, from dev_mem) of the cache arrays, for inspection and tests.
 * Layer l's arrays start at offset + l * *_layer_stride. */
typedef struct kvpop_layout_info {
  size_t kv_offset, kv_layer_stride;       /* [units][slots][2][d] (key row, value row) */
  size_t pos_offset, pos_layer_stride;     /* int32 [units][slots], -1 = empty */
  size_t score_offset, score_layer_stride; /* fp32 [units][slots] */
  size_t state_offset, state_layer_stride; /* int32 [units][4] = {n_seen, n_topk, 0, 0} */
  int32_t slots_per_unit;                  /* S + W + D + K */
  int32_t units;                           /* batch * n_kv_heads; unit = b * Hkv + h */
  int32_t row_bytes;                       /* 2 * d * sizeof(dtype) */
  int32_t topk_base;                       /* first long-range slot, S + W + D */
} kvpop_layout_info;

/* Device bytes the caller must allocate for `cfg` (cache, slot metadata,
 * split-K and prefill scratch).  Validates cfg.  Host only.
 * Page §3 "Fixed-budget pruning" and §C.1 "Mask Definition": every KV head
 * keeps at most B = S + W + K tokens, the same budget for every head, so the
 * cache of a layer is units x (S + W + D + K) slots, fixed at creation
 * (D = the staging ring of delayed scoring, §E.4).  The pages quote
 * compression ratios (75%, 88%) without a formula; this library reads them
 * as CR = 1 - B / ref_context and checks cfg.compression_ratio against it.
 * Errors: KVPOP_ERR_INVALID_ARG (null argument; bad dtype, flag or scorer
 * pointer; compression ratio out of [0, 1) or not matching the budget),
 * KVPOP_ERR_BAD_SHAPE (shape outside the supported set). */
int kvpop_cache_bytes(const kvpop_config* cfg, size_t* bytes);

/* Binds a caller-allocated device buffer (>= kvpop_cache_bytes, 256-byte
 * aligned, on the current device) and initialises it (empty cache,
 * synchronously, after all work queued on the device).  The buffer must outlive the handle.  *out receives the
 * handle (host memory owned by the library until kvpop_destroy).
 * Page §3 "Fixed-budget pruning" (a hard, fixed-size cache: eviction is
 * permanent, so the cache never grows past its budget) and §C.1 (the budget
 * is reached once the sequence is long enough; until then every slot that
 * holds a token is attended).  Errors: KVPOP_ERR_INVALID_ARG (null, short or
 * misaligned buffer, buffer not device memory), KVPOP_ERR_BAD_SHAPE (cfg
 * outside the supported shapes), KVPOP_ERR_CUDA (a CUDA call failed); *out
 * is NULL then. */
int kvpop_create(const kvpop_config* cfg, void* dev_mem, size_t bytes, kvpop_handle** out);

/* Page §I "KVpop Pseudocode" (score every KV entry, keep the sinks, the
 * recent window and the running-prefix top-k of the eligible tokens) and
 * §C.1 "Mask Definition", applied to a whole prompt chunk at once.
 * Appends a chunk of n_tokens prompt tokens to layer `layer` (positions
 * n_seen .. n_seen + n_tokens - 1).  k, v: device [b][Hkv][n_tokens][d].
 * ext_scores: device fp32 [b][Hkv][n_tokens] (required with
 * KVPOP_FLAG_EXTERNAL_SCORES, ignored otherwise).  After the call the layer
 * holds the running prefix top-k state at its last token (page §I): the
 * long-range slots keep the K best eligible tokens; survivors keep their
 * slots and admitted tokens fill free/vacated slots in ascending order.
 * Must precede the layer's first decode step (else KVPOP_ERR_ORDER);
 * 0 <= n_tokens <= max_prefill_chunk.  Errors (nothing enqueued):
 * KVPOP_ERR_INVALID_ARG (bad handle or layer, negative n_tokens, null k or v,
 * missing ext_scores), KVPOP_ERR_BAD_SHAPE (n_tokens > max_prefill_chunk),
 * KVPOP_ERR_ORDER, KVPOP_ERR_CONTEXT_OVERFLOW (positions would reach
 * max_context); KVPOP_ERR_CUDA if a launch fails. */
int kvpop_prefill(kvpop_handle* h, int32_t layer, const void* k, const void* v, int32_t n_tokens,
                  const float* ext_scores, void* stream);

/* One decode step of one layer for all batch rows: page §3 "Fixed-budget
 * pruning" (sinks + protected window + running top-k, eviction permanent),
 * §C.1 "Mask Definition" (during decoding attention runs directly over the
 * retained cache entries), §E.4 "Delayed Readout" (the token u = q - w
 * becomes eligible at q; with the staging ring, D steps later) and §I
 * "KVpop Pseudocode" (the running prefix top-k rule).  With p = the layer's
 * position counter:
 *  1. window append and boundary update: the token leaving the window (after
 *     D staging steps when D > 0) is scored by the MLP on [k; v] (or its
 *     caller score) and replaces the minimum of the long-range set only if
 *     its key (score, -position) is strictly larger; while the long-range set
 *     is not full it takes the next free slot; the new token's k/v is written
 *     to its window slot;
 *  2. GQA attention of the new queries over all occupied slots (softmax,
 *     scale 1/sqrt(d), fp32 accumulation).
 * q: device [b][Hq][d]; k_new, v_new: device [b][Hkv][d]; out: device
 * [b][Hq][d] (same element type); ext_score: device fp32 [b][Hkv], the score
 * of the token being appended (required with KVPOP_FLAG_EXTERNAL_SCORES).
 * q, k_new, v_new and out must be 16-byte aligned (KVPOP_ERR_INVALID_ARG
 * otherwise).  The position counter then advances by one.  Errors (nothing
 * enqueued): KVPOP_ERR_INVALID_ARG (bad handle or layer, null or misaligned
 * pointer, missing ext_score), KVPOP_ERR_CONTEXT_OVERFLOW (the position
 * counter has reached max_context), KVPOP_ERR_BAD_SHAPE; KVPOP_ERR_CUDA if
 * the launch fails.  Device-side failures (a bounded wait that gave up,
 * debug-check mismatches) are reported later by kvpop_get_error. */
int kvpop_decode_step(kvpop_handle* h, int32_t layer, const void* q, const void* k_new, const void* v_new,
                      void* out, const float* ext_score, void* stream);

/* kvpop_decode_step for callers that cannot allocate device memory.
 * The KVpop pages have no counterpart: this is a deployment variant.
 *
 * Who needs it: code that runs where nobody may call cudaMalloc -- a plugin
 * inside a serving engine whose memory planner owns every device byte and
 * hands the plugin only the tensors it planned, or a latency-critical decode
 * loop that must not risk the device-wide synchronisation a cudaMalloc or
 * cudaFree can cause.  This call allocates nothing and calls no allocating
 * routine.  Its split-K partials and arrival tickets live in one static
 * device buffer that is part of the library image
 * (KVPOP_NOALLOC_SCRATCH_BYTES per GPU), not in the handle's buffer; the
 * handle's own split-K region is left untouched.
 *
 * Arguments, results and errors are those of kvpop_decode_step, plus:
 *  - KVPOP_ERR_SCRATCH_LIMIT (nothing enqueued) when the handle needs more
 *    scratch than the static buffer holds.  The need is
 *    units * 64 * G * (head_dim + 2) * 4 bytes plus units * 4, each part
 *    rounded up to 256 bytes (units = batch * n_kv_heads, G = n_q_heads /
 *    n_kv_heads); with G = 4, head_dim = 128 that is up to 126 units.
 *  - KVPOP_ERR_INVALID_ARG when the current device is not the handle's.
 *  - Set-up: the first call on a device (with that device current) looks up
 *    the buffer's device address once and keeps it for the process; make
 *    that first call before any stream capture begins.
 *  - Every call on a device shares the one buffer, which keeps what the last
 *    call left there.  The call clears the arrival tickets (the only part
 *    that must start at zero) on `stream` before its kernel; the partials
 *    are always written before they are read.  Calls whose work overlaps on
 *    the GPU (other streams, other handles, other host threads) race on the
 *    buffer and give wrong results: order them on one stream or by events. */
int kvpop_decode_step_noalloc(kvpop_handle* h, int32_t layer, const void* q, const void* k_new,
                              const void* v_new, void* out, const float* ext_score, void* stream);

/* The two halves of kvpop_decode_step (same passages: page §3, §C.1, §E.4,
 * §I), for callers that schedule them apart
 * (same arguments and semantics; append must precede attend for each step).
 * kvpop_decode_append: step 1 only (window append, boundary scoring and
 * argmin-replace); advances the position counter.
 * kvpop_decode_attend: step 2 only, over the cache as it stands (the query of
 * the token appended last).  Calling attend again without an append repeats
 * the same attention. */
int kvpop_decode_append(kvpop_handle* h, int32_t layer, const void* k_new, const void* v_new,
                        const float* ext_score, void* stream);
int kvpop_decode_attend(kvpop_handle* h, int32_t layer, const void* q, void* out, void* stream);

/* Parallel sparse prefill attention (page §C "Efficient Running Top-k Sparse
 * Attention": §C.1 Mask Definition, §C.2 Fenwick-Tree Cutoff Computation).
 * Computes, for every position q of a prompt of n_tokens tokens (positions
 * 0 .. n_tokens - 1) and every query head, the attention output under the
 * fixed-budget mask: q attends to exactly the set a decode step at q would
 * attend to -- the sinks, the recent W + D positions (its own included) and
 * the running top-k of the tokens eligible at q (scored as kvpop_prefill
 * scores them, decay included) -- with softmax scale 1/sqrt(d) and fp32
 * accumulation.  Does not read or change the cache or its position counter;
 * any layer's scorer weights may be used at any time.
 *
 * Running cutoffs: with m = q - W - D, token j (S <= j <= n_tokens-1-W-D)
 * is in the long-range set exactly for m in [j, c_j); c_j = INT32_MAX when j
 * is still kept at the last position, c_j = j when it is never admitted.
 * Tokens that never become eligible in the prompt get -1.
 *
 * q: device [b][Hq][n_tokens][d]; k, v: device [b][Hkv][n_tokens][d];
 * out: device [b][Hq][n_tokens][d] (config.dtype); lse: device fp32
 * [b][Hq][n_tokens] receiving each row's natural-log softmax normaliser
 * log sum_j exp(q.k_j / sqrt(d)), or NULL; ext_scores: device fp32
 * [b][Hkv][n_tokens] (required with KVPOP_FLAG_EXTERNAL_SCORES, ignored
 * otherwise).  q, k, v, out and workspace must be 16-byte aligned, lse 4-byte
 * aligned.
 * workspace: caller-owned device scratch of at least
 * kvpop_prefill_attention_workspace_bytes(n_tokens) bytes; after the call its
 * first units * n_tokens int32 hold the cutoffs c_j ([units][n_tokens]).
 * Errors: KVPOP_ERR_INVALID_ARG (null or misaligned pointer, workspace too
 * small, bad layer), KVPOP_ERR_BAD_SHAPE (G not dividing 64, head_dim other
 * than 64/128, S + K + W + D + P above 16384 where P = 64/G for fp32 and
 * 256/G for bf16, more than 65535 units, the mLSTM scorer),
 * KVPOP_ERR_CONTEXT_OVERFLOW (n_tokens > max_context); nothing is enqueued
 * then.  n_tokens = 0 is a no-op. */
int kvpop_prefill_attention_workspace_bytes(const kvpop_handle* h, int32_t n_tokens, size_t* bytes);
int kvpop_prefill_attention(kvpop_handle* h, int32_t layer, const void* q, const void* k, const void* v,
                            int32_t n_tokens, const float* ext_scores, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream);

/* The attention stage of kvpop_prefill_attention alone, from the running
 * cutoffs that a previous kvpop_prefill_attention call of the same prompt
 * (same layer's scorer, same k, v and n_tokens) left in `workspace`: the
 * prompt is not scored again and the cutoffs are not recomputed (page §C.2:
 * the cutoffs are computed once and the mask is evaluated from them on the
 * fly).  For a caller that runs several query sets over one prompt's mask.
 * The result equals that call's bit for bit when q, k and v are the same.
 * Arguments, layouts and errors as kvpop_prefill_attention (no ext_scores);
 * the workspace contents are the caller's responsibility. */
int kvpop_prefill_attention_from_cutoffs(kvpop_handle* h, int32_t layer, const void* q, const void* k, const void* v,
                                         int32_t n_tokens, void* out, float* lse, void* workspace,
                                         size_t workspace_bytes, void* stream);

/* kvpop_prefill and kvpop_prefill_attention in one call, for a whole prompt
 * on an empty layer: the prompt is scored once, its attention outputs (and
 * log-normalisers, if lse is not NULL) are computed under the running top-k
 * mask, and the layer's cache is built from the same scores and cutoffs --
 * the long-range slots receive the tokens whose cutoff is INT32_MAX (kept at
 * the last position) in ascending position order, exactly what kvpop_prefill
 * of the whole prompt as one chunk places.  Afterwards the layer is ready for
 * decode steps (position counter n_tokens).  Arguments, layouts, workspace
 * and errors as kvpop_prefill_attention, plus KVPOP_ERR_ORDER when the layer
 * has seen any token.  Page §C.1 / §C.2 (mask and cutoffs) and §I (running
 * prefix top-k). */
int kvpop_prefill_with_attention(kvpop_handle* h, int32_t layer, const void* q, const void* k, const void* v,
                                 int32_t n_tokens, const float* ext_scores, void* out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Copies layer `layer`'s slot -> position map (int32 [units][slots]), slot
 * scores (fp32 [units][slots]) and per-unit state (int32 [units][4]) to HOST
 * buffers; any of them may be NULL.  Synchronises `stream`.  Test and
 * diagnostic call; no passage of the pages defines it.  Errors:
 * KVPOP_ERR_INVALID_ARG (bad handle or layer), KVPOP_ERR_CUDA. */
int kvpop_inspect(kvpop_handle* h, int32_t layer, int32_t* pos_out, float* score_out, int32_t* state_out,
                  void* stream);

/* Fills *out with the layout of the device buffer.  Diagnostic call; no
 * passage of the pages defines it.  KVPOP_ERR_INVALID_ARG on a null argument. */
int kvpop_get_layout(const kvpop_handle* h, kvpop_layout_info* out);

/* Failure reporting of this library (no passage of the pages defines it).
 * Synchronises the device and reads the device error word.  Returns KVPOP_OK
 * if no kernel recorded an error, KVPOP_ERR_CONTEXT_OVERFLOW / _TIMEOUT /
 * _DEVICE otherwise (device_bits, if not NULL, receives the KVPOP_DEVERR_*
 * bits), or KVPOP_ERR_CUDA if the device reported an asynchronous error. */
int kvpop_get_error(kvpop_handle* h, int32_t* device_bits);

/* Clears the device error word (asynchronously, on `stream`).  Failure
 * reporting of this library; no passage of the pages defines it. */
int kvpop_clear_error(kvpop_handle* h, void* stream);

/* Test hook (no passage of the pages defines it): ORs `bits` into the device
 * error word on `stream`, so host-side failure handling can be exercised
 * without making any kernel fail. */
int kvpop_debug_poison_error(kvpop_handle* h, int32_t bits, void* stream);

/* Test hook (no passage of the pages defines it), honoured only by builds of
 * this library compiled with KVPOP_TEST_HOOKS, which also shorten the decode
 * kernel's merge-queue waits; other builds return KVPOP_ERR_INVALID_ARG and
 * change nothing.  hook = 1: in every later decode step, one consumer warp
 * finishes its work but never reports that it is done, so its CTA's merge
 * helpers wait until their bound runs out and the error word records
 * KVPOP_DEVERR_TIMEOUT (the kernel still returns; no copy is in flight
 * during that wait).  hook = 0 turns it off. */
int kvpop_debug_set_hook(kvpop_handle* h, int32_t hook);

/* Releases the handle's host state.  Does not touch the device buffer.
 * Resource management of this library; no passage of the pages defines it.
 * KVPOP_ERR_INVALID_ARG on NULL. */
int kvpop_destroy(kvpop_handle* h);

/* ---------------------------------------------------------------------------
 * Heads of new tokens, and the paged (full) cache.
 *
 * A model rarely prunes every layer: the layers, or the sequences, that keep
 * every token hold them in pages.  These calls stand beside the fixed-budget
 * ones: kvpop_qk_norm_rope makes the queries and keys that kvpop_prefill,
 * kvpop_decode_step and the paged cache take; kvpop_paged_append and
 * kvpop_paged_attend are kvpop_decode_append and kvpop_decode_attend without
 * a budget; kvpop_paged_gather hands a sequence's rows to kvpop_prefill or
 * kvpop_prefill_with_attention, which prune it.  No passage of the KVpop pages
 * defines them.  The conventions at the top of this file hold, with one
 * addition: a call may be made while another device than the handle's is
 * current (the stream must belong to the handle's device). */

/* Rows [batch][token][head][head_dim]: the address of the first element and
 * the strides of the first three dimensions in elements; the last dimension is
 * contiguous.  data must be 16-byte aligned and every stride of a dimension
 * longer than one a multiple of 16 bytes and not negative.  A stride of 0
 * (a broadcast) is taken for inputs only.  Rows that are written must not
 * overlap each other, nor an input of the call, except that q_out may be q
 * and k_out may be k (the same address and strides). */
typedef struct kvpop_rows {
  void* data;
  int64_t batch_stride, token_stride, head_stride;
} kvpop_rows;

/* Norm and position rotation of query and key heads:
 *   y = x / sqrt(mean(x^2) + eps) * weight        (skipped where weight is NULL)
 *   (a, b) -> (a cos - b sin, b cos + a sin), angle = position * inv_freq[i]
 * for the pairs i < rot_dim / 2: elements (i, i + rot_dim / 2), or with
 * interleaved (2i, 2i + 1); elements from rot_dim on are not turned.  Angles
 * are formed as 64-bit fractions of a turn (any int32 position): for
 * frequencies up to 1 they are off by at most 2^-32 turns, and at position p
 * by p 2^-54.6 more.  The rest is fp32, the sum of squares too (elements
 * beyond 2^60, or below 2^-60 with eps = 0, leave its range and are not
 * normalised to the formula), and the result is rounded once.  rot_scale multiplies cosine and sine (1 for plain
 * rotation).  All pointers are device memory, read while the call runs. */
typedef struct kvpop_rope {
  const float* q_weight;    /* fp32 [head_dim] or NULL, 16-byte aligned */
  const float* k_weight;    /* fp32 [head_dim] or NULL, 16-byte aligned */
  const double* inv_freq;   /* fp64 [rot_dim / 2], finite */
  float eps;                /* >= 0 */
  float rot_scale;
  int32_t rot_dim;          /* multiple of 8, 0 <= rot_dim <= head_dim; 0 = no rotation */
  int32_t interleaved;      /* 0 or 1 */
} kvpop_rope;

/* Norm and rotation of the heads of batch * n_tokens tokens.  q, q_out: rows
 * with n_q_heads heads; k, k_out: rows with n_kv_heads heads; positions:
 * device int32 [batch][n_tokens].  dtype KVPOP_DTYPE_*, head_dim 64 or 128.
 * Runs on the device that q lies on.  batch or n_tokens = 0 is a no-op;
 * batch * n_tokens <= 2^30.
 * Errors (nothing enqueued): KVPOP_ERR_INVALID_ARG (null or misaligned
 * pointer, bad stride, q not device memory, eps negative or not finite),
 * KVPOP_ERR_BAD_SHAPE; KVPOP_ERR_CUDA if the launch fails. */
int kvpop_qk_norm_rope(int32_t dtype, int32_t head_dim, int32_t n_q_heads, int32_t n_kv_heads,
                       const kvpop_rope* rope, int32_t batch, int32_t n_tokens, const kvpop_rows* q,
                       const kvpop_rows* k, const int32_t* positions, const kvpop_rows* q_out,
                       const kvpop_rows* k_out, void* stream);

/* How a paged cache holds its rows (kvpop_paged_config.cache_format). */
#define KVPOP_CACHE_NATIVE 0   /* in dtype */
#define KVPOP_CACHE_E4M3 1     /* 8 bits (e4m3) with one fp32 scale per key row and per value row; dtype bf16 only */

typedef struct kvpop_paged_config {
  int32_t n_layers;      /* >= 1 */
  int32_t n_q_heads;     /* a multiple of n_kv_heads, at most 16 per KV head */
  int32_t n_kv_heads;    /* 1..1024 */
  int32_t head_dim;      /* 64 or 128 */
  int32_t page_size;     /* tokens of a page: 16, 32, 64, 128 or 256 */
  int32_t n_pages;       /* pages of each layer; n_pages * page_size and n_pages * n_kv_heads < 2^31 */
  int32_t max_batch;     /* most sequences of one kvpop_paged_attend: 1..1024 */
  int32_t dtype;         /* of q, k, v and outputs: KVPOP_DTYPE_* */
  int32_t cache_format;  /* KVPOP_CACHE_* */
} kvpop_paged_config;

typedef struct kvpop_paged_handle kvpop_paged_handle;

/* Offsets (bytes, from dev_mem) of a paged cache's arrays; layer l's start at
 * offset + l * *_layer_stride.  A caller may read and write them directly,
 * ordered with the calls that use them. */
typedef struct kvpop_paged_layout_info {
  size_t pages_offset, pages_layer_stride;     /* [n_pages][n_kv_heads][2 (key, value)][page_size][head_dim] held elements */
  size_t scales_offset, scales_layer_stride;   /* fp32 [n_pages][n_kv_heads][2][page_size]; 0, 0 for KVPOP_CACHE_NATIVE */
} kvpop_paged_layout_info;

/* Device bytes of a paged cache.  Host only.  Errors: KVPOP_ERR_INVALID_ARG
 * (null argument; unknown dtype or cache_format; e4m3 with fp32),
 * KVPOP_ERR_BAD_SHAPE. */
int kvpop_paged_bytes(const kvpop_paged_config* cfg, size_t* bytes);

/* Binds a caller-allocated buffer (>= kvpop_paged_bytes, 256-byte aligned, on
 * the current device) and clears it to zero, synchronously, after all
 * work queued on the device.  The buffer must outlive the handle.  Errors as kvpop_create. */
int kvpop_paged_create(const kvpop_paged_config* cfg, void* dev_mem, size_t bytes, kvpop_paged_handle** out);

/* Writes keys and values of batch * n_tokens tokens into layer `layer`.
 * k, v: rows with n_kv_heads heads.  slots: device int32 [batch][n_tokens];
 * token t goes to row slots[t] % page_size of page slots[t] / page_size, a
 * negative slot writes nothing (padding), one past the last page writes
 * nothing and records KVPOP_DEVERR_BAD_INDEX.  With KVPOP_CACHE_E4M3, per row:
 *   scale = max |x| * c,  c = fp32(1 / 448),  held = e4m3(x / scale)
 * (product and quotient rounded to fp32, then to nearest even, at most 448).
 * A row whose scale is below the smallest normal fp32 number is held as
 * zeros with scale 0; a row with an infinity or a NaN gets a NaN scale and
 * reads back as NaN.  Two tokens of one call must not share a slot (which
 * one's bytes stay would be undefined, element by element; other rows are
 * not touched).  n_tokens = 0 is a no-op; batch * n_tokens <= 2^30.  Errors (nothing enqueued):
 * KVPOP_ERR_INVALID_ARG, KVPOP_ERR_BAD_SHAPE; KVPOP_ERR_CUDA. */
int kvpop_paged_append(kvpop_paged_handle* h, int32_t layer, const kvpop_rows* k, const kvpop_rows* v,
                       const int32_t* slots, int32_t batch, int32_t n_tokens, void* stream);

/* kvpop_qk_norm_rope and kvpop_paged_append in one launch: queries go to
 * q_out, keys are normalised, turned and written to their slots without being
 * rounded in between (with KVPOP_CACHE_E4M3 they are quantised from fp32),
 * values are written as they are.  Queries of padding tokens (negative slots)
 * are still written.  Arguments and errors as those two calls. */
int kvpop_paged_append_qkv(kvpop_paged_handle* h, int32_t layer, const kvpop_rope* rope, const kvpop_rows* q,
                           const kvpop_rows* k, const kvpop_rows* v, const int32_t* positions,
                           const int32_t* slots, const kvpop_rows* q_out, int32_t batch, int32_t n_tokens,
                           void* stream);

/* Reads `batch` sequences back: token i < lens[b] of sequence b, held in row
 * i % page_size of page page_table[b * table_stride + i / page_size], goes to
 * row (b, i) of k_out and v_out (rows with n_kv_heads heads and n_tokens
 * tokens per sequence), in dtype.  Rows at and past lens[b] are left as they
 * were.  page_table: device int32, table_width entries per sequence; lens:
 * device int32 [batch].  Sequences may share pages.  A length that is
 * negative or past n_tokens or table_width * page_size, or a page outside
 * [0, n_pages), records KVPOP_DEVERR_BAD_INDEX: the length is cut to the
 * range, and the rows of such a page are left as they were.  Errors (nothing
 * enqueued): KVPOP_ERR_INVALID_ARG, KVPOP_ERR_BAD_SHAPE; KVPOP_ERR_CUDA. */
int kvpop_paged_gather(kvpop_paged_handle* h, int32_t layer, const int32_t* page_table, int64_t table_stride,
                       int32_t table_width, const int32_t* lens, int32_t batch, int32_t n_tokens,
                       const kvpop_rows* k_out, const kvpop_rows* v_out, void* stream);

/* Options of kvpop_paged_attend; a null pointer means all zero.  scale and
 * softcap, where not 0, lie in [2^-100, 2^100]. */
typedef struct kvpop_attend_options {
  float scale;      /* > 0, or 0 = 1 / sqrt(head_dim) */
  float softcap;    /* > 0: scores become softcap * tanh(score / softcap); 0 = none */
  int32_t window;   /* > 0: the last `window` tokens of each sequence alone are attended; 0 = all */
} kvpop_attend_options;

/* Attention of one new token per sequence over its pages:
 *   s_j = scale q . k_j (capped),  out = sum_j softmax(s)_j v_j
 * over the tokens j < lens[b] (the last `window` of them), one launch; the
 * work of all sequences is split evenly over the GPU along
 * the cache's length and joined in a fixed order, so equal calls give equal
 * bits.  q, out: device [batch][n_q_heads][head_dim] in dtype, 16-byte
 * aligned, and out may be q; lse: device fp32 [batch][n_q_heads] receiving log sum_j e^(s_j),
 * or NULL.  page_table, lens as kvpop_paged_gather; 0 <= batch <= max_batch,
 * table_width * page_size <= 2^30.
 * Scores, the softmax's statistics and all sums are fp32.  The weights of
 * bf16 and e4m3 rows are held in 16 bits (two bf16 terms), so that each
 * token's part of an element is right to 2^-16 of itself down to 2^-100, and
 * bf16 outputs differ from those of fp32 weights in an occasional last place.
 * Attended values whose weighted sum passes fp32's range, infinite ones among
 * them, give infinities or NaN in their element.
 * A sequence with no token gets out = 0, lse = -inf.  Infinities and NaN in
 * tokens that are not attended do not reach the result; a NaN or +inf score
 * gives NaN.  A length that is negative or past table_width * page_size
 * (cut to the range) or a page outside [0, n_pages) (its tokens are left
 * out) records KVPOP_DEVERR_BAD_INDEX.  Calls on one handle share its
 * scratch: order them on one stream or by events, replays of captured graphs
 * among them.  Errors (nothing enqueued): KVPOP_ERR_INVALID_ARG,
 * KVPOP_ERR_BAD_SHAPE; KVPOP_ERR_CUDA. */
int kvpop_paged_attend(kvpop_paged_handle* h, int32_t layer, const void* q, const int32_t* page_table,
                       int64_t table_stride, int32_t table_width, const int32_t* lens, int32_t batch,
                       const kvpop_attend_options* options, void* out, float* lse, void* stream);

/* Layout, errors and release of a paged handle, as the kvpop_ calls of the
 * same names. */
int kvpop_paged_get_layout(const kvpop_paged_handle* h, kvpop_paged_layout_info* out);
int kvpop_paged_get_error(kvpop_paged_handle* h, int32_t* device_bits);
int kvpop_paged_clear_error(kvpop_paged_handle* h, void* stream);
int kvpop_paged_destroy(kvpop_paged_handle* h);

/* Static description of a status code (diagnostic; no passage defines it). */
const char* kvpop_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* KVPOP_H */
