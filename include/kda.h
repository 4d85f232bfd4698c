/*
 * kda.h -- C ABI of the GB300 gated-delta-rule forward library (libkda.so).
 *
 * The library computes the forward pass of the gated delta rule in its general
 * per-channel form, Kimi Delta Attention (KDA), and its special cases Gated
 * DeltaNet (one decay per head and token) and DeltaNet (no decay, log-decay 0).
 * For each sequence b, value head h and token t of the sequence, with key head
 * kh = h / (num_v_heads / num_k_heads) and S the d_v x d_k state of the
 * derivation ("You Could Have Come Up With Kimi Delta Attention", sec. 4, the
 * boxed KDA update; Modular MAX "gated_delta" module, the five per-token steps):
 *
 *     k^ = k[t,kh] / sqrt(|k[t,kh]|^2 + 1e-6)        (when l2norm_qk != 0)
 *     q^ = scale * q[t,kh] / sqrt(|q[t,kh]|^2 + 1e-6)
 *     S  = S Diag(exp(g[t,h]))                         forget (per key channel)
 *     e  = beta[t,h] (v[t,h] - S k^)                   predict and correct
 *     S  = S + e k^T                                   write
 *     o[t,h] = S q^                                    read, after the write
 *
 * Prefill runs the chunkwise (WY/UT) schedule of the same recurrence ("From
 * Attention to Learned Memory", sec. 4; KDA page sec. 6), which is exact up to
 * rounding; decode runs one token per sequence.
 *
 * Conventions shared by every entry point
 *   - All data pointers are DEVICE pointers; the caller allocates and owns every
 *     buffer (inputs, outputs, state pool, workspace).  The library never
 *     allocates, frees or synchronises on these paths.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t, passed as
 *     void*; NULL is the legacy default stream).  Inputs must stay valid until
 *     the stream reaches the enqueued work.
 *   - Layouts are row-major, token-major (ragged batches are concatenated along
 *     the token axis, as in the Modular gated_delta module):
 *         q, k          [T, num_k_heads, d_k]   (row stride settable, see below)
 *         v             [T, num_v_heads, d_v]
 *         beta          [T, num_v_heads]                     fp32
 *         log_decay g   [T, num_v_heads]        (SCALAR)     fp32, g = log alpha <= 0
 *                       [T, num_v_heads, d_k]   (PER_CHANNEL)
 *         state_pool    [num_slots, num_v_heads, d_k, d_v]   (the transpose of the
 *                       derivation's d_v x d_k state: key channel = row)
 *         o             [T, num_v_heads, d_v]                fp32
 *   - q/k/v/beta/g are read only, o is write only; the pool slots named by
 *     slot_idx are read, then overwritten in place with the final state; every
 *     other slot is left untouched.  Slots named twice in one call race.
 *   - Errors: argument problems are found on the host before anything is
 *     enqueued and returned as a status; nothing is launched then.  Problems
 *     only the device can see (offsets not monotone or not ending at
 *     total_tokens, a slot index >= num_slots, repeated slots under
 *     KDA_FLAG_CHECKED; on the tensor-core prefill path, a per-channel
 *     log-decay outside its domain, see KDA_DEVERR_DECAY_RANGE) set a device
 *     error word and the affected work is skipped -- no trap, no fault; read it
 *     with kda_get_device_error().
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 1

typedef enum kda_status {
  KDA_OK = 0,
  KDA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, bad enum value */
  KDA_ERR_UNSUPPORTED = 2, /* valid but not implemented: head size, chunk, dtype combination */
  KDA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than kda_prefill_workspace_size */
  KDA_ERR_CUDA = 4,        /* a CUDA runtime call or a launch failed */
  KDA_ERR_DEVICE = 5       /* kda_get_device_error: the device flagged bad offsets/slots */
} kda_status_t;

typedef enum kda_dtype { KDA_DTYPE_F32 = 0, KDA_DTYPE_BF16 = 1 } kda_dtype_t;

typedef enum kda_decay_kind {
  KDA_DECAY_SCALAR = 0,     /* Gated DeltaNet: one log-decay per (token, value head) */
  KDA_DECAY_PER_CHANNEL = 1 /* KDA: one log-decay per (token, value head, key channel) */
} kda_decay_kind_t;

/* Check every sequence's offsets and slot and that slots are distinct on the
 * device (without it, offsets and slot ranges are still checked, distinctness is not). */
#define KDA_FLAG_CHECKED 1u
/* Run the prefill on CUDA cores in fp32 even where the tensor-core path applies
 * (bf16 q/k/v, d = 128, chunk 64, whose operands are fp16/bf16 with fp32
 * accumulation).  fp32 q/k/v and the other head sizes and chunks always use it. */
#define KDA_FLAG_CUDA_CORES 2u
/* Tensor-core path only: run it as one kernel per (sequence, value head, value
 * tile) that walks the sequence's chunks, with only the chunk table (16 bytes per
 * chunk) and one flag per sequence and value head as workspace; its per-channel
 * factors are anchored at each chunk's middle token, which bounds the decay it takes
 * (see KDA_DEVERR_DECAY_RANGE).  Without it the path runs as two kernels: a chunk-parallel
 * one that writes every chunk's operands of the state recurrence to the workspace
 * (57,856 bytes per chunk and value head) and a sequential one over each
 * sequence's chunks, which keeps the chunk-local work off the sequential path.
 * The two forms round the same operands the same way; their results agree to
 * the tolerance, not bit for bit.  In kda_prefill_bwd the flag bounds the
 * workspace instead (see there). */
#define KDA_FLAG_COMPACT 4u
/* Additive write in place of the delta rule: the correction subtracts no
 * prediction, e_t = beta_t v_t, so S_t = Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 * (stored orientation: row = key channel).  With per-channel decay this is Gated
 * Linear Attention, with scalar decay Mamba-2 (beta_t its write step size) or
 * RetNet (a constant decay), and with zero log-decay and beta = 1 plain causal
 * linear attention ("Linear attention visualized": the naive linear attention,
 * RetNet, Mamba-2 and GLA sections; "From Attention to Learned Memory", sec. 1-2).
 * Accepted by every prefill path, the decode step and the verify window (whose
 * records then hold beta_t v_t); the Gated DeltaProduct entry points, whose method
 * is defined on the delta rule, return KDA_ERR_UNSUPPORTED for it. */
#define KDA_FLAG_NO_DELTA 8u

/* Device error codes (kda_get_device_error). */
#define KDA_DEVERR_NONE 0
#define KDA_DEVERR_OFFSETS 1   /* input_row_offsets not monotone / not 0..total_tokens */
#define KDA_DEVERR_SLOT_RANGE 2 /* slot_idx[b] >= num_slots */
#define KDA_DEVERR_SLOT_DUP 3   /* a slot named twice (KDA_FLAG_CHECKED only) */
#define KDA_DEVERR_TIMEOUT 4    /* a bounded wait inside a kernel gave up; its work is incomplete */
/* KDA_DEVERR_DECAY_RANGE: tensor-core prefill path, per-channel decay outside its domain.
 * The default two-kernel form takes any log-decay g <= 1/64 (a forget gate up to
 * exp(1/64)); a larger g is outside it.  The compact form (KDA_FLAG_COMPACT) also needs
 * every channel's cumulative log-decay to stay within 79 nats of its value at the chunk's
 * middle token.  The (sequence, value head) pairs with such a chunk are skipped: their o rows
 * and their slot's state keep their previous contents, every other pair is computed.  The
 * fp32 CUDA-core path (KDA_FLAG_CUDA_CORES) takes any finite log-decay. */
#define KDA_DEVERR_DECAY_RANGE 5
#define KDA_DEVERR_ACCEPTED 6    /* kda_fold_accepted: accepted[b] > window */
#define KDA_DEVERR_PAGE 7        /* kda_cache_*: a page, length, parent or reference count out of range, or
                                    fewer free pages than are asked for */

typedef struct kda_params {
  int32_t num_seqs;    /* B: sequences in the ragged batch (prefill) or decode batch */
  int32_t num_k_heads; /* HK: heads of q and k */
  int32_t num_v_heads; /* HV: heads of v, beta, g, o and the state; HV % HK == 0 */
  int32_t d_k;         /* key head size; 16 or 128 */
  int32_t d_v;         /* value head size; must equal d_k */
  int32_t num_slots;   /* slots in state_pool */
  int64_t total_tokens;/* T: rows of the token-major tensors (prefill; ignored by decode) */
  int32_t chunk;       /* prefill chunk length C: 16, 32 or 64 (ignored by decode) */
  int32_t qkv_dtype;   /* kda_dtype_t of q, k, v */
  int32_t state_dtype; /* kda_dtype_t of state_pool (bf16 is rounded to nearest even) */
  int32_t decay_kind;  /* kda_decay_kind_t of log_decay */
  float scale;         /* query scale; <= 0 selects 1/sqrt(d_k) */
  int32_t l2norm_qk;   /* nonzero: L2-normalise q and k rows before use */
  uint32_t flags;      /* KDA_FLAG_* */
  /* Elements between consecutive tokens of q, k, v; 0 means dense
   * (HK*d_k, HK*d_k, HV*d_v).  Lets q, k, v be column blocks of one packed
   * [T, 2*HK*d_k + HV*d_v] buffer.  Must keep rows 16-byte aligned. */
  int64_t q_row_stride;
  int64_t k_row_stride;
  int64_t v_row_stride;
} kda_params_t;

/* Version of this ABI (KDA_ABI_VERSION).  Never fails. */
int kda_abi_version(void);

/* Static, NUL-terminated description of a status code.  Never fails. */
const char *kda_status_string(kda_status_t status);

/*
 * Bytes of device workspace kda_prefill_fwd needs for these parameters
 * (an upper bound that depends only on the params, not on the offsets).
 * Returns KDA_ERR_INVALID_ARG / KDA_ERR_UNSUPPORTED for parameters that
 * kda_prefill_fwd would reject; *bytes is then left unchanged.
 */
kda_status_t kda_prefill_workspace_size(const kda_params_t *p, size_t *bytes);

/*
 * 1 if kda_prefill_fwd would run these parameters on the tensor-core path
 * (bf16 q/k/v, d = 128, chunk 64, KDA_FLAG_CUDA_CORES clear: fp16/bf16 MMA
 * operands with fp32 accumulation), 0 if on the fp32 CUDA-core path, -1 if the
 * parameters are invalid.  Never touches the GPU.
 */
int kda_prefill_uses_tensor_cores(const kda_params_t *p);

/*
 * Chunkwise prefill over a ragged batch ("You Could Have Come Up With Kimi
 * Delta Attention", sec. 6 and the pipeline of sec. 6.6; "From Attention to
 * Learned Memory", sec. 4, WY/UT transform and blocked triangular inverse;
 * Modular "gated_delta" module for the ragged batch, GQA and slot pool).
 *
 *   q, k               [T, HK, d_k], qkv_dtype, rows 16-byte aligned
 *   v                  [T, HV, d_v], qkv_dtype
 *   beta               [T, HV] fp32
 *   log_decay          [T, HV] or [T, HV, d_k] fp32 (decay_kind); 4-byte aligned, and
 *                      16-byte aligned for KDA_DECAY_PER_CHANNEL (its rows are copied in
 *                      16-byte pieces), else KDA_ERR_INVALID_ARG
 *   input_row_offsets  [B+1] uint32: sequence b is tokens [off[b], off[b+1]);
 *                      off[0] = 0, non-decreasing, off[B] = T.  Empty sequences
 *                      are allowed and leave their slot untouched.
 *   slot_idx           [B] uint32, each < num_slots: the pool slot holding
 *                      sequence b's initial state, overwritten with its final state
 *   state_pool         [num_slots, HV, d_k, d_v], state_dtype, in place
 *   o                  [T, HV, d_v] fp32, written for every token
 *   workspace          device scratch of >= kda_prefill_workspace_size bytes,
 *                      256-byte aligned; contents on entry are ignored
 * Returns KDA_OK once the work is enqueued.
 */
kda_status_t kda_prefill_fwd(const kda_params_t *p, const void *q, const void *k, const void *v,
                             const float *beta, const float *log_decay,
                             const uint32_t *input_row_offsets, const uint32_t *slot_idx,
                             void *state_pool, float *o, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * The front end before the recurrence ("Pass 1" of the Modular "gated_delta" module, which
 * consumes its output; SiLU features as in "From Attention to Learned Memory", sec. 1; the
 * decay built from a log-rate and a softplus step as in the Mamba-2 section of "Linear
 * attention visualized"): over the packed projection x = [Q | K | V] (conv_dim = 2 HK d_k +
 * HV d_v channels per token) a depthwise causal convolution of `width` (1..4) taps and SiLU,
 *
 *     y[t, c] = SiLU(conv_bias[c] + sum_{i < width} conv_weight[c, i] x[t - width + 1 + i, c]),
 *
 * where the width - 1 inputs before a sequence's first token come from its slot of conv_state
 * (oldest first; zeros when conv_state is NULL), and afterwards the slot holds the sequence's
 * last width - 1 inputs (an empty sequence leaves it alone); plus the gates
 *
 *     beta = sigmoid(b),   log_decay = -exp(A_log[h]) softplus(a + dt_bias).
 *
 *   x, y         [T, conv_dim], qkv_dtype, 16-byte aligned; y's column blocks are q, k, v for
 *                kda_prefill_fwd through q/k/v_row_stride = conv_dim
 *   conv_weight  [conv_dim, width] fp32       conv_bias [conv_dim] fp32 or NULL
 *   a            [T, HV] (SCALAR) or [T, HV, d_k] (PER_CHANNEL) fp32; b [T, HV] fp32
 *   A_log        [HV] fp32 or NULL (rate 1)   dt_bias [HV] or [HV * d_k] fp32 or NULL
 *   input_row_offsets  [B + 1] as kda_prefill_fwd (T = total_tokens), or NULL for the
 *                decode form: one token per sequence, T = num_seqs
 *   slot_idx     [B] (required with conv_state)
 *   conv_state   [num_slots, conv_dim, width - 1], qkv_dtype, or NULL; read and written in place
 *   log_decay    the shape of a, fp32;  beta [T, HV] fp32
 * The row strides in p must be 0 (dense x and y).  Offsets out of order and slots out of
 * range set the device error word; nothing is read or written out of bounds.
 */
kda_status_t kda_conv_gates_fwd(const kda_params_t *p, int32_t width, const void *x,
                                const float *conv_weight, const float *conv_bias, const float *a,
                                const float *b, const float *A_log, const float *dt_bias,
                                const uint32_t *input_row_offsets, const uint32_t *slot_idx,
                                void *conv_state, void *y, float *log_decay, float *beta,
                                void *stream);

/*
 * Backward pass of kda_prefill_fwd: the gradients of a loss w.r.t. every input,
 * given its gradients w.r.t. the outputs o and the final states.  The chunk form
 * of the forward ("You Could Have Come Up With Kimi Delta Attention", sec. 6) is
 * differentiated by the chain rule: the state gradient runs as a reverse scan
 * over each sequence's chunks (the transpose of the forward's state recursion),
 * the rest chunk-parallel; the L2 normalisation of q and k and the query scale
 * are differentiated too ("From Attention to Learned Memory", sec. 3, gives the
 * linear-attention backward in full; the delta rule's follows the same recurrence).
 * fp32 arithmetic throughout; with bf16 q/k/v at d = 128 and chunk 64 the scan's
 * two directions and the contractions over the value dimension run on tensor
 * cores with tf32 operands (10-bit mantissa, fp32 range) and fp32 accumulation,
 * everything else on CUDA cores.
 *
 *   q, k, v, beta, log_decay, input_row_offsets, slot_idx: as kda_prefill_fwd
 *   state_pool  [num_slots, HV, d_k, d_v], state_dtype, read only: the INITIAL
 *               states (the pool as it was before the forward call)
 *   d_o         [T, HV, d_v] fp32: dLoss/do
 *   d_state     [num_slots, HV, d_k, d_v] fp32 or NULL (zero): dLoss/d(final
 *               state) of the touched slots
 *   dq, dk      [T, HK, d_k] fp32 (summed over the value heads of each key head)
 *   dv          [T, HV, d_v] fp32          dbeta [T, HV] fp32
 *   dlog_decay  the shape of log_decay, fp32
 *   d_state0    [num_slots, HV, d_k, d_v] fp32 or NULL: dLoss/d(initial state),
 *               written at the touched slots only; may alias d_state
 *   workspace   >= kda_prefill_bwd_workspace_size bytes, 256-byte aligned
 * q, k, v 16-byte aligned with 16-byte aligned rows (as for the forward), every
 * other array 4-byte aligned.  KDA_FLAG_NO_DELTA differentiates the additive
 * write; KDA_FLAG_CUDA_CORES is ignored.  Device-side checks (offsets, slots) set
 * the error word and skip the work, as in the forward.
 *
 * Workspace.  By default it holds every chunk's per-(chunk, value head) matrices,
 * about 0.6 MB per chunk and value head (9.3 GB for 2 x 16384 tokens, 32 heads).
 * KDA_FLAG_COMPACT (bf16 q/k/v, d = 128, chunk 64; ignored elsewhere) bounds it:
 * the chunks run in windows of wc chunk positions per sequence,
 * wc = max(1, 512 / (num_seqs * HV)), so the per-chunk matrices exist for
 * max(512, num_seqs * HV) (chunk, value head) slots, plus the state entering
 * every window after a sequence's first (64 KB per window and value head at
 * d = 128) and one state gradient per (sequence, value head): 421 MiB for
 * 2 x 16384 tokens, 32 heads.  A forward sweep over the windows stores those
 * entering states; the backward sweep then reruns each window's chunk-local stage
 * and forward scan from its checkpoint, latest window first, with the same
 * arithmetic per chunk, so the gradients equal the default form's bit for bit.
 * The call reads the longest sequence's chunk count back to the host once (a
 * synchronisation of `stream`) to size the sweeps.
 */
kda_status_t kda_prefill_bwd_workspace_size(const kda_params_t *p, size_t *bytes);
kda_status_t kda_prefill_bwd(const kda_params_t *p, const void *q, const void *k, const void *v,
                             const float *beta, const float *log_decay,
                             const uint32_t *input_row_offsets, const uint32_t *slot_idx,
                             const void *state_pool, const float *d_o, const float *d_state,
                             float *dq, float *dk, float *dv, float *dbeta, float *dlog_decay,
                             float *d_state0, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * One recurrent decode step: one token for each of B = num_seqs sequences
 * ("You Could Have Come Up With Kimi Delta Attention", sec. 5, fused recurrent
 * kernel; Modular "gated_delta" module, the five per-token steps).
 *
 *   q, k        [B, HK, d_k], qkv_dtype     v  [B, HV, d_v], qkv_dtype
 *   beta        [B, HV] fp32                log_decay [B, HV] or [B, HV, d_k] fp32
 *   slot_idx    [B] uint32, each < num_slots
 *   state_pool  [num_slots, HV, d_k, d_v], state_dtype, updated in place
 *   o           [B, HV, d_v] fp32
 * total_tokens and chunk are ignored.  Needs no workspace.
 */
kda_status_t kda_decode_step(const kda_params_t *p, const void *q, const void *k, const void *v,
                             const float *beta, const float *log_decay, const uint32_t *slot_idx,
                             void *state_pool, float *o, void *stream);

/*
 * Speculative-decode verification (Modular MAX "gated_delta" module: the verify
 * kernel runs the recurrence over a verify window and records a ring instead of
 * writing the state back; the fold applies a verify's accepted records to the
 * pool).  The module does not spell out a record; here one record is what a
 * token's state update needs, so that folding it replays that update exactly:
 *
 *     record = [ k^ (d_k) | e (d_v) | alpha (d_k; for SCALAR decay one value
 *                followed by 3 padding elements) ]   fp32
 *     fold:    S <- S Diag(alpha) + e k^T     (the forget and write steps)
 *
 * kda_ring_record_elems returns the record length in fp32 elements
 * (2 d_k + d_v, or d_k + d_v + 4), or -1 for invalid parameters.
 */
int kda_ring_record_elems(const kda_params_t *p);

/*
 * Runs `window` tokens of each of B = num_seqs sequences from its pool slot
 * without modifying the pool: writes every token's output and ring record.
 *   q, k        [B*window, HK, d_k]  (token t of sequence b is row b*window + t)
 *   v           [B*window, HV, d_v]     beta [B*window, HV] fp32
 *   log_decay   [B*window, HV] or [B*window, HV, d_k] fp32
 *   slot_idx    [B] uint32              state_pool read only
 *   o           [B*window, HV, d_v] fp32
 *   ring        [B, window, HV, kda_ring_record_elems] fp32, 16-byte aligned
 * window must be 1..64.  total_tokens and chunk are ignored.
 */
kda_status_t kda_verify_window(const kda_params_t *p, const void *q, const void *k, const void *v,
                               const float *beta, const float *log_decay, const uint32_t *slot_idx,
                               int32_t window, const void *state_pool, float *o, float *ring,
                               void *stream);

/*
 * Applies the first accepted[b] records of sequence b's verify window to its
 * pool slot, in token order (accepted[b] = 0 leaves the slot unchanged).  The
 * result equals accepted[b] decode steps of those tokens from the same state.
 *   ring       as written by kda_verify_window with the same p and window
 *   accepted   [B] uint32, each <= window (larger values set KDA_DEVERR_ACCEPTED
 *              on the device and leave that slot unchanged)
 *   slot_idx   [B] uint32; state_pool updated in place
 */
kda_status_t kda_fold_accepted(const kda_params_t *p, const float *ring, int32_t window,
                               const uint32_t *accepted, const uint32_t *slot_idx,
                               void *state_pool, void *stream);

/*
 * Gated DeltaProduct ("Linear attention visualized", Gated Delta Product section and
 * its virtual-sequence table).  Every token carries n_h transitions, each with its own
 * key, value and gate; the state decays once (by the token's log_decay) before the
 * first, the n_h predict / correct / write steps follow in order, and the token's query
 * reads the state after the last.  n_h = 1 is kda_prefill_fwd.  Computed as the gated
 * delta rule over the virtual sequence of T * n_h positions (decay on the first
 * substep, query on the last, every n_h-th output kept) on the same prefill path.
 *
 *   n_h                1..64 substeps per token
 *   q                  [T, HK, d_k], one query per token (q_row_stride between tokens)
 *   k                  [T, n_h, HK, d_k] (k_row_stride between substep rows)
 *   v                  [T, n_h, HV, d_v] (v_row_stride between substep rows)
 *   beta               [T, n_h, HV] fp32
 *   log_decay          [T, HV] or [T, HV, d_k] fp32, one per token
 *   input_row_offsets, slot_idx, state_pool: as kda_prefill_fwd, over tokens
 *   o                  [T, HV, d_v] fp32, one output per token
 *   workspace          >= kda_gdp_workspace_size(p, n_h, 0) bytes, 256-byte aligned
 * The workspace also holds the virtual queries, log-decays and outputs
 * (T * n_h * (HK*d_k*qkv size + HV*gate width*4 + HV*d_v*4) bytes) ahead of the
 * prefill's own workspace.  Errors as kda_prefill_fwd; n_h outside 1..64 is
 * KDA_ERR_INVALID_ARG, T * n_h >= 2^31 is KDA_ERR_UNSUPPORTED.
 */
kda_status_t kda_gdp_prefill_fwd(const kda_params_t *p, int32_t n_h, const void *q,
                                 const void *k, const void *v, const float *beta,
                                 const float *log_decay, const uint32_t *input_row_offsets,
                                 const uint32_t *slot_idx, void *state_pool, float *o,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * One Gated DeltaProduct decode step: one token (n_h transitions) for each of
 * B = num_seqs sequences, read from and written back to slot_idx[b] of the pool.
 * Arrays as kda_gdp_prefill_fwd with T = B and no offsets; total_tokens is ignored,
 * chunk 0 means 64.  Workspace: kda_gdp_workspace_size(p, n_h, 1) bytes.
 */
kda_status_t kda_gdp_decode_step(const kda_params_t *p, int32_t n_h, const void *q,
                                 const void *k, const void *v, const float *beta,
                                 const float *log_decay, const uint32_t *slot_idx,
                                 void *state_pool, float *o, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * Workspace bytes of kda_gdp_prefill_fwd (decode = 0) or kda_gdp_decode_step
 * (decode = 1) for these parameters and n_h.  Returns the status the call would
 * return for invalid parameters; *bytes is then left unchanged.
 */
kda_status_t kda_gdp_workspace_size(const kda_params_t *p, int32_t n_h, int32_t decode,
                                    size_t *bytes);

/*
 * Waits for `stream`, then returns the device error word of the current device
 * in *code (KDA_DEVERR_*) and clears it.  Returns KDA_ERR_DEVICE when the word
 * was set, KDA_OK when it was clear, KDA_ERR_CUDA when a CUDA call failed.
 */
kda_status_t kda_get_device_error(void *stream, int32_t *code);

/*
 * Prefill without any device allocation: same inputs, outputs and results as
 * kda_prefill_fwd, but its scratch lives in a fixed array inside the library
 * instead of a caller-provided workspace.  There is no counterpart on the pages.
 *
 * For callers that cannot allocate device memory at the point where they run
 * the prefill: code hosted inside an engine that owns the device's memory
 * budget and hands out no allocator, or a runtime that reserves all of its
 * memory at start-up.  They still pass every input and output buffer.
 *
 *   - The scratch is KDA_NO_ALLOC_SCRATCH_BYTES (64 MiB) of device memory that
 *     every GPU which loads the library holds until the process exits.
 *     Problems whose workspace exceeds it are rejected with KDA_ERR_WORKSPACE
 *     before anything is enqueued.
 *   - The default two-kernel tensor-core form needs the chunk table and 57,856
 *     bytes of chunk records per chunk and value head: about 1,150 chunk-heads
 *     (some 4,600 tokens x 16 value heads at chunk 64) fit.  Larger problems run
 *     the compact single-kernel form instead (as with KDA_FLAG_COMPACT: the chunk
 *     table and a flag per sequence and value head, which fits any practical
 *     batch), which is slower and takes a narrower per-channel decay range (see
 *     KDA_DEVERR_DECAY_RANGE); kda_prefill_no_alloc_form() says which form a call
 *     with these parameters runs.  The fp32 CUDA-core path needs about 150 KB per
 *     chunk and value head (roughly 1,700 tokens x 16 heads at d = 128, chunk 64).
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.  Later calls allocate nothing and enqueue
 *     nothing on the stream but the kernel launches.
 *   - All calls share the one array and it keeps the last call's contents
 *     (nothing in it needs to start at zero).  Calls whose work overlaps on the
 *     GPU -- different streams, or different host threads -- race on it: order
 *     them on one stream.
 * Arguments, layouts, errors and the device error word are as in
 * kda_prefill_fwd.  This entry point calls no cudaMalloc / cudaFree.
 */
#define KDA_NO_ALLOC_SCRATCH_BYTES (64u << 20)
kda_status_t kda_prefill_fwd_no_alloc(const kda_params_t *p, const void *q, const void *k,
                                      const void *v, const float *beta, const float *log_decay,
                                      const uint32_t *input_row_offsets, const uint32_t *slot_idx,
                                      void *state_pool, float *o, void *stream);

/*
 * Which form kda_prefill_fwd_no_alloc runs for these parameters (no counterpart on
 * the pages): 0 the two-kernel tensor-core form, 1 the compact single-kernel
 * tensor-core form (the chunk records do not fit the scratch, or KDA_FLAG_COMPACT is
 * set), 2 the fp32 CUDA-core path, -1 rejected (invalid parameters, or a workspace
 * larger than KDA_NO_ALLOC_SCRATCH_BYTES).  Never touches the GPU.
 */
int kda_prefill_no_alloc_form(const kda_params_t *p);

/*
 * The layer around the recurrence: the projections into the front end and out of the
 * recurrence, the norms on both sides of a block, and the output norm with its gate.  All
 * three read and write token-major rows; sums, norms and accumulators are fp32.  Work is
 * enqueued on `stream`; zero tokens is a valid call (sums over no tokens are zero).
 */
typedef enum kda_activation {
  KDA_ACT_NONE = 0,
  KDA_ACT_RELU = 1,
  KDA_ACT_SILU = 2,   /* z sigmoid(z) */
  KDA_ACT_GELU = 3,   /* z Phi(z), Phi the normal distribution function (the erf form) */
  KDA_ACT_SIGMOID = 4
} kda_activation_t;

/* kda_linear_*: the base of x, w or d_y is not 16-byte aligned (a column block at an odd
 * offset).  Adds an aligned copy of that bf16 operand to the workspace; without it an unaligned
 * base is KDA_ERR_INVALID_ARG.  Rows that are not a multiple of 16 bytes apart need no flag. */
#define KDA_FLAG_UNALIGNED_X 16u
#define KDA_FLAG_UNALIGNED_W 32u
#define KDA_FLAG_UNALIGNED_DY 64u

typedef struct kda_linear_params {
  int64_t tokens;       /* T: rows of x and y */
  int32_t in_features;  /* K >= 1 */
  int32_t out_features; /* N >= 1 */
  int32_t dtype;          /* kda_dtype_t of x, w and pre_act (and of dx) */
  int32_t y_dtype;        /* kda_dtype_t of y (backward: of d_y) */
  int32_t residual_dtype; /* kda_dtype_t of residual (forward) */
  int32_t dw_dtype;       /* kda_dtype_t of dw (backward) */
  int32_t activation;     /* kda_activation_t */
  float scale;            /* s; any finite value */
  /* elements between rows; 0 means dense.  y_row_stride is y's, or d_y's in the backward. */
  int64_t x_row_stride, w_row_stride, y_row_stride, residual_row_stride;
  uint32_t flags;         /* KDA_FLAG_CUDA_CORES (fp32 arithmetic on CUDA cores), KDA_FLAG_UNALIGNED_* */
} kda_linear_params_t;

/*
 * Projection with its epilogue:
 *
 *     z[t, n] = sum_k x[t, k] w[n, k] + bias[n]
 *     y[t, n] = residual[t, n] + scale act(z[t, n])
 *
 *   x         [T, K]   w [N, K]     one dtype, aligned to their elements; any row stride
 *   bias      [N] fp32 or NULL      residual [T, N] or NULL (may be y itself: same pointer,
 *                                   dtype and stride)
 *   y         [T, N], y_dtype       pre_act [T, N] dense, dtype, or NULL: receives z
 *   workspace >= kda_linear_workspace_size(p, 0) bytes, 256-byte aligned (NULL when 0)
 * bf16 operands are multiplied on tensor cores with fp32 accumulation; those whose base or rows
 * are not 16-byte aligned are first copied into aligned rows of the workspace.  fp32 operands
 * are split into three bf16 parts in the workspace (24 bits in all), whose six leading products
 * the tensor cores sum in fp32; sums that are not finite are formed again from the operands, so that
 * infinities and NaN come out as in fp32, and values below 2^-109 keep fewer than 24 bits (their
 * last part is subnormal and counts as zero).
 * KDA_FLAG_CUDA_CORES multiplies in fp32 on CUDA cores instead.  The forward of up to 2 tokens, or
 * of up to 8 where w would have to be copied, runs on CUDA cores and reads both operands in place.
 */
kda_status_t kda_linear_fwd(const kda_linear_params_t *p, const void *x, const void *w,
                            const float *bias, const void *residual, void *y, void *pre_act,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward of kda_linear_fwd.  With dz = scale act'(z) d_y (z as the forward wrote it):
 *
 *     dx = dz w        dw = dz^T x        dbias = sum_t dz
 *
 * and d_residual = d_y, which needs no work.
 *   d_y       [T, N], y_dtype       pre_act [T, N] dense, dtype (NULL with KDA_ACT_NONE)
 *   dx        [T, K] dense, dtype, or NULL      dw [N, K] dense, dw_dtype, or NULL
 *   dbias     [N] fp32 or NULL
 *   workspace >= kda_linear_workspace_size(p, 1) bytes, 256-byte aligned
 * With bf16 operands dz is rounded to bf16 (to nearest) before the two products, as the
 * tensor cores read it; with KDA_ACT_NONE and a bf16 d_y the products read d_y itself and scale
 * multiplies their fp32 sums.  dbias is summed from the unrounded dz.  Where dz
 * is rounded, dx and dw carry its rounding beside their own, some 1.4 times the error of their own
 * alone; fp32 operands keep dz whole.
 */
kda_status_t kda_linear_bwd(const kda_linear_params_t *p, const void *x, const void *w,
                            const void *pre_act, const void *d_y, void *dx, void *dw, float *dbias,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of kda_linear_fwd (backward = 0) or kda_linear_bwd (backward = 1). */
kda_status_t kda_linear_workspace_size(const kda_linear_params_t *p, int32_t backward,
                                       size_t *bytes);

typedef struct kda_norm_params {
  int64_t tokens;         /* T */
  int32_t features;       /* N of residual_norm (1..16384); head size D of gated_norm (1..1024) */
  int32_t num_heads;      /* gated_norm: H >= 1; residual_norm: ignored */
  int32_t x_dtype;        /* x, y, d_y, dx, a per-token gate; gated_norm: of o and d_o */
  int32_t h_dtype;        /* residual_norm: residual, h, d_h, d_residual */
  int32_t gate_dtype;     /* gated_norm: gate, d_gate; residual_norm: ignored */
  int32_t y_dtype;        /* y, d_y */
  int32_t gate_per_token; /* residual_norm: gate is [T, N] (nonzero) or [N] fp32 (zero) */
  int32_t activation;     /* gated_norm: KDA_ACT_SIGMOID, KDA_ACT_SILU or KDA_ACT_NONE */
  float eps;              /* > 0: added to the mean square */
  float scale;            /* residual_norm: the residual scale s */
  int64_t gate_row_stride; /* elements between tokens of a per-token gate; 0 means dense */
} kda_norm_params_t;

/*
 * The norms around a block in one pass: the (optional) norm of the block's output, its gate and
 * residual scale, the residual add, and the norm before the next block.  Per token, with
 * rms(a) = a / sqrt(mean(a^2) + eps):
 *
 *     u = post_weight ? rms(x) post_weight : x
 *     h = residual + scale gate u
 *     y = rms(h) weight                                (from the fp32 h, before its rounding)
 *
 *   x [T, N], x_dtype               residual [T, N], h_dtype, or NULL (zero)
 *   gate [N] fp32 or [T, N] x_dtype, or NULL (one)
 *   post_weight, weight [N] fp32; post_weight may be NULL; weight and y may be NULL together
 *   h [T, N], h_dtype, or NULL      y [T, N], y_dtype
 * Rows are dense but a per-token gate's, aligned to their elements.  h may be residual, and y
 * or h may be x, when the dtypes agree.
 */
kda_status_t kda_residual_norm_fwd(const kda_norm_params_t *p, const void *x, const void *residual,
                                   const void *gate, const float *post_weight,
                                   const float *weight, void *h, void *y, void *stream);

/*
 * Backward of kda_residual_norm_fwd, given h as the forward wrote it (or, without anything to
 * add, x itself as h):
 *
 *     dh = d_h + rms'(h)^T (d_y weight)     d_residual = dh      d_weight = sum_t d_y rms(h)
 *     du = scale gate dh                    d_gate = scale u dh  (summed over t for [N])
 *     dx = post_weight ? rms'(x)^T (du post_weight) : du         d_post_weight = sum_t du rms(x)
 *
 *   d_y [T, N], y_dtype, or NULL with weight = NULL; d_h [T, N], h_dtype, or NULL (zero)
 *   dx [T, N], x_dtype        d_residual [T, N], h_dtype, or NULL (may be d_h)
 *   d_gate like gate          d_weight, d_post_weight [N] fp32
 *   (d_gate, d_weight, d_post_weight: needed when gate, weight, post_weight are given)
 *   workspace >= kda_norm_workspace_size bytes, 256-byte aligned
 * The sums over tokens are formed in a fixed order: repeated calls give the same bits.
 */
kda_status_t kda_residual_norm_bwd(const kda_norm_params_t *p, const void *x, const void *h,
                                   const void *gate, const float *post_weight,
                                   const float *weight, const void *d_y, const void *d_h, void *dx,
                                   void *d_residual, void *d_gate, float *d_post_weight,
                                   float *d_weight, void *workspace, size_t workspace_bytes,
                                   void *stream);

/*
 * The output norm of the recurrence: per token and head
 *
 *     y[t, h] = rms(o[t, h]) weight act(gate[t, h])
 *
 *   o [T, H, D], x_dtype (fp32 as kda_prefill_fwd writes it)
 *   gate [T, H, D], gate_dtype, rows of H * D elements gate_row_stride apart
 *   weight [D] fp32      y [T, H, D], y_dtype
 */
kda_status_t kda_gated_norm_fwd(const kda_norm_params_t *p, const void *o, const void *gate,
                                const float *weight, void *y, void *stream);

/*
 * Backward of kda_gated_norm_fwd: d_o [T, H, D] x_dtype (fp32: what kda_prefill_bwd takes as
 * d_o), d_gate [T, H, D] dense, gate_dtype, d_weight [D] fp32 (in a fixed order).
 * workspace >= kda_norm_workspace_size bytes, 256-byte aligned.
 */
kda_status_t kda_gated_norm_bwd(const kda_norm_params_t *p, const void *o, const void *gate,
                                const float *weight, const void *d_y, void *d_o, void *d_gate,
                                float *d_weight, void *workspace, size_t workspace_bytes,
                                void *stream);

/* Workspace bytes of kda_residual_norm_bwd (gated = 0) or kda_gated_norm_bwd (gated = 1). */
kda_status_t kda_norm_workspace_size(const kda_norm_params_t *p, int32_t gated, size_t *bytes);

/*
 * The key-value cache of a hybrid model's softmax attention layers, which stand between the
 * recurrent ones.  The cache of a layer is two pools of pages (keys and values): page q, row r and
 * key head h at element q page_stride + r page_row_stride + h page_head_stride, head_dim
 * elements each, so that [num_pages, page_size, HK, d], [num_pages, HK, page_size, d] and any other order are read
 * in place.  A sequence's token j lies in row j % page_size of page block_table[b][j / page_size];
 * one table serves all layers.  Entries that a call does not need are not read and may hold -1.
 *
 * Problems only the device can see (a page, length or position out of range) set KDA_DEVERR_PAGE;
 * what they touch is then skipped: an append writes no row, an attention reads zeros in place of a page and
 * takes a sequence whose length does not fit its row of the table for an empty one, an update or a compaction changes
 * nothing.
 */

/* Rotary positions.  head_dim 1..1024, rot_dim even, 0 < rot_dim <= head_dim. */
typedef struct kda_rotary_params {
  int64_t tokens;         /* T */
  int32_t num_q_heads;    /* H >= 0 */
  int32_t num_k_heads;    /* HK >= 0 */
  int32_t head_dim;       /* d */
  int32_t rot_dim;        /* R: channels turned; those from R on pass */
  int32_t dtype;          /* kda_dtype_t of q, k and the outputs */
  int32_t interleaved;    /* pairs (2i, 2i + 1); otherwise (i, i + R / 2) */
  int32_t wide_positions; /* positions are int64 (nonzero) or int32 */
  float magnitude;        /* m */
  /* elements between tokens; 0 means dense */
  int64_t q_row_stride, k_row_stride, q_out_row_stride, k_out_row_stride;
} kda_rotary_params_t;

/*
 * Turns each pair (a, b) of a head's channels at position p by the angle p frequencies[i]:
 *
 *     (a, b) -> m (a cos - b sin, b cos + a sin)
 *
 *   q [T, H, d], k [T, HK, d] (NULL with no heads)   positions [T], negative ones too; the angle is
 *   off by up to 2^-28 + |p f| 2^-55 of a turn       frequencies [R / 2] fp64, radians per position
 *   q_out, k_out: may be q, k (same pointer and stride); otherwise they share no memory with q, k or one another
 * kda_rotary_bwd is the transposed map, for gradients.
 */
kda_status_t kda_rotary_fwd(const kda_rotary_params_t *p, const void *q, const void *k,
                            const void *positions, const double *frequencies, void *q_out,
                            void *k_out, void *stream);
kda_status_t kda_rotary_bwd(const kda_rotary_params_t *p, const void *d_q, const void *d_k,
                            const void *positions, const double *frequencies, void *dq_out,
                            void *dk_out, void *stream);

typedef struct kda_cache_params {
  int64_t tokens;         /* append: T, rows of q, k and v; attention: ignored */
  int32_t num_seqs;       /* B */
  int32_t num_q_heads;    /* H: a multiple of HK */
  int32_t num_kv_heads;   /* HK */
  int32_t head_dim;       /* d: append 1..1024; attention a multiple of 16 bytes up to 256 elements */
  int32_t rot_dim;        /* append: R, as in kda_rotary_params_t; 0 turns nothing */
  int32_t dtype;          /* kda_dtype_t of q, k, v and the pages (append: of q_out) */
  int32_t o_dtype;        /* attention: kda_dtype_t of o */
  int32_t interleaved;    /* append: as in kda_rotary_params_t */
  int32_t page_size;      /* rows of a page, >= 1 */
  int32_t max_pages;      /* entries of a block_table row */
  int32_t num_pages;      /* pages of the pools */
  int32_t window;         /* attention: queries per sequence, 1..64 */
  int32_t span;           /* attention: keys a query sees, its own included; 0 means all */
  float magnitude;        /* append: m */
  float scale;            /* attention: 0 means 1 / sqrt(d) */
  float softcap;          /* attention: cap of the scores, 0 means none */
  int64_t q_row_stride, k_row_stride, v_row_stride, q_out_row_stride; /* elements; 0 means dense */
  int64_t page_stride, page_row_stride, page_head_stride;             /* elements; of both pools */
} kda_cache_params_t;

/*
 * New tokens into the cache: q and k turned (as kda_rotary_fwd), k and v written into the pages.
 * Token t of sequence b, the i-th of its new ones, stands at position start[b] + i.
 *
 *   q [T, H, d] or NULL (H = 0)     k, v [T, HK, d]
 *   input_row_offsets [B + 1], or NULL: one token per sequence (T = B).  Tokens from its last entry on
 *   belong to no sequence; nothing of them is written
 *   frequencies [R / 2] or NULL (R = 0)      q_out [T, H, d], may be q
 *   start [B] tokens already in the cache
 * The pages of the new positions must be in the table.  A page row that two tokens are given races.  The two pools
 * share no memory, and none with q, k, v or q_out.
 */
kda_status_t kda_cache_append(const kda_cache_params_t *p, const void *q, const void *k, const void *v,
                              const double *frequencies, void *key_pages, void *value_pages,
                              const int32_t *block_table, const int32_t *start,
                              const uint32_t *input_row_offsets, void *q_out, void *stream);

/*
 * Attention of a window of W queries per sequence (W = 1: a decode step) over its cache.  Query w of
 * sequence b is row b W + w, at position p = lens[b] - W + w; its own key is in the cache.  For head
 * h, key head h / (H / HK):
 *
 *     s_j = c(scale q . k_j) + slopes[h] (j - p)      max(0, p - span + 1) <= j <= p
 *     o = softmax(s) v,   lse = log sum_j e^(s_j)     c(x) = softcap tanh(x / softcap)
 *
 *   q [B W, H, d]      lens [B]: tokens in the cache, the window's included
 *   slopes [H] fp32 or NULL      o [B W, H, d] dense, o_dtype      lse [B W, H] fp32 or NULL
 *   workspace >= kda_cache_attention_workspace_size(p) bytes, 256-byte aligned; calls that may run at
 *   the same time need one each
 * A query that sees no key (p < 0, an empty sequence) gets o = 0 and lse = -infinity.  What a query
 * does not see does not reach it, NaN and infinities included.  Scores, sums and o are formed in
 * fp32; with bf16 pages the products are exact and the softmax's weights multiply v with 16 bits, with 24 where o is
 * fp32.  Pages, their strides and q are 16-byte aligned.  Repeated calls give the same bits.  KDA_ERR_UNSUPPORTED:
 * tables so wide that B HK max_pages page_size passes some 2^33 (2^36 / rows of a key head).
 */
kda_status_t kda_cache_attention(const kda_cache_params_t *p, const void *q, const void *key_pages,
                                 const void *value_pages, const int32_t *block_table,
                                 const int32_t *lens, const float *slopes, void *o, float *lse,
                                 void *workspace, size_t workspace_bytes, void *stream);
kda_status_t kda_cache_attention_workspace_size(const kda_cache_params_t *p, size_t *bytes);

typedef struct kda_cache_rows_params {
  int32_t rows;      /* S: rows of the table as it is */
  int32_t rows_out;  /* update: rows of the new table; compact: ignored */
  int32_t max_pages; /* entries of a row */
  int32_t page_size;
  int32_t num_pages;
} kda_cache_rows_params_t;

/*
 * A cache's tables from one step to the next.  Row r holds lens[r] tokens; refs[q] counts the
 * references to page q, the table's and any others; a page is free where it is 0.  New row i goes
 * on from row parent[i] (-1: from nothing) with its first kept[i] = min(lens[parent[i]], new_lens[i])
 * tokens, and has pages for new_lens[i].  So a row goes on (parent i), forks (several rows of one
 * parent), is cut back (a shorter new_lens), grows, begins, or ends (no row goes on from it).
 *
 *   - Pages that the kept tokens fill are shared.  A page that they end inside is kept by the lowest
 *     row that ends in it, if no full row and no one outside the table refers to it; the other rows get a fresh
 *     page there and a line in the list of copies, for kda_cache_copy.
 *   - Fresh pages are the free ones from the lowest on, row by row.  Pages that this call frees are
 *     not handed out by it.
 *   - The old tables are left as they are, and valid: only pages that they hold free are handed out.
 *
 *   block_table [S, max_pages]   lens [S]   refs [num_pages]   parent [rows_out] or NULL (row i from
 *   row i; rows_out = rows)      new_lens [rows_out]
 *   out_table [rows_out, max_pages], -1 behind a row's pages   out_lens, kept [rows_out]   out_refs
 *   [num_pages]   copy_src, copy_dst [rows_out]: the copies, then -1
 *   workspace >= kda_cache_rows_workspace_size bytes, 256-byte aligned
 * An entry of -1 among a row's pages is one that it has given back (behind a span): it stays -1.
 * The outputs share no memory with the inputs.  With KDA_DEVERR_PAGE (a row that names a free page or one that is
 * not there, and not enough free pages, among its reasons) the new rows are empty, out_refs is refs and nothing is to be
 * copied.  refs has to count every reference of the table.  A page that is held more often than it says is
 * found where it says 0 or where its count would fall below 0; otherwise it is not, and becomes free too early.
 */
kda_status_t kda_cache_update(const kda_cache_rows_params_t *p, const int32_t *block_table,
                              const int32_t *lens, const int32_t *refs, const int32_t *parent,
                              const int32_t *new_lens, int32_t *out_table, int32_t *out_lens,
                              int32_t *out_refs, int32_t *kept, int32_t *copy_src,
                              int32_t *copy_dst, void *workspace, size_t workspace_bytes,
                              void *stream);

/*
 * Used pages to the front of the pools: of n pages in use, the k-th from page n on goes to the k-th
 * free page before n.
 *   out_table [S, max_pages], out_refs [num_pages]: with the pages' new places
 *   page_map [num_pages]: where each page goes, -1 for a free one
 *   copy_src, copy_dst [num_pages / 2]: the moves, then -1
 * Workspace, outputs and the old tables' validity as in kda_cache_update; with KDA_DEVERR_PAGE
 * (a row naming a free page) every page stays.
 */
kda_status_t kda_cache_compact(const kda_cache_rows_params_t *p, const int32_t *block_table,
                               const int32_t *lens, const int32_t *refs, int32_t *out_table,
                               int32_t *out_refs, int32_t *page_map, int32_t *copy_src,
                               int32_t *copy_dst, void *workspace, size_t workspace_bytes,
                               void *stream);
kda_status_t kda_cache_rows_workspace_size(const kda_cache_rows_params_t *p, size_t *bytes);

/*
 * pool[dst[i]] = pool[src[i]] for each i before the list's first negative src (behind which all are
 * negative), for each of num_pools pools of num_pages pages: pages of a cache, or slots of a state or
 * convolution pool (a forked sequence's recurrent state).  Page q of pool j is page_bytes[j] bytes at
 * pools[j] + q page_strides[j].
 *   pools, page_bytes, page_strides   HOST arrays of num_pools entries
 *   src, dst [n] int32
 * No page may be written twice or both read and written; an index >= num_pages (or a negative dst)
 * sets KDA_DEVERR_PAGE and is skipped.
 */
kda_status_t kda_cache_copy(void *const *pools, const int64_t *page_bytes,
                            const int64_t *page_strides, int32_t num_pools, const int32_t *src,
                            const int32_t *dst, int64_t n, int32_t num_pages, void *stream);

/*
 * Measurement aid (no counterpart on the pages).  Registers up to 8 CUDA events
 * (cudaEvent_t handles passed as void*, created by the caller) that later
 * kda_prefill_fwd / kda_decode_step calls on this process record on their
 * stream: events[0] before the first kernel, events[i] after the i-th kernel.
 * Lets a benchmark time each kernel with CUDA events on the stream the kernel
 * runs on.  count = 0 (or events = NULL) clears the registration.  The handles
 * must stay valid while registered; calls from several threads share it.
 * Returns KDA_ERR_INVALID_ARG for count < 0 or > 8.
 */
kda_status_t kda_set_stage_events(void *const *events, int32_t count);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
