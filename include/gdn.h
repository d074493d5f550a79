/*
 * libgdn -- gated delta-rule linear-attention scan for AMD Instinct MI355X (gfx950).
 *
 * The operator is the gated delta-net linear attention with a matrix-valued
 * recurrent state per head ("[Research] Explore linear attention for the
 * streaming video models", section "We already ship a hybrid linear-attention
 * model"); the state is written one token at a time as standard delta-rule
 * linear attention does ("Video DeltaNet: A Video-Native Hybrid Attention for
 * Livestream Video Generation", section "Methodology in Plain English").
 * Per (batch b, head h), with the state S in R^{dv x dk} (fp32):
 *
 *   q^_t = q_t / max(|q_t|_2, 1e-6),   k^_t = k_t / max(|k_t|_2, 1e-6)
 *   S_t  = a_t S_{t-1} (I - beta_t k^_t k^_t^T) + beta_t v_t k^_t^T,  a_t = exp(log_alpha_t)
 *   o_t  = S_t q^_t
 *
 * Directions:
 *   GDN_DIR_FORWARD       causal scan t = 0..T-1; the forward-only causal
 *                         form used for streaming rollout (the issue's
 *                         "Open questions and risks": causal streaming scan).
 *   GDN_DIR_REVERSE       the same recurrence run from t = T-1 down to 0.
 *   GDN_DIR_BIDIRECTIONAL out = forward readout + reverse readout, each
 *                         direction with its own (log_alpha, beta) and its own
 *                         initial state ("Video DeltaNet", "Methodology in
 *                         Plain English": forward and backward recurrent
 *                         states whose readouts are added).  Both readouts
 *                         include the current token unless an exclusive
 *                         option bit (below) says otherwise.
 *
 * Streaming: the final state of one call is the initial state of the next
 * (the streaming state lifecycle of the issue's "Suggested phases", phase 1);
 * chaining calls over consecutive token ranges equals one call over their
 * concatenation.
 *
 * Layouts (all row-major and contiguous; base pointers 16-byte aligned):
 *   q, k       [B, T, H, dk]   dtype (fp32 or bf16), finite (any length:
 *                              the scan normalises them itself)
 *   v          [B, T, H, dv]   dtype, finite
 *   log_alpha  [dirs, B, T, H] fp32, finite and <= 0 (caller's contract)
 *   beta       [dirs, B, T, H] fp32, finite (beta in [0,1] keeps the
 *                              transition non-expansive)
 *   state_in   [dirs, B, H, dv, dk] fp32, or NULL for a zero initial state
 *   state_out  [dirs, B, H, dv, dk] fp32, or NULL to skip writing it
 *   out        [B, T, H, dv]   fp32
 * dirs = 2 for GDN_DIR_BIDIRECTIONAL, else 1 (slot 0 then holds the single
 * direction's gates and states).
 *
 * Ownership and execution: every pointer is caller-owned device memory; the
 * library allocates no device memory, does not synchronise and reads no
 * environment variables.  The work is ordered on `stream` (NULL: the default
 * stream) and completes asynchronously.  For long single-direction scans
 * whose state chain leaves compute units free (and fp32 bidirectional ones
 * with few sequences) the chunk
 * preparation runs concurrently with the state chain, on a library stream
 * forked from `stream` and joined back to it with events (one stream and two
 * events per device, created on the first such call and kept until the
 * process ends): the work still starts after earlier work on `stream`, and
 * later work on `stream` still waits for all of it.  While `stream` is being
 * captured into a HIP graph, both kernels are enqueued one after the other on
 * `stream` (no library stream or event is created or used), so a captured
 * call -- the first call of the process included -- replays the serial order.
 * GDN_OPT_SERIAL keeps everything on `stream` always.
 * Calls may come from several host threads at once, each with its own
 * buffers and workspace: the library stream and events are shared under a
 * lock, and the preparation passes of concurrent calls run one after another
 * on that stream (results are those of the same calls made one at a time).
 * state_in == state_out is allowed (in-place streaming carry); any other
 * overlap between `out`, the state buffers, the workspace and the inputs is
 * rejected.  Results are bitwise deterministic for fixed inputs and chunk
 * size, concurrent or not: there are no atomic reductions (the second visit
 * of a chunk in a bidirectional scan adds the stored readout of the first
 * visit in a fixed order; it waits for that readout's flag for about a
 * second at most, after which the outputs it could not combine are NaN).  The value-tile width changes the schedule, never
 * the arithmetic.
 *
 * Errors: argument problems are reported before anything is enqueued and
 * leave every output untouched.  GDN_ERR_HIP reports a failed launch; faults
 * during execution surface at the caller's next synchronisation, as with any
 * stream work.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARGUMENT = 1,   /* NULL/misaligned pointer, bad size, overlap, bad direction */
  GDN_ERR_UNSUPPORTED = 2,        /* dk, dv, chunk, tile or dtype outside the compiled set */
  GDN_ERR_WORKSPACE_TOO_SMALL = 3,
  GDN_ERR_HIP = 4                 /* a kernel launch failed */
} gdn_status_t;

typedef enum {
  GDN_DIR_FORWARD = 0,
  GDN_DIR_REVERSE = 1,
  GDN_DIR_BIDIRECTIONAL = 2
} gdn_direction_t;

typedef enum {
  GDN_DTYPE_F32 = 0,
  GDN_DTYPE_BF16 = 1
} gdn_dtype_t;

/* Bits of gdn_problem_t.options. */
typedef enum {
  GDN_OPT_SERIAL = 1,       /* run both kernels one after the other on `stream` */
  GDN_OPT_NO_ERASE = 2,     /* the erase-free variant: S_t = a_t S_{t-1} + beta_t v_t k^_t^T,
                               i.e. gated linear attention with per-token write strength
                               beta (SANA-Video 2.0 review: the hybrid's linear layers are
                               gated linear attention, and its "Future work" relates them to
                               the delta rule by dropping the delta-rule update) */
  GDN_OPT_EXCLUSIVE_FORWARD = 4,  /* the forward direction reads its memory before the
                               token's own write: o_t = a_t S_{t-1} q^_t */
  GDN_OPT_EXCLUSIVE_REVERSE = 8   /* the same for the reverse direction: o_t = a_t S_{t+1} q^_t.
                               Both bits: the two scans of a bidirectional call cover the
                               disjoint regions s < t and s > t (the current token is left to
                               a local operator); the reverse bit alone: s <= t and s > t,
                               every token once ("Video DeltaNet", "Methodology in Plain
                               English": each direction sees its own non-overlapping part
                               of the sequence, and the prompt's state enters each
                               direction at half weight, S_T / 2 -- here the caller's
                               state_in).
                               Final states are unchanged by either bit. */,
  GDN_OPT_TEST_NO_PREPARATION = 1 << 16  /* testing only: the chunk preparation pass is not
                               launched, so the state chain waits on ready flags that never
                               clear; its bounded waits expire (about a second) and every
                               output and final state is NaN.  This exercises the behaviour
                               under a preparation pass starved of the GPU: results that
                               cannot be trusted are NaN, never silently wrong. */
} gdn_option_t;

/* Problem description.  Supported: dk in {64, 128}; dv in {64, 128};
 * chunk in {0 (= 64), 16, 32, 64, 128} (the chunked form is exact at any chunk
 * length: "Video DeltaNet", Key Contributions item 4, chunk-wise scans; results
 * agree between chunk lengths to rounding, 64 is the fastest on MI355X);
 * dv_tile in {0, 16, 32} (0: 32 when 16-wide
 * state-chain workgroups would outnumber the compute units of the current
 * device, else 16; exclusive readouts on bf16 operands take 16 and reject
 * 32: they carry the state and the decayed q.k tile as bf16 hi + lo parts,
 * whose staging fits 16-column tiles only).  16- and 128-token chunks: bf16
 * operands reject the exclusive readouts and the readout epilogue (their low
 * parts are carried by the 32/64-token chain only); 128-token chunks: fp32
 * operands with dk = 128
 * take dv_tile 16 and reject 32 (the chain's staging would exceed a compute
 * unit's LDS); B, H >= 1, B*H <= 65535;
 * 0 <= T <= 2^30 and
 * (T + 64) * H * max(dk, dv) * 4 < 2^32 (one batch element's rows, fp32,
 * fit 32-bit byte offsets). */
typedef struct {
  int64_t B, T, H, dk, dv;
  int32_t dtype;            /* gdn_dtype_t: type of q, k, v */
  int32_t chunk;            /* tokens per chunk of the chunked evaluation */
  int32_t dv_tile;          /* value columns per workgroup of the state chain */
  int32_t options;          /* OR of gdn_option_t bits (0: delta rule, chosen schedule);
                               other bits are invalid */
  void* workspace;          /* caller-owned device memory, 256-byte aligned */
  size_t workspace_bytes;
  void* stream;             /* hipStream_t; NULL = default stream */
  void* timing_events;      /* NULL, or hipEvent_t[4] (caller-owned): recorded
                               before and after the chunk-preparation kernel on
                               the stream it runs on, then before and after the
                               state-chain kernel on `stream` (per-kernel
                               timing; the epilogue, if any, runs after the
                               last of them) */
  /* Readout epilogue ("Video DeltaNet", "Key Contributions" item 1: the
   * linear branch's readout is RMS-normalised and sigmoid-gated).  With
   * gate != NULL, after the scan, every (token, head) row of `out` becomes
   *   out = norm_weight * o / sqrt(mean_dv(o^2) + norm_eps) * sigmoid(gate),
   * o being the row as the scan computed it (inclusive or exclusive, both
   * directions summed).  A separate pass on `stream`: the channels of one
   * row are split over several state-chain workgroups.  Zero-initialise
   * these fields (as make_problem-style helpers do) for no epilogue. */
  const void* gate;          /* NULL, or [B, T, H, dv] of the type of q, 16-byte aligned */
  const float* norm_weight;  /* [dv] fp32, shared by the heads; required with gate */
  float norm_eps;            /* epilogue only: finite, >= 0 */
} gdn_problem_t;

/* Bytes of workspace gdn_forward needs for this problem and direction
 * (0 if the problem is invalid or unsupported, and for T = 0, which needs
 * none).  It depends on p->options as well: exclusive readouts on bf16
 * operands need about 2 C bytes more per token and head.  Pure host
 * arithmetic. */
size_t gdn_workspace_bytes(const gdn_problem_t* p, int32_t direction);

/* Enqueue the scan described by `p` on p->stream.  See the file comment for
 * layouts; `direction` is a gdn_direction_t. */
gdn_status_t gdn_forward(const gdn_problem_t* p,
                         const void* q, const void* k, const void* v,
                         const float* log_alpha, const float* beta,
                         const float* state_in, float* state_out,
                         float* out, int32_t direction);

/* ---- The same scan without a caller-provided workspace ----------------------
 *
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the
 * workspace is a fixed array the library holds in device memory,
 * GDN_NOALLOC_SCRATCH_BYTES per device that loads the library, kept until the
 * process ends.  Arguments, layouts, results and errors are those of
 * gdn_forward, except:
 *  - p->workspace and p->workspace_bytes are ignored;
 *  - a problem whose workspace (gdn_workspace_bytes) exceeds
 *    GDN_NOALLOC_SCRATCH_BYTES is rejected with GDN_ERR_WORKSPACE_TOO_SMALL
 *    before anything is enqueued (e.g. 480p streaming frames of 1560 tokens at
 *    12 heads need about 6 MB; a whole 480p bidirectional block, about 300 MB,
 *    does not fit);
 *  - both kernels always run one after the other on p->stream (no library
 *    stream or event is created);
 *  - the first call on a device looks up that device's array
 *    (hipGetSymbolAddress); no call allocates device memory.
 * Every call on one device uses that device's single array, which keeps the
 * last call's contents: calls that overlap in time on one device (on
 * different streams, or from several host threads) race on it and must be
 * ordered by the caller.  Nothing in the array has to start at zero. */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

gdn_status_t gdn_forward_noalloc(const gdn_problem_t* p,
                                 const void* q, const void* k, const void* v,
                                 const float* log_alpha, const float* beta,
                                 const float* state_in, float* state_out,
                                 float* out, int32_t direction);

/* ---- Frame-wise delta operator (Video Delta Attention) ---------------------
 *
 * The memory is written once per latent frame instead of once per token.
 * The write is a regularised least-squares problem: the new memory balances
 * its squared distance from the decayed previous memory against the squared
 * recall errors of all the frame's keys at once ("Video DeltaNet", "Key
 * Contributions" item 2 and "Methodology in Plain English").  Its solution is
 * the page's closed form
 *
 *   S_t = (a_t S_{t-1} + B_t) (I + A_t)^{-1},
 *   A_t = sum_{i in frame t} beta_i k^_i k^_i^T,  B_t = sum_{i in frame t} beta_i v_i k^_i^T,
 *
 * and every token i of frame t reads o_i = S_t q^_i (q^, k^ normalised as
 * above).  Frames are consecutive runs of `frame` tokens (the last may be
 * shorter).  One decay per frame, a_t = exp(log_alpha_t); one write strength
 * per token (beta >= 0 keeps the transition non-expansive).  Directions as for
 * gdn_forward: the reverse scan visits the frames last to first, the
 * bidirectional output is the sum of both readouts.
 *
 * Options on the same machinery:
 *  - GDN_VDA_OPT_ADDITIVE: the additive frame write the page contrasts the
 *    operator with ("Main Findings", last item: SANA-WM's batched per-token
 *    corrections with 1/sqrt(U) key scaling, U = the frame's token count):
 *    S_t = a_t S_{t-1} (I - A_t / U) + B_t / sqrt(U).
 *  - readout_lag = d > 0: the disjoint-region readout ("Methodology in Plain
 *    English": the forward and reverse memories see non-overlapping parts of
 *    the video, and the text's state starts each direction at half weight,
 *    S_T/2).  A token of
 *    frame t reads the forward state after frame t - d and the reverse state
 *    after frame t + d; where that frame does not exist, the direction's
 *    initial state (zero without state_in).  d = 0 reads its own frame's state.
 *  - gate != NULL: the readout epilogue ("Key Contributions" item 1: the
 *    linear branch's RMS normalisation and sigmoid gate), applied to the
 *    summed readout o of each (token, head) before it is stored:
 *    out = norm_weight * o / sqrt(mean_dv(o^2) + norm_eps) * sigmoid(gate).
 *
 * Layouts: q, k, v, beta, state_in, state_out and out as for gdn_forward;
 *   log_alpha  [dirs, B, NF, H] fp32, NF = ceil(T / frame);
 *   gate       [B, T, H, dv] of the type of q (16-byte aligned);
 *   norm_weight [dv] fp32, shared by the heads.
 * Supported: dk, dv in {64, 128}; frame >= 1; fp32 or bf16 q, k, v; the same
 * size limit as gdn_problem_t.  Same ownership, execution and error contract
 * as gdn_forward (everything on `stream`; no allocation; no synchronisation;
 * `out` must not overlap any input, gate and norm_weight included). */
typedef enum { GDN_VDA_OPT_ADDITIVE = 1 } gdn_vda_option_t;

typedef struct {
  int64_t B, T, H, dk, dv;
  int64_t frame;            /* tokens per frame */
  int32_t dtype;            /* gdn_dtype_t: type of q, k, v and gate */
  int32_t options;          /* 0 or GDN_VDA_OPT_ADDITIVE */
  int32_t readout_lag;      /* >= 0 */
  float norm_eps;           /* epilogue only: finite, >= 0 */
  const void* gate;         /* NULL (no epilogue) or [B, T, H, dv] */
  const float* norm_weight; /* [dv]; required with gate */
  void* workspace;          /* caller-owned device memory, 256-byte aligned */
  size_t workspace_bytes;
  void* stream;             /* hipStream_t; NULL = default stream */
  void* timing_events;      /* NULL, or hipEvent_t[4] (caller-owned), recorded on
                               `stream` before the per-frame kernel, after it,
                               after the frame chain and after the readout */
} gdn_vda_problem_t;

/* Workspace bytes of gdn_vda_forward (0 if invalid or unsupported, or T = 0):
 * three fp32 matrices per frame, head and direction. */
size_t gdn_vda_workspace_bytes(const gdn_vda_problem_t* p, int32_t direction);

/* Enqueue the frame-wise operator described by `p` on p->stream. */
gdn_status_t gdn_vda_forward(const gdn_vda_problem_t* p,
                             const void* q, const void* k, const void* v,
                             const float* log_alpha, const float* beta,
                             const float* state_in, float* state_out,
                             float* out, int32_t direction);

/* ---- What a recurrent layer runs around its scan, and its single-token form --
 *
 * The short causal convolution in front of the scan, rotary positions on q
 * and k, the other common recurrent scan (a selective state space), and the
 * single-token steps of these recurrences.  Everything below runs on the
 * problem's `stream`, allocates nothing, does not synchronise, can be captured
 * into a graph, and uses no atomics: results are bitwise deterministic.
 * Calls whose workspaces or states overlap must be ordered by the caller.
 * Errors as for gdn_forward: a rejected call leaves every buffer untouched.
 *
 * Rows and strides.  An operand described with strides holds, for sequence b
 * and token t, one row of contiguous channels at element b * stride_b +
 * t * stride_t (strides in elements, >= 0); base pointers need only the
 * alignment of their type.  Aligned operands are faster: 16-byte aligned
 * pointers and strides that keep every row so.  The rows of an output must
 * not meet each other, nor any row of another operand (rows of one wider
 * buffer that lie beside each other may share it), except where an in-place
 * call is allowed.
 *
 * Packed batches.  With seq_offsets != NULL ([B + 1] int32 in device memory,
 * from 0 rising to at most T), sequence b is the rows seq_offsets[b] ..
 * seq_offsets[b+1] - 1 of buffers of T rows; stride_b is not used.  A sequence
 * may be empty; rows behind the last sequence are not touched.  Offsets
 * outside 0..T are clamped to it, so no call reads or writes out of bounds.
 * Without it every sequence has T tokens.
 *
 * State slots.  A recurrent state lives in one of `slots` rows of a state
 * buffer.  With state_index != NULL ([B] int32 in device memory), sequence b
 * uses row state_index[b]; an index outside 0..slots-1 means no state (a
 * prompt then starts from zero and writes no final state; a step skips the
 * row: its output row and every state stay as they were).  No two sequences
 * of one call may name the same slot.  Without it, slots = B and sequence b
 * uses row b.
 *
 * Rows of no sequence.  GDN_LAYER_OPT_ZERO_UNUSED, an option of the calls with
 * packed batches or slots, sets the rows of `out` that the paragraphs above
 * leave alone (behind the last sequence; of a step without a slot) to zero: for
 * an output that holds nothing yet.
 *
 * A float parameter pointer is fp32; x-like operands are fp32 or bf16
 * (`dtype`).  All arithmetic is fp32 with one rounding at the end. */

typedef enum { GDN_LAYER_OPT_ZERO_UNUSED = 256 } gdn_layer_option_t;

typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 } gdn_activation_t;

/* Short causal depthwise convolution over time:
 *   y[t] = act(bias + sum_{j < width} weight[:, j] * x[t - (width - 1) + j]),
 * rows before the sequence's first coming from its state: the last width - 1
 * input rows, oldest first.
 *   x, out     rows of D channels (dtype)
 *   weight     [D, width] fp32; bias [D] fp32 or NULL
 *   state_in   [slots, width - 1, D] (dtype), or NULL for zeros
 *   state_out  the same, or NULL; may be state_in (an in-place carry)
 * Supported: width 2, 3 or 4; B, D >= 1, T >= 0. */
typedef struct {
  int64_t B, T, D;
  int64_t x_stride_b, x_stride_t;
  int64_t out_stride_b, out_stride_t;
  int64_t slots;
  int32_t dtype;             /* gdn_dtype_t: type of x, out and the states */
  int32_t width;
  int32_t activation;        /* gdn_activation_t */
  int32_t options;           /* 0 or GDN_LAYER_OPT_ZERO_UNUSED */
  const int32_t* seq_offsets;
  const int32_t* state_index;
  void* stream;
} gdn_conv_problem_t;

gdn_status_t gdn_conv_forward(const gdn_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                              const void* state_in, void* state_out, void* out);

/* One new token for each of B sequences: row b of x and out lies at element
 * b * stride_b (T, stride_t and seq_offsets are not used); `state` is read and
 * advanced in place. */
gdn_status_t gdn_conv_step(const gdn_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                           void* state, void* out);

/* Selective state space scan: per channel d an fp32 state h of N entries,
 *   dt'  = softplus(dt + dt_bias)   (without GDN_SSM_OPT_SOFTPLUS: dt + dt_bias)
 *   h_n  = exp(dt' A[d, n]) h_n + dt' x B[t, g, n]
 *   y    = sum_n h_n C[t, g, n] + skip[d] x
 *   out  = y * z * sigmoid(z)       (without z: y)
 * with g = d / (D / G), the group of the channel.
 *   x, dt, z, out  rows of D channels (dtype); z may be NULL
 *   A              [D, N] fp32, <= 0 with dt' >= 0 (caller's contract: a
 *                  decay above 1 overflows)
 *   Bm, Cm         rows of G * N contiguous elements (dtype)
 *   dt_bias, skip  [D] fp32, or NULL
 *   state_in       [slots, D, N] fp32, or NULL for zeros
 *   state_out      the same, or NULL; may be state_in (an in-place carry)
 * Supported: 1 <= N <= 256, G divides D, stride_t < 2^26. */
typedef enum { GDN_SSM_OPT_SOFTPLUS = 1 } gdn_ssm_option_t;

typedef struct {
  int64_t B, T, D, N, G;
  int64_t x_stride_b, x_stride_t;
  int64_t dt_stride_b, dt_stride_t;
  int64_t z_stride_b, z_stride_t;
  int64_t b_stride_b, b_stride_t;   /* rows of Bm */
  int64_t c_stride_b, c_stride_t;   /* rows of Cm */
  int64_t out_stride_b, out_stride_t;
  int64_t slots;
  int32_t dtype;             /* gdn_dtype_t: type of x, dt, z, Bm, Cm and out */
  int32_t options;           /* of GDN_SSM_OPT_SOFTPLUS, GDN_LAYER_OPT_ZERO_UNUSED */
  const int32_t* seq_offsets;
  const int32_t* state_index;
  const void* z;
  const float* dt_bias;
  const float* skip;
  void* workspace;           /* gdn_ssm_forward: caller-owned device memory, 256-byte aligned */
  size_t workspace_bytes;
  void* stream;
} gdn_ssm_problem_t;

/* Workspace bytes of gdn_ssm_forward (0 if invalid or unsupported, or where
 * none is needed: enough sequences and channels to fill the GPU, or short
 * sequences).  It depends on the sizes and on whether seq_offsets is given.
 * Calls that may run at the same time, replayed graphs among them, need a
 * workspace each. */
size_t gdn_ssm_workspace_bytes(const gdn_ssm_problem_t* p);

gdn_status_t gdn_ssm_forward(const gdn_ssm_problem_t* p, const void* x, const void* dt, const float* A,
                             const void* Bm, const void* Cm, const float* state_in, float* state_out, void* out);

/* One new token for each of B sequences (rows at b * stride_b; T, stride_t and
 * seq_offsets are not used); `state` is read and advanced in place. */
gdn_status_t gdn_ssm_step(const gdn_ssm_problem_t* p, const void* x, const void* dt, const float* A, const void* Bm,
                          const void* Cm, float* state, void* out);

/* Rotary positions on q and k.  Pair i < rot / 2 of every head is turned by
 * the angle position * inv_freq[i], taken in 64 bits (off by at most 2^-51 of
 * itself: below fp32's rounding for angles up to 2^26), and scaled:
 *   (u, v) -> scale * (u cos - v sin, v cos + u sin)
 * in the half layout (u, v) = (x[i], x[i + rot / 2]); with
 * GDN_ROTARY_OPT_INTERLEAVED (x[2i], x[2i + 1]).  Channels from rot on pass
 * through.  GDN_ROTARY_OPT_INVERSE turns back (the gradient of the call, with
 * the same scale).
 *   q, k        head h of token (b, t) at b * stride_b + t * stride_t +
 *               h * stride_h, d contiguous channels; k may be NULL (Hk = 0)
 *   q_out,k_out the same; each may be its input, with the input's strides
 *   inv_freq    [rot / 2] fp64
 *   positions   [axes, B, T], int32 or int64 (position_bits 32 or 64), or NULL
 *               (position_bits 0, one axis): position0 + t.  With several axes
 *               the first section[0] pairs take axis 0, the next section[1]
 *               axis 1 and so on; the sections add up to rot / 2.
 * Supported: rot even, 2 <= rot <= d <= 256, 1 to 4 axes, Hq, Hk <= 65536,
 * B * T < 2^31. */
typedef enum { GDN_ROTARY_OPT_INTERLEAVED = 1, GDN_ROTARY_OPT_INVERSE = 2 } gdn_rotary_option_t;

typedef struct {
  int64_t B, T, Hq, Hk, d, rot;
  int64_t q_stride_b, q_stride_t, q_stride_h;
  int64_t k_stride_b, k_stride_t, k_stride_h;
  int64_t q_out_stride_b, q_out_stride_t, q_out_stride_h;
  int64_t k_out_stride_b, k_out_stride_t, k_out_stride_h;
  int64_t position0;
  int32_t dtype;
  int32_t options;
  int32_t position_bits;
  int32_t axes;
  int32_t section[4];        /* pairs per axis */
  float scale;
  void* stream;
} gdn_rotary_problem_t;

gdn_status_t gdn_rotary(const gdn_rotary_problem_t* p, const void* q, const void* k, const double* inv_freq,
                        const void* positions, void* q_out, void* k_out);

/* The token scan's single-token step: one token of gdn_forward (forward
 * direction) for each of B sequences, the state advanced in place:
 *   S' = a S (I - beta k^ k^T) + beta v k^T,  o = S' q^
 * with q^, k^ normalised and a = exp(log_alpha), as in gdn_forward.  Options:
 * GDN_OPT_NO_ERASE, GDN_OPT_EXCLUSIVE_FORWARD (o = a S q^) and
 * GDN_LAYER_OPT_ZERO_UNUSED; gate, norm_weight and norm_eps are gdn_problem_t's
 * readout epilogue.
 *   q, k       [B, H, dk] (dtype); v, gate [B, H, dv] (dtype), 16-byte aligned
 *   log_alpha, beta  [B, H] fp32
 *   state      [slots, H, dv, dk] fp32, 16-byte aligned
 *   out        [B, H, dv] fp32
 * Supported: dk, dv in {64, 128}, B * H < 2^31. */
typedef struct {
  int64_t B, H, dk, dv;
  int64_t slots;
  int32_t dtype;
  int32_t options;
  const int32_t* state_index;
  const void* gate;
  const float* norm_weight;
  float norm_eps;
  void* stream;
} gdn_step_problem_t;

gdn_status_t gdn_step(const gdn_step_problem_t* p, const void* q, const void* k, const void* v,
                      const float* log_alpha, const float* beta, float* state, float* out);

/* ---- A paged cache of keys and values, and a new token's attention over it ----
 *
 * The softmax block of a hybrid model keeps the keys and values of past tokens
 * in pools of pages: k_cache, v_cache [pages, Hk, page, d], contiguous, 16-byte
 * aligned.  The token at position p of sequence b lies in page
 * page_table[b, p / page] (page_table [B, table_width] int32 in device memory),
 * row p % page.  A position outside 0 .. table_width * page - 1, or whose page
 * number is outside 0 .. pages - 1, has no place: it is not written, not read
 * and not attended to.  No two tokens of one gdn_kv_write may have one place.
 *
 * Formats of a pool:
 *   GDN_KV_F32, GDN_KV_BF16  the rows' own type (`dtype`)
 *   GDN_KV_MXFP8             e4m3 codes, a byte a channel
 *   GDN_KV_MXFP4             e2m1 codes, [pages, Hk, page, d / 2] bytes, the even
 *                            channel in the low half
 * The last two hold one scale byte per 32 channels beside the codes, k_scales,
 * v_scales [pages, Hk, page, d / 32] (4-byte aligned): a byte s scales by 2^(s - 127).
 * Writing chooses the least power of two, 2^-110 or more, with which the
 * block's largest magnitude is at most 448 (6 for e2m1), and rounds x / 2^(s -
 * 127) to the nearest code, ties to even: the only rounding.  A block that
 * holds an infinity or a NaN gets byte 255 and reads back as NaN; magnitudes
 * that round to 2^128 read back as infinities.  A pool of zero bytes holds zeros.
 *
 * Supported: d 64, 128 or 256; page a power of two, 16 to 1024; Hk <= 65536;
 * B * T and B * table_width < 2^31. */
typedef enum { GDN_KV_F32 = 0, GDN_KV_BF16 = 1, GDN_KV_MXFP8 = 2, GDN_KV_MXFP4 = 3 } gdn_kv_format_t;

/* Rows of K and V into the cache, and back out of it.
 *   k, v   head h of token (b, t) at b * stride_b + t * stride_t + h * stride_h,
 *          d contiguous channels (dtype); packed with seq_offsets
 *   start  [B] int32, position of each sequence's first row; NULL: 0
 * Token t of sequence b has position start[b] + t.  gdn_kv_read leaves the rows
 * of tokens without a place, and rows of no sequence, as they were; with
 * GDN_LAYER_OPT_ZERO_UNUSED they become zero. */
typedef struct {
  int64_t B, T, Hk, d;
  int64_t pages, page, table_width;
  int64_t k_stride_b, k_stride_t, k_stride_h;
  int64_t v_stride_b, v_stride_t, v_stride_h;
  int32_t dtype;             /* gdn_dtype_t: type of the rows */
  int32_t format;            /* gdn_kv_format_t */
  int32_t options;           /* gdn_kv_read: 0 or GDN_LAYER_OPT_ZERO_UNUSED; else 0 */
  const int32_t* seq_offsets;
  const int32_t* page_table;
  const int32_t* start;
  void* stream;
} gdn_kv_problem_t;

gdn_status_t gdn_kv_write(const gdn_kv_problem_t* p, const void* k, const void* v, void* k_cache, void* v_cache,
                          void* k_scales, void* v_scales);
gdn_status_t gdn_kv_read(const gdn_kv_problem_t* p, const void* k_cache, const void* v_cache, const void* k_scales,
                         const void* v_scales, void* k, void* v);

/* Attention of one new token per sequence over the cache: query head h reads
 * head h / (Hq / Hk) of the cache, and with the visible positions p (p <
 * lengths[b], and with window > 0 only p >= lengths[b] - window or p < sinks)
 *   s_p = scale q . k_p,  out = sum_p exp(s_p) v_p / sum_p exp(s_p),
 *   lse = log(sum_p exp(s_p))
 * Where no weight is above zero (no visible position, or every score minus
 * infinity) out is zero and lse minus infinity; a score of plus infinity or NaN
 * makes its row and lse NaN.  A channel with an infinite visible value is infinite
 * in a cache of the rows' own type if that token's weight is 2^-100 of the largest
 * or more; else, as in quantised caches, infinite or NaN.  fp32 queries make NaN of
 * a quantised key that reads back as an infinity.  Weights below 2^-126 of the
 * largest count as zero.  Sums are fp32, those of q . k before the scale, those of
 * values before they are divided: finite values of 2^127 / lengths[b] or more may
 * overflow.  What lies in places that are not
 * visible, NaN included, has no influence.  lengths beyond the table's reach
 * count as that.
 *   q, out  head h of sequence b at b * stride_b + h * stride_h, d contiguous
 *           channels (dtype)
 *   lengths [B] int32; lse [B, Hq] fp32, or NULL
 * Supported: as above, Hk divides Hq, Hq <= 65536, B * Hq < 2^31. */
typedef struct {
  int64_t B, Hq, Hk, d;
  int64_t pages, page, table_width;
  int64_t q_stride_b, q_stride_h;
  int64_t out_stride_b, out_stride_h;
  int64_t window, sinks;     /* 0: all positions; sinks only with a window */
  int32_t dtype;             /* gdn_dtype_t: type of q and out */
  int32_t format;            /* gdn_kv_format_t */
  float scale;
  const int32_t* page_table;
  const int32_t* lengths;
  void* workspace;           /* caller-owned device memory, 256-byte aligned */
  size_t workspace_bytes;
  void* stream;
} gdn_attention_problem_t;

/* Workspace bytes of gdn_attention_step (0 if invalid, unsupported, or where
 * none is needed): it depends on the sizes alone.  Calls that may run at the
 * same time, replayed graphs among them, need a workspace each. */
size_t gdn_attention_workspace_bytes(const gdn_attention_problem_t* p);

gdn_status_t gdn_attention_step(const gdn_attention_problem_t* p, const void* q, const void* k_cache, const void* v_cache,
                                const void* k_scales, const void* v_scales, void* out, float* lse);

/* ---- The seam between two blocks: norm, gate, residual, norm ------------------
 *
 * Per row of D channels, x the residual stream and y a block's output:
 *   u = post_weight * y / sqrt(mean(y^2) + eps)     (post_weight NULL: u = y)
 *   h = residual_scale * x + gate * u               (gate NULL: 1)
 *   n = weight * h / sqrt(mean(h^2) + eps)          (weight NULL: no n)
 * n is computed from h before h is rounded.  Squares and their sums are fp32: a
 * row whose sum passes 2^128 norms to zero, squares below 2^-149 are lost.
 *   x, y, h, n   rows of D channels (dtype), strided, packed with seq_offsets;
 *                y may be NULL (then h = residual_scale * x; gate and
 *                post_weight NULL); h may be NULL, or x (in place)
 *   gate         [D] fp32 (gate_stride_b 0), or [B, D] (gate_stride_b D)
 *   weight, post_weight  [D] fp32
 * The backward call takes the gradients dh (NULL: zero) and dn (with weight),
 * at h's and n's strides, and gives
 *   dx, dy               rows (dtype) at strides of their own; dy with y; dx may be dh
 *   dgate                like gate; dpost_weight, dweight [D] fp32
 * each NULL where it is not wanted.  Sums over rows are fp32 in a fixed order.
 * Supported: D <= 16384, B * T < 2^31, eps finite and >= 0. */
typedef struct {
  int64_t B, T, D;
  int64_t x_stride_b, x_stride_t;
  int64_t y_stride_b, y_stride_t;
  int64_t h_stride_b, h_stride_t;    /* of h and dh */
  int64_t n_stride_b, n_stride_t;    /* of n and dn */
  int64_t dx_stride_b, dx_stride_t;
  int64_t dy_stride_b, dy_stride_t;
  int64_t gate_stride_b;
  int32_t dtype;
  int32_t options;                   /* 0 or GDN_LAYER_OPT_ZERO_UNUSED (h, n, dx and dy) */
  float residual_scale, eps;
  const int32_t* seq_offsets;
  const float* gate;
  const float* post_weight;
  const float* weight;
  void* workspace;                   /* gdn_norm_backward: caller-owned device memory, 256-byte aligned */
  size_t workspace_bytes;
  void* stream;
} gdn_norm_problem_t;

gdn_status_t gdn_norm_forward(const gdn_norm_problem_t* p, const void* x, const void* y, void* h, void* n);

/* Workspace bytes of gdn_norm_backward (0 if invalid or unsupported, or where
 * no gradient is summed over rows): it depends on the sizes, on whether
 * seq_offsets, gate, post_weight and weight are given, and on gate_stride_b. */
size_t gdn_norm_workspace_bytes(const gdn_norm_problem_t* p);

gdn_status_t gdn_norm_backward(const gdn_norm_problem_t* p, const void* x, const void* y, const void* dh, const void* dn,
                               void* dx, void* dy, float* dgate, float* dpost_weight, float* dweight);

/* Static description of a status code. */
const char* gdn_status_string(int32_t status);

/* Library version string. */
const char* gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
