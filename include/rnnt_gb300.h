/*
 * rnnt_gb300.h -- C ABI of the fused RNN-T (transducer) loss for GB300 (sm_103a).
 *
 * One call computes, for a batch of B utterances, the per-sample RNN-T loss
 * (negative log-likelihood summed over every alignment) and, optionally, its
 * gradient with respect to the joiner logits, with the semantics of
 * torchaudio.functional.rnnt_loss.  The operation and its arguments are the
 * ones of the rnnt-loss-ascend README ("optimized_transducer"):
 *   - section 参数说明 (parameter table): compact 2D logits, int32 targets and
 *     lengths, blank, clamp, fused_log_softmax, per-sample loss, grad with
 *     the shape of the logits;
 *   - section 约束说明 (constraints): float32/float16 logits (bfloat16 added
 *     here), blank in
 *     [-V, V-1] with -1 meaning V-1, sum of T_b*(U_b+1) equal to the number
 *     of logit rows, clamp <= 0 meaning no clipping;
 *   - section 架构设计 (architecture): a two-phase interface, workspace size
 *     first, then the fused launch;
 *   - section 核心梯度融合公式 / 精度保证: the gradient formula and the check that
 *     the alpha-side and beta-side losses agree.
 * Status codes follow the RNNTStatus convention of the ESPnet GPURNNT docs
 * (cost_and_grad returns success or RNNT_STATUS_INVALID_VALUE).
 *
 * Memory and streams: every pointer argument named "device" must point to
 * memory the current CUDA device can access.  The library allocates nothing
 * and keeps no state between calls other than per-device kernel attributes
 * (and, for rnnt_loss_fused_noalloc, its fixed scratch array); all work is
 * enqueued on `stream` and the host never synchronises.
 */
#ifndef RNNT_GB300_H
#define RNNT_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *rnnt_stream_t;

typedef enum {
    RNNT_OK = 0,
    RNNT_INVALID_VALUE = 1,       /* bad argument (host) or bad lengths/targets (device) */
    RNNT_WORKSPACE_TOO_SMALL = 2, /* workspace_bytes below rnnt_workspace_size()         */
    RNNT_LAUNCH_FAILED = 3,       /* a kernel launch returned a CUDA error               */
    RNNT_LOSS_MISMATCH = 4,       /* alpha-side and beta-side losses disagree (or NaN)   */
    RNNT_TIMEOUT = 5              /* a bounded device wait gave up                       */
} rnnt_status_t;

/* Storage type of the logits and the gradient (arithmetic is float32 for
 * every type; bfloat16 is this library's addition to the README's
 * float32/float16). */
typedef enum { RNNT_F32 = 0, RNNT_F16 = 1, RNNT_BF16 = 2 } rnnt_dtype_t;

typedef enum { RNNT_RED_NONE = 0, RNNT_RED_SUM = 1, RNNT_RED_MEAN = 2 } rnnt_reduction_t;

/* Largest supported target length (U_b <= RNNT_MAX_TARGET_LENGTH, so a lattice
 * is at most 1024 nodes wide). */
#define RNNT_MAX_TARGET_LENGTH 1023

/*
 * rnnt_workspace_size -- bytes of device scratch rnnt_loss_fused needs.
 * README 架构设计, first phase of the two-phase interface.
 *   B     number of samples (>= 1)
 *   rows  number of logit rows, sum over b of T_b*(U_b+1) (>= 1)
 *   V     vocabulary size including blank (>= 1)
 *   dt    logit element type
 *   bytes out: required size; about 36 bytes per logit row plus O(B).
 * Returns RNNT_INVALID_VALUE for a NULL `bytes` or out-of-range sizes.
 */
rnnt_status_t rnnt_workspace_size(int32_t B, int64_t rows, int32_t V, rnnt_dtype_t dt,
                                  size_t *bytes);

/*
 * rnnt_loss_fused -- loss and gradient of a batch in one call (README 架构设计,
 * second phase; 参数说明 for the arguments).
 *
 *   logits            device, (rows, V) row-major contiguous, dt.  Sample b owns
 *                     rows [off_b, off_b + T_b*(U_b+1)), off_b = sum_{i<b}
 *                     T_i*(U_i+1); inside a sample, row t*(U_b+1)+u holds the
 *                     joiner output for frame t after u emitted labels.
 *                     Must be 16-byte aligned.  Raw logits when
 *                     fused_log_softmax != 0, log-probabilities otherwise.
 *   targets           device int32, (B, targets_stride) row-major; row b holds
 *                     the U_b labels of sample b followed by ignored padding.
 *                     Labels must lie in [0, V) and differ from blank.
 *   targets_stride    1 <= targets_stride <= RNNT_MAX_TARGET_LENGTH, and
 *                     >= max_b U_b.
 *   logit_lengths     device int32 [B], T_b >= 1.
 *   target_lengths    device int32 [B], 0 <= U_b <= targets_stride.
 *   B                 batch size >= 1.
 *   blank             in [-V, V-1]; a negative value counts from the end.
 *   clamp             > 0 clips every gradient element to [-clamp, clamp]
 *                     before the reduction scale; <= 0 disables clipping.
 *   fused_log_softmax nonzero: the kernel applies log-softmax to each row.
 *   reduction         NONE / SUM / MEAN (mean over the batch).  It sets the
 *                     gradient scale (1/B for MEAN, else 1) and loss_reduced.
 *   loss              device float [B], required: per-sample loss.
 *   loss_reduced      device float [1] or NULL: sum (SUM, NONE) or mean (MEAN).
 *   grad              device (rows, V) in dt, or NULL for loss only.  It may
 *                     equal `logits` (the gradient then overwrites the
 *                     logits in place) but must not partly overlap it.  Must
 *                     be 16-byte aligned.
 *   workspace         device scratch of at least rnnt_workspace_size() bytes,
 *                     256-byte aligned, owned by the caller; it may be reused
 *                     by later calls on the same stream once this one is
 *                     enqueued (contents are rewritten every call).
 *   status_dev        device int32 [1] or NULL.  Receives RNNT_OK,
 *                     RNNT_INVALID_VALUE (device-detected: a T_b < 1, a U_b
 *                     out of range, a label out of range or equal to blank,
 *                     or rows != sum T_b*(U_b+1)) or RNNT_LOSS_MISMATCH
 *                     (alpha/beta losses differ by more than
 *                     1e-3*max(1,|loss|), or a loss is not finite).  When it
 *                     is not RNNT_OK, loss/grad contents are unspecified.
 *   stream            CUDA stream all kernels are enqueued on.
 *
 * Host-side return value: RNNT_INVALID_VALUE for NULL required pointers, bad
 * sizes/enums/blank, misaligned or partly overlapping buffers;
 * RNNT_WORKSPACE_TOO_SMALL; RNNT_LAUNCH_FAILED if a launch fails.  Nothing is
 * enqueued when a host-side check fails.
 */
rnnt_status_t rnnt_loss_fused(const void *logits, rnnt_dtype_t dt, int64_t rows, int32_t V,
                              const int32_t *targets, int32_t targets_stride,
                              const int32_t *logit_lengths, const int32_t *target_lengths,
                              int32_t B, int32_t blank, float clamp, int32_t fused_log_softmax,
                              rnnt_reduction_t reduction, float *loss, float *loss_reduced,
                              void *grad, void *workspace, size_t workspace_bytes,
                              int32_t *status_dev, rnnt_stream_t stream);

/*
 * Options of rnnt_loss_fused_ex.  A zero-initialised struct (or a NULL
 * pointer) gives the behaviour of rnnt_loss_fused.
 *
 *   fastemit_lambda   >= 0.  FastEmit weight (the fastemit_lambda argument of
 *                     the ESPnet GPURNNT docs and of compute_multiblank_grad_kernel,
 *                     after the FastEmit paper they cite): the gradient term of
 *                     every label-emission log-probability is multiplied by
 *                     1 + fastemit_lambda; blank terms and the loss are not
 *                     changed.  0 is the plain transducer gradient.
 *   padded            0: compact layout (rows = sum_b T_b*(U_b+1)).
 *                     1: padded layout of the GPURNNT docs (the activation
 *                     tensor of cost_and_grad, shape [B, T, U, V+1]; also the
 *                     torchaudio.functional.rnnt_loss layout): logits and grad are
 *                     (B, max_T, max_U + 1, V) row-major, rows must equal
 *                     B*max_T*(max_U+1), node (t, u) of sample b is row
 *                     (b*max_T + t)*(max_U+1) + u.  Rows outside a sample's
 *                     lattice (t >= T_b or u > U_b) are never read and get a
 *                     zero gradient.  T_b <= max_T and U_b <= max_U are
 *                     checked on the device (RNNT_INVALID_VALUE).
 *   max_T, max_U      padded layout only: max_T >= 1, 0 <= max_U <=
 *                     RNNT_MAX_TARGET_LENGTH, max_T*(max_U+1) < 2^31.
 *   num_big_blanks    0..RNNT_MAX_BIG_BLANKS.  Multi-blank transducer (ESPnet
 *                     compute_multiblank_grad_kernel docs and the multi-blank
 *                     paper they cite): besides `blank` (one frame), big blank
 *                     i is output big_blank_ids[i] (in [-V, V-1], negative
 *                     counting from the end; distinct, not blank, never a
 *                     label) and advances big_blank_durations[i] frames
 *                     (2..RNNT_MAX_BIG_BLANK_DURATION).  A path ends when a
 *                     blank-type step reaches frame T with every label
 *                     emitted; no step passes frame T.
 *   sigma             >= 0.  Logit under-normalisation of the same docs:
 *                     subtracted from every log-probability the lattice uses.
 *                     With num_big_blanks == 0 and sigma == 0 the call is the
 *                     standard transducer loss; otherwise it runs the
 *                     multi-blank kernels (workspace: rnnt_workspace_size_ex).
 */
#define RNNT_MAX_BIG_BLANKS 8
#define RNNT_MAX_BIG_BLANK_DURATION 16
typedef struct {
    float fastemit_lambda;
    int32_t padded;
    int32_t max_T;
    int32_t max_U;
    int32_t num_big_blanks;
    int32_t big_blank_ids[RNNT_MAX_BIG_BLANKS];
    int32_t big_blank_durations[RNNT_MAX_BIG_BLANKS];
    float sigma;
} rnnt_options_t;

/*
 * rnnt_workspace_size_ex -- workspace bytes of rnnt_loss_fused_ex with these
 * options (NULL: as rnnt_workspace_size).  The multi-blank kernels need 8
 * more bytes per big blank and lattice node.  RNNT_INVALID_VALUE as
 * rnnt_workspace_size, or for num_big_blanks outside 0..RNNT_MAX_BIG_BLANKS.
 */
rnnt_status_t rnnt_workspace_size_ex(int32_t B, int64_t rows, int32_t V, rnnt_dtype_t dt,
                                     const rnnt_options_t *options, size_t *bytes);

/*
 * rnnt_loss_fused_ex -- rnnt_loss_fused with options (FastEmit, padded
 * layout).  Same arguments, results and errors as rnnt_loss_fused, plus
 * `options` (NULL = defaults); RNNT_INVALID_VALUE for a negative or
 * non-finite fastemit_lambda or sigma, inconsistent padded sizes or invalid
 * big blanks.  The workspace is sized by rnnt_workspace_size_ex(B, rows, V,
 * dt, options) with the same `rows`.
 */
rnnt_status_t rnnt_loss_fused_ex(const void *logits, rnnt_dtype_t dt, int64_t rows, int32_t V,
                                 const int32_t *targets, int32_t targets_stride,
                                 const int32_t *logit_lengths, const int32_t *target_lengths,
                                 int32_t B, int32_t blank, float clamp, int32_t fused_log_softmax,
                                 rnnt_reduction_t reduction, float *loss, float *loss_reduced,
                                 void *grad, void *workspace, size_t workspace_bytes,
                                 int32_t *status_dev, rnnt_stream_t stream,
                                 const rnnt_options_t *options);

/*
 * rnnt_loss_fused_staged -- rnnt_loss_fused with stage timing (tracing aid).
 * Same arguments, plus stage_events: NULL, or an array of 7 cudaEvent_t
 * handles (entries may be NULL) that the call records on `stream` at its
 * stage boundaries: [0] start, [1] after offsets/schedule, [2] after the
 * row pass, [3] after the alpha/beta DP, [4] = [3] (the per-row gradient
 * coefficients are formed inside the gradient pass), [5] after the gradient
 * pass (whose last CTA also runs the loss check/reduction), [6] at the end.
 * A call that runs as one persistent kernel records [1]..[6] after it.
 * The caller creates and owns the events.
 */
rnnt_status_t rnnt_loss_fused_staged(const void *logits, rnnt_dtype_t dt, int64_t rows, int32_t V,
                                     const int32_t *targets, int32_t targets_stride,
                                     const int32_t *logit_lengths, const int32_t *target_lengths,
                                     int32_t B, int32_t blank, float clamp,
                                     int32_t fused_log_softmax, rnnt_reduction_t reduction,
                                     float *loss, float *loss_reduced, void *grad, void *workspace,
                                     size_t workspace_bytes, int32_t *status_dev,
                                     rnnt_stream_t stream, void *const *stage_events);

/*
 * rnnt_grad_scale -- multiply a gradient produced by rnnt_loss_fused by the
 * upstream gradient of the loss (the autograd backward step the README's
 * Python layer performs, section 架构设计 "Python 层").
 *   grad, dt, rows, V   the gradient buffer of a previous rnnt_loss_fused call
 *   B                   batch size of that call
 *   workspace           the workspace of that call, unmodified since (its
 *                       row offsets map rows to samples)
 *   factors             device float: factors[0] for the whole gradient
 *                       (per_sample == 0) or factors[b] for sample b's rows
 *                       (per_sample != 0).  Rows whose factor is exactly 1
 *                       are left untouched (no memory traffic).
 * The layout (compact or padded) is the one of that call; `rows` is the
 * gradient's row count passed to it.
 * Returns RNNT_INVALID_VALUE / RNNT_WORKSPACE_TOO_SMALL / RNNT_LAUNCH_FAILED
 * as rnnt_loss_fused does.
 */
rnnt_status_t rnnt_grad_scale(void *grad, rnnt_dtype_t dt, int64_t rows, int32_t V, int32_t B,
                              const void *workspace, size_t workspace_bytes,
                              const float *factors, int32_t per_sample, rnnt_stream_t stream);

/*
 * rnnt_plan -- how rnnt_loss_fused / rnnt_loss_fused_ex would run a call of
 * this shape on the current device, without running it (a planning and
 * measurement aid; no counterpart on the pages, whose README promises one
 * kernel launch per call, 价值说明 "Kernel 启动次数").
 *   B, rows, V, dt, targets_stride, fused_log_softmax   as for the call
 *   want_grad   nonzero when the call will pass a gradient buffer
 *   options     as for rnnt_loss_fused_ex, or NULL
 *   plan        out: persistent = 1 when one cooperative kernel runs the
 *               whole call (preparation, rows, recursions, gradient, check),
 *               0 for one kernel per stage; launches = kernels the call
 *               enqueues.
 * The call itself takes the per-stage kernels instead if the device
 * refuses the cooperative launch at that time.  Returns RNNT_INVALID_VALUE
 * for bad sizes, RNNT_LAUNCH_FAILED when no device is current.
 */
typedef struct {
    int32_t persistent;
    int32_t launches;
} rnnt_plan_t;

rnnt_status_t rnnt_plan(int32_t B, int64_t rows, int32_t V, rnnt_dtype_t dt,
                        int32_t targets_stride, int32_t fused_log_softmax, int32_t want_grad,
                        const rnnt_options_t *options, rnnt_plan_t *plan);

/*
 * rnnt_set_trace -- task tracing (a debugging aid; process-wide setting, not
 * thread-safe).  While a buffer is set, every rnnt_loss_fused call writes
 * records int4 {kind | sample << 2, SM id, start ns, end ns} (kind 0: row
 * chunk, 1: alpha/beta recursions of a sample, 2: gradient chunk; times
 * relative to the start of the call's preparation) at indices below
 * bytes/16.  A call that runs as one persistent kernel records every task:
 * for each sample (longest DP first) its row chunks, then every gradient
 * chunk (record = task index), and sample b's recursions at index
 * (task count + b).  A call on the per-stage kernels records the recursions
 * only: the forward and backward recursion of the i-th sample in DP order at
 * indices 2i and 2i + 1.  device_buffer must be 16-byte aligned
 * device memory that outlives the calls; NULL (or bytes < 16) turns tracing
 * off.
 */
rnnt_status_t rnnt_set_trace(void *device_buffer, size_t bytes);

/* Size of the fixed device scratch array rnnt_loss_fused_noalloc uses: 32 MiB,
 * enough for rnnt_workspace_size() up to about 900,000 logit rows. */
#define RNNT_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * rnnt_loss_fused_noalloc -- rnnt_loss_fused for callers that cannot hand
 * out device memory.  The paper has no counterpart: this is an interface of
 * this library only.
 *
 * Same arguments and results as rnnt_loss_fused without workspace and
 * workspace_bytes.  The scratch is a file-scope device array of
 * RNNT_NOALLOC_SCRATCH_BYTES bytes inside this library, one per device; the
 * call allocates nothing (no cudaMalloc/cudaFree, no allocating library
 * routine).  The first call on a device, made with that device current,
 * looks up the array's device address (cudaGetSymbolAddress) once and
 * caches it; make that first call before any stream capture.  The cached
 * address is that of the device's primary context at the time: a process
 * that destroys it (cudaDeviceReset) must not call this entry point on that
 * device afterwards.
 *
 * Every call on a device shares the one array and leaves its contents
 * behind; each call rewrites everything it reads before reading it.  Calls
 * whose kernels overlap on the GPU (other streams, other host threads)
 * race on the array and give undefined results: serialize them, e.g. on
 * one stream.  rnnt_grad_scale, which reads a caller workspace, does not
 * apply to this call's gradient.
 *
 * Returns RNNT_WORKSPACE_TOO_SMALL, before any device work, when
 * rnnt_workspace_size(B, rows, V, dt) exceeds RNNT_NOALLOC_SCRATCH_BYTES;
 * RNNT_LAUNCH_FAILED when the address lookup fails; otherwise what
 * rnnt_loss_fused returns.
 */
rnnt_status_t rnnt_loss_fused_noalloc(const void *logits, rnnt_dtype_t dt, int64_t rows,
                                      int32_t V, const int32_t *targets, int32_t targets_stride,
                                      const int32_t *logit_lengths,
                                      const int32_t *target_lengths, int32_t B, int32_t blank,
                                      float clamp, int32_t fused_log_softmax,
                                      rnnt_reduction_t reduction, float *loss,
                                      float *loss_reduced, void *grad, int32_t *status_dev,
                                      rnnt_stream_t stream);

/*
 * rnnt_selftest_wait_timeout -- diagnostic of the bounded device waits (no
 * counterpart on the pages).  Enqueues one kernel whose warp waits, with the
 * same helper the loss kernels use for their shared-memory row copies, on a
 * barrier that nothing completes; after `polls` (>= 1) polls the wait gives
 * up, and status_dev (device int32) receives RNNT_TIMEOUT, as a loss call's
 * status would.  Nothing faults, traps or stays in flight; the context stays
 * usable.  Returns RNNT_INVALID_VALUE (NULL status_dev, polls < 1) or
 * RNNT_LAUNCH_FAILED.
 */
rnnt_status_t rnnt_selftest_wait_timeout(int32_t *status_dev, int32_t polls, rnnt_stream_t stream);

/* ------------------------------------------------------------------------
 * The label side of a transducer: the embedding that feeds the prediction
 * network the labels the loss takes, and the beam search over the joiner's
 * outputs.  No counterpart on the pages, which stop at the loss.
 *
 * All of these enqueue on `stream`, allocate nothing and never synchronise.
 * status_dev (device int32, or NULL) receives RNNT_OK, or RNNT_INVALID_VALUE
 * for what only the device can see.  Host-side errors are returned before
 * anything is enqueued.  Unless said otherwise pointers are device pointers
 * aligned to their element size; wider alignment (16 bytes, row strides too)
 * gives wider accesses.
 */

/*
 * rnnt_embed -- label embedding with scaling.
 *
 * Each of the B sequences has P = S + (has_start ? 1 : 0) places.  With
 * has_start, place 0 holds `start` (blank, as a rule: the prediction network's
 * first input); place p after it holds tokens[b][p - has_start].
 *
 *   out[b, p, :] = round(scale * weight[token, :]), in float32 and rounded
 *   once; zeros where the token is negative or stands at or past lengths[b].
 *
 *   weight         (V, D) in dt, rows weight_stride >= D elements apart.
 *   tokens         int32 (B, S), rows tokens_stride >= S apart; NULL if S = 0.
 *                  Any negative token is padding (rnnt_beam_select writes -1
 *                  for hypotheses that emit nothing).  Tokens at or past
 *                  lengths[b] are not read.
 *   lengths        int32 [B], or NULL: every token counts.
 *   start          in [-V, V-1], a negative value counting from the end;
 *                  ignored without has_start.
 *   out            (B, P, D) contiguous in dt; must not overlap weight.
 *   status_dev     RNNT_INVALID_VALUE for a token >= V (its place gets
 *                  zeros) or a length outside [0, S] (taken as the nearer bound).
 * 1 <= D <= 2^20, 1 <= B * P < 2^31.
 */
rnnt_status_t rnnt_embed(const void *weight, rnnt_dtype_t dt, int32_t V, int32_t D,
                         int64_t weight_stride, const int32_t *tokens, int64_t tokens_stride,
                         const int32_t *lengths, int32_t B, int32_t S, int32_t has_start,
                         int32_t start, float scale, void *out, int32_t *status_dev,
                         rnnt_stream_t stream);

/* rnnt_embed_grad_workspace_size -- bytes of device scratch of rnnt_embed_grad:
 * 0 up to 4096 places, else about 16 + D/4 bytes per place. */
rnnt_status_t rnnt_embed_grad_workspace_size(int32_t B, int32_t S, int32_t has_start, int32_t V,
                                             int32_t D, size_t *bytes);

/*
 * rnnt_embed_grad -- gradient of rnnt_embed with respect to weight:
 *
 *   grad_weight[v, :] = round(scale * sum over places with token v of grad_out[b, p, :])
 *
 * and zeros for ids that do not occur.  The places are sorted by id; sums are
 * float32 in an order that depends on the tokens alone, so the same inputs
 * give the same bits.  grad_out at padding is not read.
 *
 *   grad_out       (B, P, D) contiguous in dt.
 *   grad_weight    (V, D) contiguous in dt, every row written; must not
 *                  overlap grad_out.
 *   workspace      rnnt_embed_grad_workspace_size() bytes, 256-byte aligned (NULL
 *                  if that is 0); contents are rewritten every call.
 * tokens, lengths, start and status_dev as for rnnt_embed.
 */
rnnt_status_t rnnt_embed_grad(const void *grad_out, rnnt_dtype_t dt, const int32_t *tokens,
                              int64_t tokens_stride, const int32_t *lengths, int32_t B, int32_t S,
                              int32_t has_start, int32_t start, int32_t V, int32_t D, float scale,
                              void *grad_weight, void *workspace, size_t workspace_bytes,
                              int32_t *status_dev, rnnt_stream_t stream);

/* Most hypotheses of a batch item, and the largest vocabulary, of the beam search. */
#define RNNT_MAX_BEAM 64
#define RNNT_MAX_BEAM_VOCAB (1 << 20)

/* rnnt_beam_workspace_size -- bytes of device scratch of rnnt_beam_select on the
 * current device; with rows of up to 32 KB, 0 for up to 8 hypotheses, and for
 * up to 16 where the device runs clusters of 16 thread blocks (a GB300 does). */
rnnt_status_t rnnt_beam_workspace_size(int32_t B, int32_t K, int32_t V, int32_t Ko,
                                       rnnt_dtype_t dt, size_t *bytes);

/*
 * rnnt_beam_select -- one step of beam search: of every batch item the Ko best
 * extensions of its K hypotheses.
 *
 * Hypothesis k with score s offers, for each output v whose logit is above
 * -inf, the candidate s + x_v - logsumexp(x) (s + x_v without
 * fused_log_softmax).  A finished hypothesis offers itself alone: its score
 * unchanged and token -1, whatever its logits hold.  One of score -inf offers
 * nothing.  Candidates are ordered by value (to 40 bits), equal ones by
 * hypothesis, then by token.
 *
 *   logits         (B, K, V) in dt: item b's hypothesis k starts at element
 *                  b * batch_stride + k * beam_stride, its V logits adjacent.
 *   scores         float [B, K].
 *   finished       uint8 [B, K] (0 or not), or NULL: none.
 *   out_scores     float [B, Ko], best first; within 5e-6 of the value and one
 *                  float32 rounding (without fused_log_softmax: the rounding).
 *                  A candidate beyond float32's range keeps its place in the
 *                  order, its token and its parent, and its score is -inf
 *                  (+inf above the range).
 *   out_tokens     int32 [B, Ko]: the selected output, -1 for a finished one.
 *   out_parents    int32 [B, Ko]: the hypothesis it extends.
 *                  Places left over when fewer than Ko candidates exist get
 *                  score -inf, token -1, parent -1.  The outputs must not
 *                  overlap the inputs.
 *   workspace      rnnt_beam_workspace_size() bytes, 256-byte aligned (NULL if that is
 *                  0).
 *   status_dev     RNNT_INVALID_VALUE for a score of +inf or NaN, or a
 *                  hypothesis whose logits hold one; such a hypothesis offers
 *                  nothing.  RNNT_LAUNCH_FAILED for a selection that lost its
 *                  order on the device (none is known to): all its places
 *                  are left over.
 */
rnnt_status_t rnnt_beam_select(const void *logits, rnnt_dtype_t dt, int32_t B, int32_t K, int32_t V,
                               int64_t batch_stride, int64_t beam_stride, const float *scores,
                               const uint8_t *finished, int32_t Ko, int32_t fused_log_softmax,
                               float *out_scores, int32_t *out_tokens, int32_t *out_parents,
                               void *workspace, size_t workspace_bytes, int32_t *status_dev,
                               rnnt_stream_t stream);

/* Most states of one rnnt_beam_reorder call. */
#define RNNT_MAX_STATES 16

/* A state of the hypotheses: rows of row_bytes adjacent bytes, one for every
 * (batch item, hypothesis) and every index of up to three further axes (sizes
 * n, 1 where unused).  Strides are in bytes and not negative. */
typedef struct {
    const void *src;
    void *dst;
    int64_t row_bytes;
    int32_t n[3];
    int64_t src_stride[3];
    int64_t dst_stride[3];
    int64_t src_batch;
    int64_t src_beam;
    int64_t dst_batch;
    int64_t dst_beam;
} rnnt_state_t;

/*
 * rnnt_beam_reorder -- the states of the selected hypotheses: for every state,
 * batch item b and k < Ko, row(s) dst[b, k] = src[b, parents[b, k]]; zeros
 * where the parent is -1.
 *
 *   states         HOST array of n_states (1 to RNNT_MAX_STATES); read during
 *                  the call only.  No dst may overlap or interleave with a
 *                  src (keep two buffers per state).
 *   parents        int32 [B, Ko], each in [-1, K): out_parents of
 *                  rnnt_beam_select.  Another value counts as -1 and sets
 *                  status_dev to RNNT_INVALID_VALUE.
 */
rnnt_status_t rnnt_beam_reorder(const rnnt_state_t *states, int32_t n_states,
                                const int32_t *parents, int32_t B, int32_t K, int32_t Ko,
                                int32_t *status_dev, rnnt_stream_t stream);

/* ------------------------------------------------------------------------
 * Learning from a teacher: the top logits of a teacher's lattice rows, the loss
 * of a student against them, and the drawing of labels.  No counterpart on the
 * pages.  What is said of the label side above holds here as well.
 */

/* Most outputs kept of a teacher's row, and the largest vocabulary, of these operators. */
#define RNNT_MAX_TOP 64
#define RNNT_MAX_TOP_VOCAB (1 << 20)

/*
 * rnnt_top_logits -- of every row of V logits x the k largest with their ids, and
 * what remains.
 *
 *   values[r], ids[r]   the k largest logits above -inf in descending order, equal
 *                       ones by id; places left over get -inf and id -1.
 *   rest[r]             log sum exp(x_j / temperature) over the outputs without a
 *                       place; -inf where there is none.  A finite value outside
 *                       float32's range is the nearer end of it.
 *
 *   logits         (rows, V) contiguous in dt.
 *   logit_lengths, target_lengths
 *                  int32 [B], or both NULL: every row counts.  With lengths the
 *                  rows are those of the padded (B, max_T, max_U + 1, V) layout;
 *                  what a row outside its sequence holds is not used, and all its
 *                  places are left over.  B, max_T and max_U are ignored without.
 *   values         (rows, k) in dt;  ids int32 (rows, k);  rest float (rows).
 *                  They must not overlap logits or one another.
 *   status_dev     RNNT_INVALID_VALUE for a row that holds NaN or +inf (all its
 *                  places are left over), or lengths outside the layout (taken
 *                  as the nearer bound).
 * 1 <= k <= min(V, RNNT_MAX_TOP), V <= RNNT_MAX_TOP_VOCAB, 1e-4 <= temperature <= 1e4.
 */
rnnt_status_t rnnt_top_logits(const void *logits, rnnt_dtype_t dt, int64_t rows, int32_t V,
                              const int32_t *logit_lengths, const int32_t *target_lengths,
                              int32_t B, int32_t max_T, int32_t max_U, int32_t k,
                              double temperature, void *values, int32_t *ids, float *rest,
                              int32_t *status_dev, rnnt_stream_t stream);

/* rnnt_distill_workspace_size -- bytes of device scratch of rnnt_distill_loss: 4 per row,
 * 8 per sample, and 8 per part of a sample's sum (64 of them at most). */
rnnt_status_t rnnt_distill_workspace_size(int32_t B, int64_t rows, size_t *bytes);

/*
 * rnnt_distill_loss -- the divergence of a student's lattice rows from a teacher's,
 * summed over the rows of each sample, and its gradient.
 *
 * A row's teacher has up to k places, each a logit and the id of its output, and
 * optionally a rest, the log-sum-exp of its remaining logits over the temperature
 * tau.  p is the softmax over the places' logits / tau and the rest; q is the
 * softmax of the student's logits x / tau, q_r its sum over the outputs without
 * a place.
 *
 *   row      tau^2 * [ sum_k p_k log(p_k / q_id(k)) + p_r log(p_r / q_r) ], terms of
 *            p = 0 being 0
 *   loss[b]  weight * the sum over sample b's T_b * (U_b + 1) rows
 *   grad     d loss_reduced / d x (of the sum for RNNT_RED_NONE): per row weight * tau
 *            (/ B for the mean) times q_j - p_j for an output with a place, q_j (1 - p_r / q_r)
 *            for another, q_j without a rest
 *
 * A row whose teacher holds nothing (no place above -inf, no rest above -inf) has loss 0
 * and gradient 0, whatever its logits are.
 *
 *   logits         (rows, V) contiguous in dt, 16-byte aligned: the compact layout of
 *                  rnnt_loss_fused, or the padded one, (B, max_T, max_U + 1, V).  What
 *                  other rows hold is not used, and their gradient is 0.
 *   teacher_logits (rows, k) in teacher_dt;  teacher_ids int32 (rows, k), a negative id
 *                  being an empty place;  teacher_rest float (rows), or NULL: p is the
 *                  softmax over the places alone.
 *   logit_lengths, target_lengths   int32 [B], T_b >= 0, U_b >= 0.
 *   loss           float [B];  loss_reduced float [1] or NULL: sum (SUM, NONE) or mean (MEAN).
 *   grad           (rows, V) contiguous in dt, 16-byte aligned, or NULL: loss only.
 *   workspace      rnnt_distill_workspace_size() bytes, 256-byte aligned.
 *                  No output may overlap an input.
 *   status_dev     RNNT_INVALID_VALUE for lengths out of range (taken as the nearer bound) or,
 *                  in the compact layout, not adding up to rows (rows behind the last sample
 *                  get gradient 0); an id >= V (its place counts as empty), an id twice in
 *                  a row (the later places count as empty), a teacher's logit or rest that
 *                  is NaN or +inf; logits that are NaN or +inf, or all -inf, in a row with a
 *                  teacher (its loss and gradient are then NaN).
 * 1 <= k <= RNNT_MAX_TOP, V <= RNNT_MAX_TOP_VOCAB, 1e-4 <= temperature <= 1e4, |weight| < 1e30.
 */
rnnt_status_t rnnt_distill_loss(const void *logits, rnnt_dtype_t dt, int64_t rows, int32_t V,
                                const void *teacher_logits, rnnt_dtype_t teacher_dt,
                                const int32_t *teacher_ids, const float *teacher_rest, int32_t k,
                                const int32_t *logit_lengths, const int32_t *target_lengths,
                                int32_t B, int32_t padded, int32_t max_T, int32_t max_U,
                                double temperature, double weight, rnnt_reduction_t reduction,
                                float *loss, float *loss_reduced, void *grad, void *workspace,
                                size_t workspace_bytes, int32_t *status_dev,
                                rnnt_stream_t stream);

/*
 * rnnt_distill_grad_scale -- multiplies a gradient of rnnt_distill_loss in place by upstream
 * factors: factors[0], or with per_sample != 0 factors[b] for sample b's rows.  A
 * factor of 1 leaves its rows as they are.  The gradient has been rounded to its type
 * before: a factor that is known ahead (a gradient scaler's) belongs into the weight.
 *
 *   rows_each      rows of a sample of the padded layout, max_T * (max_U + 1); 0 for the
 *                  compact one.
 *   workspace      the one that the rnnt_distill_loss call used, unchanged since.
 */
rnnt_status_t rnnt_distill_grad_scale(void *grad, rnnt_dtype_t dt, int64_t rows, int32_t V,
                                      int32_t B, int64_t rows_each, const void *workspace,
                                      size_t workspace_bytes, const float *factors,
                                      int32_t per_sample, rnnt_stream_t stream);

/*
 * rnnt_sample -- one step of drawing: of every hypothesis one extension.
 *
 * A hypothesis with logits x and a number u in [0, 1) draws as follows.  Outputs are ordered by
 * logit (equal ones by id); with e_j = exp(x_j / temperature) those are kept that are among the
 * first top_k, of these the shortest beginning whose sum of e is at least top_p of theirs, and of
 * these the ones with e_j >= min_p * max e.  The token is the first kept id
 * at which the running sum of e over the kept ids, in the order of the ids, is above u times
 * their whole sum.  Outputs of logit -inf are never kept.  The sums decide as if held to 40 bits.
 *
 *   out_scores     scores + x_token - logsumexp(x) (scores + x_token without
 *                  fused_log_softmax), at temperature 1 and over all outputs; within 5e-6 of
 *                  the value and one float32 rounding.
 *   out_tokens     the token.  A finished hypothesis keeps its score and gets token -1, whatever
 *                  its logits hold; one of score -inf, or whose logits are all -inf, gets score
 *                  -inf and token -1.
 *
 *   logits         (B, K, V) in dt: item b's hypothesis k starts at element
 *                  b * batch_stride + k * beam_stride, its V logits adjacent.
 *   scores, random float [B, K];  finished uint8 [B, K], or NULL: none.
 *   top_k          >= 1, or 0: not used;  top_p in (0, 1], 1: not used;  min_p in [0, 1], 0: not
 *                  used;  temperature in [1e-4, 1e4].
 *   status_dev     RNNT_INVALID_VALUE for a score of NaN or +inf, a random number outside [0, 1),
 *                  or logits that hold NaN or +inf; such a hypothesis gets score -inf and token -1.
 * The outputs must not overlap the inputs or one another.  V <= RNNT_MAX_TOP_VOCAB.
 */
rnnt_status_t rnnt_sample(const void *logits, rnnt_dtype_t dt, int32_t B, int32_t K, int32_t V,
                          int64_t batch_stride, int64_t beam_stride, const float *scores,
                          const float *random, const uint8_t *finished, double temperature,
                          int32_t top_k, double top_p, double min_p, int32_t fused_log_softmax,
                          float *out_scores, int32_t *out_tokens, int32_t *status_dev,
                          rnnt_stream_t stream);

/* Static English description of a status code. */
const char *rnnt_status_string(rnnt_status_t status);

/* ABI version of this header (major * 100 + minor). */
int32_t rnnt_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RNNT_GB300_H */
