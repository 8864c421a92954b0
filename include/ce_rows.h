/*
 * ce_rows.h -- C ABI of the row-wise softmax cross-entropy library for
 * NVIDIA GB300 (sm_103a): per-row loss, mean loss, fused loss + gradient,
 * and the row argmax that closes a decode step; beside them, the rows a
 * language model's step reads from the same logits (softmax, log-softmax,
 * sampling candidates) and the join of split partial sums; and the objectives
 * over sampled answers and pairs of answers (token log-probabilities, the
 * clipped policy loss, the preference loss), each with its gradient; and the
 * choices made from a row's softmax (sampled tokens, the verification of
 * drafted ones, the routing of rows to experts, with its gradient).
 *
 * Definitions follow the API reference page "gizml:netops"
 * (gizstack.com/docs/reference/gizml/netops.md), section Functions:
 * crossEntropyRows, crossEntropyLoss, crossEntropyGrad, argmaxInto,
 * candidatesInto, splitSumInto; section Methods: Tensor.argmax; section
 * Constants: TOP_EACH, CANDIDATE_ROW.
 *
 * Common conventions of every entry point:
 *  - Logits are f32, row-major: row i starts at logits + i * stride
 *    (elements); only its first `vocab` columns are read, the padding
 *    columns vocab..stride-1 never are.
 *  - Labels are int64, one per row. Outputs are written per row; the
 *    gradient is written dense, [rows, vocab] (row i at grad + i * vocab).
 *  - All pointers are DEVICE pointers on the current CUDA device, owned by
 *    the caller; the library keeps none of them after the call returns and
 *    allocates no memory per call.
 *  - Every call only enqueues work on `stream` (NULL: the legacy default
 *    stream) and returns; nothing waits for the GPU. A result is ready once
 *    the stream has reached it.
 *  - Arguments are checked on the host before anything is launched; a
 *    rejected call returns a negative status and launches nothing:
 *      CE_EINVAL: a required pointer is NULL (while rows > 0), rows < 0,
 *                 vocab < 1, stride < vocab, vocab > 2^24 (the token
 *                 written as f32 must be exact), or a non-finite scale;
 *      CE_EALIGN: a pointer is not aligned to its element size;
 *      CE_ECUDA:  the CUDA runtime reported an error at launch
 *                 (ce_last_cuda_error() gives its code).
 *  - rows == 0 is valid and launches nothing, except that ce_loss, ce_mean
 *    and ce_grad_step (given a loss_mean) still write their mean (NaN: the
 *    mean of no rows).
 *  - A label outside [0, vocab) is found on the device: that row's loss
 *    is NaN, its gradient row gets no one-hot term, and a device counter
 *    (read by ce_device_error_count) is incremented. Nothing traps.
 *  - A row holding a NaN or +inf, or whose entries are all -inf, has a NaN
 *    loss and a NaN gradient row (the IEEE value of the definition). Its
 *    argmax still follows Tensor.argmax: NaN never wins, first of equals.
 */
#ifndef CE_ROWS_H
#define CE_ROWS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Symbols of this ABI are the library's only exported ones. */
#if defined(__GNUC__)
#define CE_API __attribute__((visibility("default")))
#else
#define CE_API
#endif

/* The CUDA runtime's cudaStream_t, without requiring CUDA headers. */
typedef struct CUstream_st *ce_stream_t;

enum ce_status {
    CE_OK = 0,
    CE_EINVAL = -1,
    CE_EALIGN = -2,
    CE_ECUDA = -3,
    CE_EDEVICE = -4, /* no CUDA device, or not an sm_103 device */
    CE_ERANGE = -5,  /* argmax_rows_noalloc: more rows than its fixed scratch holds */
};

/*
 * crossEntropyRows (gizml:netops, Functions): each row's loss
 *     m + log(sum_j exp(x_j - m)) - x[label],   m = max_j x_j,
 * as f32 into loss_rows[rows], computed on the device without a host wait.
 * The kernel evaluates the equal form (m - x[label]) + log1p(t), where t
 * sums exp(x_j - m) over all columns but one holding m, so a loss far below
 * the f32 resolution of m keeps its relative accuracy.
 *   logits:    [rows, stride] f32, read only.
 *   labels:    [rows] int64, read only.
 *   loss_rows: [rows] f32, written; must not overlap the inputs.
 */
CE_API int ce_rows(const float *logits, int64_t rows, int64_t vocab, int64_t stride,
            const int64_t *labels, float *loss_rows, ce_stream_t stream);

/*
 * The mean step of crossEntropyLoss (gizml:netops, Functions): the mean of
 * `rows` f32 row losses, accumulated in f64, written as one double to
 * *loss_mean (a device pointer; the value stays on the device, so a
 * recorded step never waits for it). The sum is a fixed-shape tree over a
 * cluster of CTAs that does not depend on the device: the same inputs give
 * the same bits on every run. The kernel is launched as a programmatic
 * dependent of the kernel before it on `stream` (it waits for that kernel to
 * complete before reading anything), so after this library's row kernels it
 * starts without a launch gap.
 *   loss_rows: [rows] f32, read only.   loss_mean: 1 double, written.
 */
CE_API int ce_mean(const float *loss_rows, int64_t rows, double *loss_mean, ce_stream_t stream);

/*
 * crossEntropyLoss (gizml:netops, Functions): ce_rows followed by ce_mean,
 * both enqueued on `stream`. loss_rows ([rows] f32) is required: it holds
 * the row losses (an output) that the mean reads.
 */
CE_API int ce_loss(const float *logits, int64_t rows, int64_t vocab, int64_t stride,
            const int64_t *labels, float *loss_rows, double *loss_mean, ce_stream_t stream);

/*
 * crossEntropyGrad (gizml:netops, Functions): the gradient
 *     grad[i, j] = (softmax_ij - [j == label_i]) * scale,
 *     softmax_ij = exp(x_ij - m_i) * f32(1 / sum_i),
 * with `scale` (e.g. 1/rows, the gradient of the mean over rows) rounded to
 * f32. One kernel reads each logit once from HBM and writes each gradient
 * once; from the same read it can also write each row's loss (as ce_rows).
 *   logits:    [rows, stride] f32, read only, unless grad == logits.
 *   labels:    [rows] int64, read only.
 *   grad:      [rows, vocab] f32 dense, written. grad == logits (in place)
 *              is allowed when stride == vocab; any other overlap is not.
 *   loss_rows: [rows] f32, or NULL.
 */
CE_API int ce_grad(const float *logits, int64_t rows, int64_t vocab, int64_t stride,
            const int64_t *labels, double scale, float *grad, float *loss_rows, ce_stream_t stream);

/*
 * The whole training-step path from one read of the logits: ce_grad's
 * gradient and row losses, each row's argmax token (argmaxInto's rule, as
 * argmax_rows writes it) and the mean loss (crossEntropyLoss, as ce_mean
 * writes it). Arguments as ce_grad, and:
 *   top:       [rows] f32, or NULL.
 *   loss_mean: 1 double on the device, or NULL; needs loss_rows (CE_EINVAL
 *              otherwise). The mean kernel is launched as a programmatic
 *              dependent of the fused kernel: it is scheduled while the fused
 *              kernel finishes and reads the row losses only once that kernel
 *              has completed, so the step costs no separate launch gap.
 */
CE_API int ce_grad_step(const float *logits, int64_t rows, int64_t vocab, int64_t stride,
                        const int64_t *labels, double scale, float *grad, float *loss_rows, float *top,
                        double *loss_mean, ce_stream_t stream);

/*
 * crossEntropyGrad and crossEntropyLoss of a batch that is in HOST memory:
 * the training step fed from the host, with the host-to-device copy
 * overlapped with the kernels. The labels, then the logits in chunks of
 * rows, are copied into caller-owned device buffers on a copy stream the
 * library keeps per device; the fused kernel (as ce_grad_step, with the
 * tokens) runs on each chunk on `stream` as soon as that chunk has landed, so
 * chunk c is computed while chunk c + 1 is copied. Then ce_mean over all the
 * rows, and the mean and tokens back to the host. Everything is enqueued: the call returns at once, and the host and
 * device buffers must stay valid, and the host outputs unread, until
 * `stream` has reached this point. Host inputs in page-locked memory copy
 * asynchronously; pageable ones work but the copies may block the caller.
 *   logits_h:    [rows, stride_h] f32, host, read only.
 *   labels_h:    [rows] int64, host, read only.
 *   logits_d:    [rows, vocab] f32 dense, device, written (the staged copy).
 *   labels_d:    [rows] int64, device, written.
 *   grad:        [rows, vocab] f32 dense, device, written; grad == logits_d
 *                (the gradient over the staged copy) is allowed.
 *   loss_rows:   [rows] f32, device, written.   top: [rows] f32 device or NULL.
 *   loss_mean:   1 double, device, written.
 *   loss_mean_h: 1 double, host, or NULL.    top_h: [rows] f32 host or NULL
 *                (needs top).
 *   chunk_rows:  rows per copied chunk; 0 picks 16 chunks (at most 64).
 * Calls that share device buffers must be ordered by their streams. The
 * same argument checks as ce_grad apply (CE_EINVAL / CE_EALIGN before any
 * copy); rows == 0 writes a NaN mean.
 */
CE_API int ce_grad_host(const float *logits_h, int64_t rows, int64_t vocab, int64_t stride_h,
                        const int64_t *labels_h, double scale, float *logits_d, int64_t *labels_d,
                        float *grad, float *loss_rows, float *top, double *loss_mean,
                        double *loss_mean_h, float *top_h, int64_t chunk_rows, ce_stream_t stream);

/*
 * argmaxInto (gizml:netops, Functions) with Tensor.argmax's rule (Methods):
 * over `rows` rows of `stride` elements, the index of the largest of the
 * first `vocab` entries -- the first of equals; NaN never wins; a row with
 * no non-NaN entry gives 0 -- written as f32 (exact, since vocab <= 2^24)
 * into top[rows]. The direct form (rows at logits + i * stride); for rows
 * given by a table of addresses see argmax_rows_indirect.
 *   logits:    [rows, stride] f32, read only.   top: [rows] f32, written.
 */
CE_API int argmax_rows(const float *logits, int64_t rows, int64_t vocab, int64_t stride, float *top,
                       ce_stream_t stream);

/*
 * argmax_rows_noalloc -- the tokens of argmax_rows (same rule, same f32
 * output) for callers that must not allocate device memory: code running
 * inside another runtime that owns and pre-plans every byte of device memory
 * (an inference server's memory planner, a plugin handed only its inputs
 * and outputs), and latency-critical decode loops where a cudaMalloc -- which
 * can synchronise the whole device -- is not acceptable. The pages have no
 * counterpart: argmaxInto takes no workspace.
 *
 * It allocates nothing: its scratch is a fixed 64 KiB array in the library's
 * own device memory (one 64-bit key per segment of the rows' even split over
 * the GPU), held on every device that loads the library until the process
 * exits. The caller still passes the logits and `top` as in argmax_rows.
 *   - A call with rows + 2 * (SMs of the device) <= 8192 always fits (7888
 *     rows on a 152-SM GB300); a call that does not fit returns CE_ERANGE
 *     and launches nothing.
 *   - The first call on a device looks up the array's device address on that
 *     device (cudaGetSymbolAddress, no allocation); make that first call
 *     before capturing any stream.
 *   - Every call uses the same array and leaves its contents there. Nothing
 *     in it needs to start at zero (each call reads only keys it wrote), but
 *     two calls that run at the same time on the GPU -- on different streams,
 *     or from different host threads -- race on it and may return wrong
 *     tokens; order them on one stream.
 */
CE_API int argmax_rows_noalloc(const float *logits, int64_t rows, int64_t vocab, int64_t stride, float *top,
                               ce_stream_t stream);

/*
 * Softmax rows: out[i, j] = exp(x_ij - m_i) * f32(1 / sum_i), the softmax of
 * crossEntropyGrad (gizml:netops, Functions) without its one-hot term and
 * scale -- the row softmax among the gpukit API page's device kernels
 * (dev.nu, gkd_softmax_rows). Same kernel, same single HBM read of each
 * logit and single write of each output as ce_grad.
 *   logits: [rows, stride] f32, read only, unless out == logits.
 *   out:    [rows, vocab] f32 dense, written. out == logits (in place) is
 *           allowed when stride == vocab; any other overlap is not.
 * A row holding a NaN or +inf, or all -inf, gives a NaN row; a -inf entry of
 * a finite row gives 0.
 */
CE_API int softmax_rows(const float *logits, int64_t rows, int64_t vocab, int64_t stride, float *out,
                        ce_stream_t stream);

/*
 * Log-softmax rows: out[i, j] = (x_ij - m_i) - log(sum_i), the log
 * probabilities of the tokens (a request's `logprobs`, guide "Tensors, GPU
 * kernels and AI models", Step 5). log(sum) is taken as log1p(t), t the sum
 * over all columns but one holding the max, so the log probability of a
 * dominant token keeps its relative accuracy. Layout, aliasing and
 * non-finite rows as softmax_rows; a -inf entry of a finite row gives -inf.
 */
CE_API int log_softmax_rows(const float *logits, int64_t rows, int64_t vocab, int64_t stride, float *out,
                            ce_stream_t stream);

/* candidatesInto's workgroup, TOP_EACH and CANDIDATE_ROW (gizml:netops, Constants). */
#define CE_CANDIDATE_THREADS 256
#define CE_TOP_EACH 4
#define CE_CANDIDATE_ROW 2048

/*
 * candidatesInto (gizml:netops, Functions; Constants TOP_EACH, CANDIDATE_ROW):
 * each row's sampling candidates. A workgroup of CE_CANDIDATE_THREADS = 256
 * threads reads the row; thread t reads columns t, t + 256, t + 512, ...
 * below vocab and keeps its CE_TOP_EACH = 4 largest values, ranked by value
 * and, among equal values, by the lower column (NaN is never kept). Row i's
 * candidates are the CE_CANDIDATE_ROW = 2048 floats at cand + 2048 * i:
 * float 2(4t + k) is thread t's rank-k value and float 2(4t + k) + 1 its
 * column as f32 (exact, vocab <= 2^24); a slot for which thread t read no
 * value holds (-inf, -1). Bit-exact: the values are copies of the logits.
 * The direct form (rows at logits + i * stride); for rows given by a table of
 * addresses see candidates_rows_indirect.
 *   logits: [rows, stride] f32, read only.
 *   cand:   [rows, 2048] f32, written; must not overlap the logits.
 */
CE_API int candidates_rows(const float *logits, int64_t rows, int64_t vocab, int64_t stride, float *cand,
                           ce_stream_t stream);

/*
 * argmaxInto and candidatesInto in their indirect form (gizml:netops,
 * Functions): the entries read "rows of `stride`, of the head blocks in
 * `blocks` when `indirect`"; the extracted sentence is garbled, and this
 * library takes its plainest reading -- row i is read at the device address
 * row_addrs[i] instead of at logits + i * stride (rows picked in place, e.g.
 * each sequence's last position, without gathering them first). Same rules,
 * outputs and kernels as argmax_rows / candidates_rows.
 *   row_addrs: [rows] uint64 device addresses of f32 rows, each with `vocab`
 *              readable floats; 8-byte aligned table, read only. Rows may
 *              repeat and may sit anywhere (4-byte aligned).
 *   top:  [rows] f32, written.   cand: [rows, 2048] f32, written.
 * An address that is null or not 4-byte aligned is detected on the device and
 * never read: that row's token is NaN, its candidates all (-inf, -1). The
 * outputs must not overlap any row.
 */
CE_API int argmax_rows_indirect(const uint64_t *row_addrs, int64_t rows, int64_t vocab, float *top,
                                ce_stream_t stream);
CE_API int candidates_rows_indirect(const uint64_t *row_addrs, int64_t rows, int64_t vocab, float *cand,
                                    ce_stream_t stream);

/*
 * splitSumInto (gizml:netops, Functions): joins `splits` partial results of
 * `total` f32 values each (part s at parts + s * total, e.g. the partial
 * products of a split reduction):
 *     y[i] = (add ? y[i] : 0) + parts[0][i] + ... + parts[splits-1][i],
 * added in f32 in split order. With add == 0 the old y is never read.
 *   y:     [total] f32, written (read first when add != 0).
 *   parts: [splits, total] f32, read only. y may be parts itself (part 0),
 *          any other overlap is rejected (CE_EINVAL).
 * total == 0 launches nothing; splits < 1 is CE_EINVAL.
 */
CE_API int split_sum(float *y, const float *parts, int64_t total, int64_t splits, int add, ce_stream_t stream);

/*
 * Vocab-sharded cross-entropy: the loss, token and gradient of rows whose
 * columns are split over slices (e.g. a language-model head whose vocabulary
 * is split over devices), with one exchange of 16 bytes per row and slice.
 * crossEntropyLoss (gizml:netops, Functions) defines the loss by the row max
 * m and exp-sum s = sum_j exp(x_j - m); both decompose over any split of the
 * columns (m = max_s m_s, s = sum_s exp(m_s - m) s_s), so:
 *   1. ce_stats on each slice            -> [rows] float4 per slice;
 *   2. gather the slices' stats in column order (the caller's exchange);
 *   3. ce_stats_combine                  -> each row's loss, token and the
 *                                           combined float4;
 *   4. ce_grad_from_stats on each slice  -> the slice of crossEntropyGrad.
 * The results equal ce_grad's on the whole rows (same rules for ties, NaN,
 * infinities and bad labels), up to f32 rounding order.
 *
 * ce_stats: per row of the slice [col0, col0 + vocab) -- `logits` points at
 * column col0 of row 0, rows `stride` apart -- the float4 (m, t, top, xl):
 *   m   the max of the slice's non-NaN values (-inf if none);
 *   t   sum of exp(x_j - m) over the slice but one element holding m; NaN if
 *       the slice holds a NaN; not meaningful when m is +-inf;
 *   top the global column of the first element holding m as f32, or -1 if
 *       the slice has no non-NaN value;
 *   xl  x[label] if col0 <= label < col0 + vocab, else 0.
 *   labels: [rows] int64 GLOBAL columns.   stats: [rows] x 4 f32, 16-byte
 *   aligned, written. col0 + vocab <= 2^24. No label is checked here.
 */
CE_API int ce_stats(const float *logits, int64_t rows, int64_t vocab, int64_t stride, int64_t col0,
                    const int64_t *labels, float *stats, ce_stream_t stream);

/*
 * ce_stats_combine: merges `shards` slices' stats (stats: [shards][rows] x 4
 * f32, slices in column order, 16-byte aligned) into each whole row's
 *   loss_rows (f32, or NULL): crossEntropyRows of the whole row;
 *   top       (f32, or NULL): the whole row's argmax token;
 *   combined  ([rows] x 4 f32, 16-byte aligned, or NULL): (M, T, top, x[label])
 *             of the whole row, the input of ce_grad_from_stats.
 * A label outside [0, vocab_total) gives a NaN loss and increments the
 * device counter, as ce_rows does.
 */
CE_API int ce_stats_combine(const float *stats, int64_t shards, int64_t rows, int64_t vocab_total,
                            const int64_t *labels, float *loss_rows, float *top, float *combined,
                            ce_stream_t stream);

/*
 * ce_grad_from_stats: the slice [col0, col0 + vocab) of crossEntropyGrad,
 *     grad[i, j] = (exp(x_ij - M_i) * f32(1 / (1 + T_i)) - [col0 + j == label_i]) * scale,
 * from the combined (M, T) of ce_stats_combine; dense [rows, vocab]. A row
 * whose M is infinite or T is NaN gives a NaN gradient row. grad == logits is
 * allowed when stride == vocab; any other overlap is not.
 */
CE_API int ce_grad_from_stats(const float *logits, int64_t rows, int64_t vocab, int64_t stride, int64_t col0,
                              const int64_t *labels, const float *combined, double scale, float *grad,
                              ce_stream_t stream);

/*
 * Objectives over sampled answers and over pairs of answers. They read the
 * same [rows, stride] logits and int64 labels as the calls above, in three
 * types, and share these conventions:
 *  - dtype: CE_F32, CE_BF16 or CE_F16, the type of the logits and of their
 *    gradient. Everything else of a row is f32; row statistics, losses and
 *    the gradient are computed in f32 and a gradient is rounded once, at the
 *    end. Sums over rows carry at least 48 bits relative to their largest
 *    partial sum and are rounded once to f32; a partial sum beyond f32 makes
 *    them infinite, also where `scale` would bring the result back.
 *  - f32 ends the range of a row's gradient factors too (scale, weight and 1 / T
 *    together with the loss's own factor): beyond it the row's gradient is not
 *    finite. A probability below 2^-126 relative to the row's largest counts
 *    as 0.
 *  - temperature T > 0 (1e-6 <= T <= 1e6): the distribution of a row is
 *    softmax(x / T); gradients are with respect to x.
 *  - weights: [rows] f32, or NULL (every row counts 1). A row of weight 0 (a
 *    prompt or padding token) takes no part: its logits, its label and its
 *    other inputs may hold anything, its outputs are 0 and its gradient row is
 *    zeros. Of such a row only the weight and the label are loaded (and the
 *    label not used).
 *  - gradients are with respect to the scaled loss and are written to rows
 *    grad_stride elements apart (grad_stride >= vocab; columns vocab and up
 *    are not written). grad == logits (in place) is allowed when grad_stride
 *    == stride (or rows == 1); any other overlap is CE_EINVAL.
 *  - Outputs and the work buffer share no byte with an input or with one
 *    another (CE_EINVAL); they may lie in the padding of the logits' rows.
 *  - A label outside [0, vocab) on a row that counts gives that row a NaN
 *    log-probability (and so a NaN loss and gradient row) and increments the
 *    device counter. A row holding a NaN or +inf, or nothing above -inf, is
 *    NaN likewise. -inf logits of other rows have probability 0; a label
 *    there has log-probability -inf.
 *  - log-probabilities and entropies carry an absolute error of a few f32
 *    roundings of log(s), not a relative one near 0; ce_rows keeps the
 *    relative accuracy of tiny losses.
 *  - rows == 0 is valid: the scalar loss is still written (0).
 *  - The calls keep nothing between them and are safe side by side on several
 *    streams, given each its own outputs and work buffer.
 */
enum ce_dtype { CE_F32 = 0, CE_BF16 = 1, CE_F16 = 2 };

/*
 * logp_rows: the log-probability of each row's label,
 *     logp = (x[label] - m) / T - log(s),  m = max_j x_j,  s = sum_j exp((x_j - m) / T),
 * and, with `entropy`, the row's entropy H = -sum_j p_j log p_j, from one read
 * of the logits: what the two losses below take as the sampling policy's and
 * the reference's log-probabilities, for a decode step's few rows or a whole
 * batch. An entry of probability 0 adds 0 to the entropy.
 *   logp:    [rows] f32, written.   entropy: [rows] f32, or NULL.
 */
CE_API int logp_rows(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                     const int64_t *labels, const float *weights, double temperature, float *logp, float *entropy,
                     ce_stream_t stream);

/* The policy loss's constants. clip_low, clip_high >= 0, INFINITY: no clip on
 * that side; kl_coef, entropy_coef and scale finite. */
typedef struct ce_policy {
    double scale, temperature, clip_low, clip_high, kl_coef, entropy_coef;
} ce_policy;

/*
 * policy_loss: the clipped policy loss of tokens sampled by an older policy,
 * with a KL term to a reference policy and an entropy bonus. Per row, with
 * r = exp(logp - old_logp), A the advantage and d = ref_logp - logp:
 *     l = max(-A r, -A clamp(r, 1 - clip_low, 1 + clip_high))
 *         + kl_coef (exp(d) - 1 - d) - entropy_coef H
 *     loss = scale * sum_i weights_i l_i
 *   old_logp, advantages: [rows] f32.   ref_logp: [rows] f32, or NULL when
 *   kl_coef == 0 (then never read).
 *   loss_rows: [rows] f32, the l_i (unweighted).   logp: [rows] f32.
 *   entropy: [rows] f32, or NULL.   loss: 1 f32, all written on the device.
 */
CE_API int policy_loss(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                       const int64_t *labels, const float *old_logp, const float *advantages, const float *ref_logp,
                       const float *weights, const ce_policy *policy, float *loss_rows, float *logp, float *entropy,
                       float *loss, ce_stream_t stream);

/*
 * policy_step: policy_loss and its gradient, with
 *     g = [-A r where -A r is the larger term, or the terms are equal] + kl_coef (1 - exp(d)):
 *     grad[i, j] = scale weights_i / T (g ([j == label] - p_j) + entropy_coef p_j (log p_j + H)).
 * Each logit is read once from HBM and each gradient written once (rows that
 * do not fit the shared memory of 16 CTAs, about 3.5 MB, are read twice).
 */
CE_API int policy_step(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                       const int64_t *labels, const float *old_logp, const float *advantages, const float *ref_logp,
                       const float *weights, const ce_policy *policy, void *grad, int64_t grad_stride,
                       float *loss_rows, float *logp, float *entropy, float *loss, ce_stream_t stream);

enum ce_preference_kind { CE_PREF_SIGMOID = 0, CE_PREF_HINGE = 1, CE_PREF_SQUARED = 2 };

/* The preference loss's constants: beta > 0, 0 <= label_smoothing <= 0.5
 * (sigmoid only), margin and scale finite; average: sequences are averaged
 * over their tokens (by weight) rather than summed. */
typedef struct ce_preference {
    double scale, temperature, beta, label_smoothing, margin;
    int kind, average;
} ce_preference;

/*
 * preference_loss: the loss of `pairs` pairs of sequences, one preferred to
 * the other. The batch's rows hold 2 * pairs sequences, sequence s being rows
 * offsets[s] .. offsets[s + 1] - 1; sequence p is the chosen one of pair p and
 * sequence pairs + p the rejected one. With L_s the sum of weights * logp over
 * a sequence (average: divided by its sum of weights; 0 where that is 0), R_s
 * the same of the reference model (0 without one),
 *     h = (L_p - L_{pairs+p}) - (R_p - R_{pairs+p}),  z = beta h - margin:
 *     sigmoid  l = -(1 - eps) log sigma(z) - eps log sigma(-z)
 *     hinge    l = max(0, 1 - z)
 *     squared  l = (h - margin - 1 / (2 beta))^2
 *     loss = scale * sum_p l_p
 * h is formed in f64; sigmoid and hinge round z once to f32 and go on in f32, so
 * the loss and the factor of a saturated pair carry a relative error of
 * |z| 2^-24. Where l has a zero, l near it carries h's absolute error.
 *   offsets: [2 * pairs + 1] int64 on the device, non-decreasing, within
 *     [0, rows]. Rows in no sequence count as rows of weight 0. A sequence may
 *     be empty (L = 0). Nothing is read or written out of range whatever the
 *     table holds: a pair with a range that is not valid has a NaN loss (so the
 *     sum is NaN too), its bad sequence no rows, and each bad range increments
 *     the device counter; of a table that decreases somewhere, the other pairs
 *     may have lost rows as well.
 *   ref_logp: [2 * pairs] f32, the R_s (seq_logp of a call on the reference
 *     model's logits), or NULL.
 *   logp: [rows] f32.   seq_logp: [2 * pairs] f32, the L_s.
 *   loss_pairs: [pairs] f32, the l_p.   loss: 1 f32, all written on the device.
 *   work: 16 bytes of scratch, 16-byte aligned; two calls that may run at the
 *     same time need one each.
 */
CE_API int preference_loss(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                           const int64_t *labels, const float *weights, const int64_t *offsets, int64_t pairs,
                           const float *ref_logp, const ce_preference *preference, float *logp, float *seq_logp,
                           float *loss_pairs, float *loss, void *work, ce_stream_t stream);

/*
 * preference_step: preference_loss and its gradient: a row of a chosen (+) or
 * rejected (-) sequence gets +- scale dl/dh weight / (sum of weights | 1) / T
 * * ([j == label] - p_j); rows in no sequence get zeros. The factor of a row is
 * known only once its pair has been read, so the logits are read twice.
 *   work: 16 * (rows + 1) bytes, 16-byte aligned, as above.
 */
CE_API int preference_step(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                           const int64_t *labels, const float *weights, const int64_t *offsets, int64_t pairs,
                           const float *ref_logp, const ce_preference *preference, void *grad, int64_t grad_stride,
                           float *logp, float *seq_logp, float *loss_pairs, float *loss, void *work,
                           ce_stream_t stream);

/*
 * The choices made from a row's softmax.
 *
 *  - Logits are CE_F32, CE_BF16 or CE_F16, rows as above, fewer than 2^31 of
 *    them; arithmetic is f32, sums over a row of 32 bits or more.
 *  - The random numbers are inputs: f32 in [0, 1); of a number that draws, one
 *    outside counts as the nearest inside, NaN as 0.
 *  - Tokens and experts are int64; -1: none. Of equal columns the lowest wins.
 *  - A row holding a NaN or +inf, or nothing above -inf, is no distribution:
 *    its token is -1 and its log-probability NaN, and the device counter
 *    (ce_device_error_count) is incremented. -inf logits of other rows are
 *    never drawn.
 *  - Outputs and the work buffer share no byte with an input or with one
 *    another (CE_EINVAL); they may lie in the padding of the logits' rows.
 *  - The calls keep nothing between them and are safe side by side on several
 *    streams, given each its own outputs and work buffer.
 */

/*
 * Bytes of scratch (host only): of sample_rows with requests = -1, else of
 * verify_drafts; negative for arguments that they refuse.
 */
CE_API int64_t choice_work(int dtype, int64_t rows, int64_t vocab, int64_t requests);

/*
 * sample_rows: a token drawn from each row's softmax at a temperature. With
 * e_j = exp((x_j - m) / T), m = max_j x_j and S = sum_j e_j, row i's token is
 *     the first k with e_0 + ... + e_k > u_i S
 * (columns in order; e_j below 2^-126 counts as 0). T = 0 is the row's argmax.
 * Where u_i S lies within the rounding of a border between two columns either may
 * be taken; the same call gives the same tokens always. A border is off by less
 * than 2^-15 of S if all roundings add up, by less than 2^-24 as measured.
 *   uniforms: [rows] f32, the u_i.
 *   temperature: 0, or in [1e-6, 1e6].   temperatures: [rows] f32, likewise,
 *     instead of it, or NULL; a row whose entry is neither counts as no
 *     distribution.
 *   tokens: [rows] int64.   logp: [rows] f32, or NULL: the token's
 *     log-probability at that temperature (0 for T = 0), as logp_rows gives it.
 *   work: scratch of choice_work(dtype, rows, vocab, -1) bytes, 16-byte
 *     aligned; two calls that may run at the same time need one each.
 */
CE_API int sample_rows(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                       const float *uniforms, double temperature, const float *temperatures, int64_t *tokens,
                       float *logp, void *work, ce_stream_t stream);

/*
 * verify_drafts: drafted tokens accepted or replaced so that what a request
 * emits is distributed as if every token had been drawn from the target model.
 * Request s is rows offsets[s] .. offsets[s + 1] - 1. With p and q the softmax
 * of a row and of its draft row at the row's temperature, (a, u) its two random
 * numbers and d its draft:
 *     d is accepted where a q_d < p_d (a as it is given: a NaN accepts
 *     nothing) and p_d > 0;
 *     otherwise a token is drawn by u, as sample_rows draws it, from
 *     max(0, p_j - q_j) in proportion; the columns beside a looked-up draft are
 *     weighed by the largest of them, and count as 0 where that one is below
 *     2^-126 of the draft's weight.
 * A request emits its accepted drafts, row by row, up to the first row that
 * accepts none, and that row's drawn token. A row without a draft draws from p:
 * the row behind the last draft of a request has none. A row at temperature 0
 * draws its argmax and accepts a draft that is it.
 *   drafts: [rows] int64; negative: the row has none (its draft row is not
 *     read). A draft of vocab or more is counted and taken for none.
 *   draft_logits: the logits that the drafts were drawn from, of the logits'
 *     type, row i at draft_logits + i * draft_stride; NULL: the drafts were
 *     looked up, not drawn, and q is 1 at d. A draft row that is no distribution
 *     is counted, its draft not accepted and the token drawn from p; so is the
 *     token where no column has p_j > q_j.
 *   offsets: [requests + 1] int64 on the device, non-decreasing, within
 *     [0, rows]. A request may have no rows. Nothing is read or written out of
 *     range whatever the table holds: a range that is not valid is counted and
 *     its request's `accepted` is -1. A row that such a table leaves to no request,
 *     or outside offsets[0] .. offsets[requests], emits nothing; one that it gives to
 *     several may emit any one's token, or none.
 *   uniforms: [rows, 2] f32, the pairs (a, u).   temperature, temperatures: as
 *     in sample_rows.
 *   accepted: [requests] int64, the drafts accepted.
 *   tokens: [rows] int64, what the row emits; -1 for a row behind the request's
 *     last, and for rows in no request.   logp: [rows] f32, or NULL: the
 *     token's log-probability under p (0 at temperature 0 and where none is
 *     emitted).
 * What is counted, is so once for a request that it ends.
 *   work: scratch of choice_work(dtype, rows, vocab, requests) bytes, as above.
 */
CE_API int verify_drafts(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride,
                         const int64_t *drafts, const void *draft_logits, int64_t draft_stride,
                         const int64_t *offsets, int64_t requests, const float *uniforms, double temperature,
                         const float *temperatures, int64_t *accepted, int64_t *tokens, float *logp, void *work,
                         ce_stream_t stream);

enum ce_route_score { CE_ROUTE_SOFTMAX = 0, CE_ROUTE_SIGMOID = 1 };

/* A router: the scores, experts per row k (1..32), the experts' groups (1..32,
 * a divisor of the experts), how many of them a row keeps (top_groups), by the
 * sum of how many of their best members (group_top: 1 or 2); whether the gates
 * are renormalised, and their scale (finite in f32). */
typedef struct ce_route {
    int score, k, groups, top_groups, group_top, renormalise;
    double scale;
} ce_route;

/*
 * route_rows: each row's experts and gates, from router logits [rows, experts],
 * experts <= 1024. With the scores s = softmax(x) or sigma(x) and c = s + bias:
 *     a row keeps the top_groups groups with the largest sum of their group_top
 *     best c (top_groups == groups: all), and of their experts the k best c,
 *     best first;
 *     gate = scale s_e, or renormalised scale s_e / (sum of the chosen's s).
 * The bias has a part in the choice only. An expert whose logit is -inf (or
 * whose c is NaN or -inf) is never chosen and counts for nothing in its group; a
 * slot that no expert is left for is -1 with a gate of 0. A row holding a NaN or
 * +inf has no experts and NaN gates, and is counted. Scores that differ by less
 * than their rounding may change places, in the groups' sums those below 2^-126
 * of the row's largest.
 *   bias: [experts] f32, or NULL.   weights: [rows] f32, or NULL; a row of
 *     weight 0 is padding: not read, no experts, gates of 0. Other weights all
 *     mean the same.
 *   chosen: [rows, k] int64.   gates: [rows, k] f32.
 *   counts: [experts] int64, or NULL: the rows that chose each expert.
 */
CE_API int route_rows(const void *logits, int dtype, int64_t rows, int64_t experts, int64_t stride,
                      const ce_route *route, const float *bias, const float *weights, int64_t *chosen, float *gates,
                      int64_t *counts, ce_stream_t stream);

/*
 * route_grad: the gradient of route_rows' gates with respect to the logits, for
 * a given choice of experts: with G = scale * gates_grad, c the chosen, f their
 * share of the sum of their scores and D = sum of f G,
 *     renormalised  softmax  grad_c = f (G - D);  sigma  f (G - D) (1 - s_c)
 *     otherwise     softmax  grad_j = s_j ([j chosen] G - sum of s_c G_c)
 *                   sigma    grad_c = s_c (1 - s_c) G
 * and 0 elsewhere, in the logits' type. An expert that a row names twice counts
 * twice. Groups and bias have no part in it (route's are not read); rows of
 * weight 0 and rows without experts get zeros.
 *   chosen: [rows, k] int64; -1: none; one outside [-1, experts) is counted and
 *     taken for none.   gates_grad: [rows, k] f32.
 *   grad: rows grad_stride >= experts apart; grad == logits (in place) is
 *     allowed when grad_stride == stride (or rows == 1).
 */
CE_API int route_grad(const void *logits, int dtype, int64_t rows, int64_t experts, int64_t stride,
                      const ce_route *route, const float *weights, const int64_t *chosen, const float *gates_grad,
                      void *grad, int64_t grad_stride, ce_stream_t stream);

/* Human-readable text of a status code (a static string). */
CE_API const char *ce_status_string(int status);

/* Library version (major * 10000 + minor * 100 + patch). */
CE_API int ce_version(void);

/* The cudaError_t code behind the calling thread's last CE_ECUDA. */
CE_API int ce_last_cuda_error(void);

/*
 * Device-side error counter of the current device, for tests and
 * diagnostics: *out = rows seen with a label outside [0, vocab), bad
 * sequence ranges, and what the choices above count, since the last reset. This call WAITS for `stream` to
 * finish.
 */
CE_API int ce_device_error_count(ce_stream_t stream, int64_t *out);

/*
 * The second device counter: waits on an asynchronous copy or a peer CTA
 * that gave up after their time limit (the output of such a call is then
 * undefined; the kernel still ran to its end). WAITS for `stream`.
 * ce_device_error_reset zeroes both counters (enqueued on `stream`).
 */
CE_API int ce_device_wait_timeouts(ce_stream_t stream, int64_t *out);
CE_API int ce_device_error_reset(ce_stream_t stream);

/*
 * Launch-plan override, for tests and tuning (not of the objectives, whose
 * kernels follow from sizes and types alone): forces the kernel family
 * (path: 0 automatic, 1 shared-memory-staged (persistent), 2 streaming from
 * global, 3 refused (formerly a ring-of-copies kernel), 4
 * shared-memory-staged with one row per cluster, 5 refused (the argmax split
 * evenly over the GPU is argmax_rows_noalloc's own plan), 6 one warp per row -- ce_rows, ce_loss,
 * argmax_rows and ce_stats only, 7 argmax through a ring of bulk-copied row
 * chunks -- argmax_rows and argmax_rows_indirect only), the CTAs that share
 * one row (cluster: 0 automatic, else 1..16; candidates_rows and path 7 take
 * at most 8) and the threads of a CTA (threads: 0 automatic, else 128 or
 * 256; 512 is rejected by every kernel family; candidates_rows and path 7
 * take 256 only).
 * Applies to every later call in the process. A forced plan that cannot
 * launch on this device makes the calls return CE_EINVAL.
 */
CE_API int ce_debug_force(int path, int cluster, int threads);

/*
 * Grid override, for tests: at most `clusters` clusters (0: no cap) in every
 * later launch of a row kernel (not argmax_rows_noalloc's, sample_rows' and
 * verify_drafts'), so that each
 * cluster loops over several rows even when the rows are few. Results are
 * the same; only the schedule changes. Returns CE_EINVAL for clusters < 0.
 */
CE_API int ce_debug_grid_cap(int64_t clusters);

/*
 * Read probe, for measurement: reads `bytes` bytes at device address p (16-byte
 * aligned, bytes a multiple of 16) once -- one CTA per SM, 32 KB chunks by
 * bulk asynchronous copies through four shared-memory stages, the fastest
 * plain read of a large buffer measured on this device -- and XORs every word
 * read into *out (4 bytes on the device, not cleared first). No page defines
 * it: it gives the ceiling of a plain read of a buffer of that size on this
 * device, to time beside a row kernel that reads the same bytes.
 */
CE_API int ce_debug_read(const void *p, int64_t bytes, uint32_t *out, ce_stream_t stream);

/*
 * The plan the library would pick (host only, launches nothing) for
 * op (0 ce_rows, 1 ce_grad, 2 argmax_rows, 3 softmax_rows, 4
 * log_softmax_rows, 5 candidates_rows) on the current device:
 * out[0] path, out[1] cluster, out[2] threads, out[3] dynamic shared bytes
 * per CTA, out[4] columns per CTA, out[5] CTAs in the grid.
 */
CE_API int ce_plan(int op, int64_t rows, int64_t vocab, int64_t stride, int64_t out[6]);

#ifdef __cplusplus
}
#endif

#endif /* CE_ROWS_H */
