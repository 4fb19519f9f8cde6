/*
 * rowops.h - C ABI of librowops, the GB300 (sm_103a) row-wise
 * normalise-and-reduce ops of a transformer training step, the
 * mixture-of-experts layer behind its router, and what lies between two
 * sublayers' products (dropout, the residual's addition and its norm).
 *
 * Every op works on row-major matrices of `rows` x `cols` with row stride `cols`
 * (fp32; the operators behind rowops_dtype also fp16, bf16, e4m3 and e2m1) and
 * launches hand-written CUDA kernels on the caller's stream.
 *
 * Common contract (applies to every entry point below):
 *   - Pointers are DEVICE pointers on the current CUDA device.  The caller owns
 *     every buffer (inputs, outputs and workspace); the library never allocates
 *     device memory and keeps no per-call state, so calls are reentrant.
 *   - Calls are asynchronous: they validate the arguments on the host, queue
 *     the kernel(s) on `stream` and return.  No call synchronises the device.
 *   - A NULL `stream` is the legacy default stream.
 *   - Return value: ROWOPS_OK, or the first error found.  Nothing is launched
 *     when an error is returned, except ROWOPS_ERR_CUDA, which reports a failed
 *     launch (the CUDA runtime's error after the launch).
 *   - rows == 0 is a successful no-op for every op (after the scalar
 *     parameters are checked), except rowops_column_sums, which still scales
 *     its output by beta.  Negative sizes, cols >= 2^31, and matrices of
 *     more than 2^60 elements are ROWOPS_ERR_SHAPE.
 *   - A pointer may be NULL only when the buffer it names is empty.
 *   - Buffers must not overlap unless the entry point says so
 *     (ROWOPS_ERR_ALIAS); overlap is checked by address range.
 *   - Every pointer must be aligned to its element type (4 bytes for float
 *     and int32_t, 8 for double, any for uint8_t); a pointer that is not is
 *     ROWOPS_ERR_ALIGN.  Beyond that any alignment is accepted: 16-byte
 *     aligned buffers with cols % 4 == 0 take the 128-bit vector path; others
 *     take scalar paths with the same results up to fp32 rounding order.
 *   - Reductions use a fixed order: repeated calls on the same inputs give
 *     bit-identical outputs.
 *
 * The definitions follow four API-documentation pages:
 *   [P1] pulsatrix HIPBackend class reference
 *   [P2] MicroGPT CuBLASBackend API page
 *   [P3] TorchLean NN.Runtime.Autograd.Engine.LibTorch.Kernels (CUDA buffer kernels FFI)
 *   [P4] oxicuda-backend ComputeBackend trait
 */
#ifndef ROWOPS_H
#define ROWOPS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ROWOPS_OK = 0,
    ROWOPS_ERR_NULL = 1,      /* a required pointer is NULL */
    ROWOPS_ERR_SHAPE = 2,     /* bad size, k, seq_len, scale, eps or grad_scale */
    ROWOPS_ERR_ALIAS = 3,     /* buffers overlap where the op forbids it */
    ROWOPS_ERR_WORKSPACE = 4, /* workspace missing, misaligned or too small */
    ROWOPS_ERR_CUDA = 5,      /* the CUDA runtime reported an error at launch */
    ROWOPS_ERR_ALIGN = 6      /* a pointer is not aligned to its element type */
} rowops_status;

/* Same object as cudaStream_t. */
typedef struct CUstream_st *rowops_stream;

/* Human-readable name of a status code (static string, never NULL). */
const char *rowops_status_string(int status);

/* Number of kernels this library has queued since it was loaded (all devices,
 * all threads).  Diagnostic counter for benchmarks. */
uint64_t rowops_kernel_launches(void);

/* Number of times a pipelined kernel of this library gave up a bounded wait on
 * the current device since the library was loaded (0 in correct operation; a
 * kernel that gives up leaves its outputs incomplete).  Synchronous: copies a
 * counter from the device; returns 0xffffffff if the copy fails. */
uint32_t rowops_pipeline_timeouts(void);

/*
 * Row softmax, max-subtracted.  [P1] softmax_rows(in, out, rows, cols); [P2]
 * softmax_rows(x); [P4] softmax(..., axis) on the last axis.
 *   y_ij = exp(x_ij - m_i) / sum_k exp(x_ik - m_i),  m_i = max_k x_ik.
 * x, y: rows x cols.  y may be exactly x (in place, as [P1] allows); any other
 * overlap is ROWOPS_ERR_ALIAS.  cols == 0 is a no-op ([P3]'s softmax accepts
 * empty tensors).
 */
int rowops_softmax_fwd(const float *x, float *y, int64_t rows, int64_t cols,
                       rowops_stream stream);

/*
 * Softmax backward from the output.  [P1] softmax_rows_backward(y, dy, dx, ...);
 * [P2] softmax_backward(s, ds).
 *   dx_ij = y_ij * (dy_ij - sum_k y_ik * dy_ik).
 * y, dy, dx: rows x cols.  dx must not overlap y or dy ([P1]).  cols == 0 is a
 * no-op.
 */
int rowops_softmax_bwd(const float *y, const float *dy, float *dx, int64_t rows, int64_t cols,
                       rowops_stream stream);

/*
 * Scaled causal attention softmax.  [P2] fused_attn_softmax(scores, scale) on the
 * stacked (batch*heads*seq_len, seq_len) score rows of
 * causal_mask_batched(scores, seq_len): row r is query i = r mod seq_len and
 *   p_rj = exp(scale*s_rj - m_r) / sum_{k<=i} exp(scale*s_rk - m_r)  for j <= i,
 *   p_rj = 0 (exactly +0.0)                                       for j > i,
 * with m_r = max_{k<=i} scale*s_rk.  Only the entries j <= i of `scores` are
 * read.  Requires seq_len >= 1, cols == seq_len, rows % seq_len == 0 and
 * 0 < scale < inf (else ROWOPS_ERR_SHAPE).  p must not overlap scores.
 */
int rowops_attn_softmax_fwd(const float *scores, float *p, int64_t rows, int64_t cols,
                            int64_t seq_len, float scale, rowops_stream stream);

/*
 * Backward of rowops_attn_softmax_fwd with respect to the raw scores, from its
 * output p.  [P2] fused_attn_softmax_backward(s, ds, scale).
 *   c_r = sum_{k<=i} p_rk dp_rk,  ds_rj = scale * p_rj * (dp_rj - c_r) for j <= i,
 *   ds_rj = 0 (exactly +0.0) for j > i.
 * Only the entries j <= i of p and dp are read.  Same shape rules as the
 * forward.  ds must not overlap p or dp.
 */
int rowops_attn_softmax_bwd(const float *p, const float *dp, float *ds, int64_t rows,
                            int64_t cols, int64_t seq_len, float scale, rowops_stream stream);

/*
 * Hard-masked row softmax.  [P3] stable row-wise hard-masked softmax.
 *   A_i = { j : mask_ij != 0 },  y_ij = exp(x_ij - max_{A_i} x) / sum_{A_i} exp(.)
 *   for j in A_i;  y_ij = +0.0 for j not in A_i;  a row with empty A_i is all +0.0.
 * x, y: rows x cols fp32; mask: rows x cols bytes, any nonzero byte allows.  y may
 * be exactly x; any other overlap (with x or mask) is ROWOPS_ERR_ALIAS.  cols == 0
 * is a no-op.
 */
int rowops_masked_softmax(const float *x, const uint8_t *mask, float *y, int64_t rows,
                          int64_t cols, rowops_stream stream);

/*
 * Per-row log-sum-exp, max-subtracted.  [P1] logsumexp_rows(in, out, rows, cols).
 *   lse_i = m_i + log sum_j exp(x_ij - m_i).
 * x: rows x cols; lse: rows.  cols == 0 writes -inf (log of an empty sum); a row
 * whose maximum is +-inf gets that maximum.  lse must not overlap x.
 */
int rowops_logsumexp(const float *x, float *lse, int64_t rows, int64_t cols,
                     rowops_stream stream);

/*
 * Fused softmax cross-entropy loss and logits gradient for integer targets.
 * [P2] fused_softmax_ce_grad(logits, targets) -> (Float64 loss, grad).
 *   loss_i = lse_i - x_{i,t_i}
 *   grad_ij = grad_scale * (softmax(x_i)_j - [j == t_i])
 *   *mean_loss = (1/rows) * sum_i loss_i   (fixed summation order; summed as a
 *   double-word fp32 value, about 48 significant bits, and returned as a double;
 *   a sum that is not finite in that form is redone in double)
 * logits, grad: rows x cols fp32; targets: rows int32; row_loss: rows fp32
 * (written, then reduced into the mean); mean_loss: ONE double in device memory.
 * grad_scale = 1/rows gives the gradient of the mean loss.  A target outside
 * [0, cols) cannot be checked without a device sync, so it is defined instead:
 * that row's row_loss is NaN (hence *mean_loss is NaN) and its gradient row is
 * grad_scale * softmax with no one-hot term.  cols == 0 and a non-finite
 * grad_scale are ROWOPS_ERR_SHAPE.  No output may overlap another buffer.
 */
int rowops_softmax_ce(const float *logits, const int32_t *targets, float *grad,
                      float *row_loss, double *mean_loss, int64_t rows, int64_t cols,
                      float grad_scale, rowops_stream stream);

/*
 * LayerNorm forward over the columns.  [P1] layer_norm_forward(); [P2]
 * layer_norm_forward(x, gamma, beta); [P3] layer normalisation returning
 * (output, normalized, invStd).
 *   mu_i = mean_j x_ij,  v_i = mean_j (x_ij - mu_i)^2 (population variance),
 *   inv_std_i = 1/sqrt(v_i + eps),  xhat_ij = (x_ij - mu_i) * inv_std_i,
 *   out_ij = gamma_j * xhat_ij + beta_j.
 * x, out, xhat: rows x cols; gamma, beta: cols; inv_std: rows.  cols == 0,
 * eps < 0 or non-finite eps are ROWOPS_ERR_SHAPE.  No output may overlap another
 * buffer.
 */
int rowops_layernorm_fwd(const float *x, const float *gamma, const float *beta, float *out,
                         float *xhat, float *inv_std, int64_t rows, int64_t cols, float eps,
                         rowops_stream stream);

/* Bytes of device workspace rowops_layernorm_bwd needs for this shape (a pure
 * function of rows and cols; 0 when rows or cols is 0 or negative). */
size_t rowops_layernorm_bwd_workspace(int64_t rows, int64_t cols);

/*
 * LayerNorm backward.  [P3] layer-normalisation VJP returning (dX, dGamma,
 * dBeta); [P2] layer_norm_backward(grad, norm, std_inv, gamma); [P1]
 * layer_norm_backward() for dX and column_sums() for the parameter sums.
 *   g'_ij = dy_ij * gamma_j
 *   dx_ij = inv_std_i * (g'_ij - mean_k g'_ik - xhat_ij * mean_k (g'_ik xhat_ik))
 *   dgamma_j = sum_i dy_ij * xhat_ij,   dbeta_j = sum_i dy_ij   (overwritten)
 * dy, xhat, dx: rows x cols; gamma, dgamma, dbeta: cols; inv_std: rows.  The
 * column sums are deterministic: fixed blocks of rows write partial sums into
 * `workspace` (at least rowops_layernorm_bwd_workspace(rows, cols) bytes of
 * 16-byte aligned device memory; its contents need not be initialised and are
 * garbage afterwards), then a second kernel, a programmatic dependent of the
 * first, adds the partials in a fixed order.  The workspace size depends on
 * rows, cols and the current device's SM count (the partials are per CTA or
 * per cluster of a grid sized to one wave); query it with the device current
 * that will run the call.  Concurrent calls need separate workspaces.
 * cols == 0 is ROWOPS_ERR_SHAPE; a short, NULL or misaligned workspace is
 * ROWOPS_ERR_WORKSPACE.  No output may overlap another buffer.  Rows of
 * 384..1024 floats whose CTA blocks are too large for shared memory stream
 * through a bulk-copy ring whose waits are bounded: a wait that runs out (a
 * defect) leaves dx, dgamma and dbeta incomplete and counts one timeout, so
 * callers that must know check rowops_pipeline_timeouts() after
 * synchronizing.
 */
int rowops_layernorm_bwd(const float *dy, const float *gamma, const float *xhat,
                         const float *inv_std, float *dx, float *dgamma, float *dbeta,
                         int64_t rows, int64_t cols, void *workspace, size_t workspace_bytes,
                         rowops_stream stream);

/*
 * LayerNorm backward that allocates nothing and takes no workspace.  The pages
 * have no counterpart; this is a convenience of this library.
 *
 * Some callers cannot obtain device memory when they need this op: code that
 * runs under a fixed device-memory budget set aside up front, plugins whose
 * host framework owns every allocation and offers no scratch space, or code
 * that must not enter an allocator at all (inside an allocator's own
 * out-of-memory path, for instance).  For them this entry point computes
 * what rowops_layernorm_bwd computes (bit for bit wherever both run the same
 * CTA count; see below), with the same argument rules, using a workspace that
 * lives inside the library: a fixed array of
 * rowops_layernorm_bwd_noalloc_max_bytes() bytes (1 MiB) of device memory,
 * which every GPU that loads the library holds until the process exits.
 *
 *   - The first call on each device looks up that array's device address
 *     (with the device current); make that first call before any stream
 *     capture.  Later calls reuse the address for the life of the process, so
 *     a device reset (cudaDeviceReset) after the first call on that device is
 *     not supported.
 *   - Errors are reported in this order: the argument checks of
 *     rowops_layernorm_bwd (shape, NULL, alignment, overlap), then the size
 *     check below, then a failed address lookup (ROWOPS_ERR_CUDA).
 *   - Each CTA's partial sums take 8 * cols bytes.  Rows of up to 1024 floats
 *     fit for every row count: the launch uses only as many CTAs as the array
 *     holds partials for (rows of 863..1024 floats then run on fewer CTAs
 *     than rowops_layernorm_bwd uses where a CTA's rows fit in shared memory,
 *     so dgamma and dbeta are added in another order and dx may come from the
 *     other stage-1 kernel; both agree with rowops_layernorm_bwd within the
 *     parity bounds).  Wider rows fit while rows is small enough
 *     (e.g. 64 rows of 2048 floats, 8 rows of 16384); larger shapes are
 *     refused with ROWOPS_ERR_WORKSPACE.
 *   - All calls on a device share the one array, and it keeps the contents of
 *     the last call.  Nothing in it needs to start at zero: each call writes
 *     every partial sum it later reads.  Calls that can overlap on the GPU
 *     (different streams, no ordering between them) race on the array and may
 *     return wrong dgamma/dbeta; order them, or use rowops_layernorm_bwd with
 *     separate workspaces.
 *   - Bounded waits that run out are counted as for rowops_layernorm_bwd:
 *     check rowops_pipeline_timeouts() after synchronizing.
 *   - It never calls cudaMalloc, cudaFree or any other allocating routine.
 */
int rowops_layernorm_bwd_noalloc(const float *dy, const float *gamma, const float *xhat,
                                 const float *inv_std, float *dx, float *dgamma, float *dbeta,
                                 int64_t rows, int64_t cols, rowops_stream stream);

/* Size in bytes of the array rowops_layernorm_bwd_noalloc uses (1 MiB). */
size_t rowops_layernorm_bwd_noalloc_max_bytes(void);

/*
 * Top-k kept mask.  [P3] kept mask (Spec.MoE.kept): entry i of a row is kept
 * when fewer than k entries of the row beat it; entry j beats entry i when
 * x_j > x_i, or when neither is larger and j < i.
 *   kept_ij = 1.0f if #{ j' : j' beats j } < k, else 0.0f.
 * The result is exact (comparisons and counts only) and equals the literal
 * compare-and-count for every input, NaN included (a NaN is neither larger nor
 * smaller than anything, so it ties).  x, kept: rows x cols fp32.  Requires
 * 1 <= k <= cols ([P1] top_k_rows precondition), else ROWOPS_ERR_SHAPE.  kept
 * must not overlap x.
 */
int rowops_topk_kept(const float *x, float *kept, int64_t rows, int64_t cols, int64_t k,
                     rowops_stream stream);

/*
 * Fused MoE router: hard-masked softmax and the top-k kept mask of its output in
 * one pass.  [P3] hard-masked softmax followed by [P3] kept mask (Spec.MoE.kept)
 * on the probabilities.
 *   p = rowops_masked_softmax(x, mask);  kept = rowops_topk_kept(p, k)
 * computed together: p is stored and the mask is decided on the same fp32
 * values, so both outputs equal the two separate calls bit for bit, while p is
 * never read back (13 instead of 17 bytes of HBM traffic per element).
 * x, p, kept: rows x cols fp32; mask: rows x cols bytes.  p may be exactly x;
 * kept must not overlap x, mask or p.  1 <= k <= cols, else ROWOPS_ERR_SHAPE.
 */
int rowops_router_masked_topk(const float *x, const uint8_t *mask, float *p, float *kept,
                              int64_t rows, int64_t cols, int64_t k, rowops_stream stream);

/*
 * Per-row top k values and their columns.  [P1] top_k_rows(in, values, indices,
 * rows, cols, k, largest).
 *   values[i][r], indices[i][r]: the entry of row i ranked r (0-based) among the
 *   k largest (largest != 0) or smallest, its column as a whole-number float.
 * Rank order: NaN ranks above every number (first for largest, last for
 * smallest); equal values (NaNs among themselves, -0 with +0) keep the lower
 * column first.  The output values are the input's bits (sign of zero and NaN
 * payload kept).  x: rows x cols; values, indices: rows x k.  Requires
 * 1 <= k <= cols <= 2^24 ([P1] precondition), else ROWOPS_ERR_SHAPE.  Outputs
 * must not overlap x or each other.  Exact (selection only).
 */
int rowops_top_k_rows(const float *x, float *values, float *indices, int64_t rows, int64_t cols,
                      int64_t k, int largest, rowops_stream stream);

/*
 * RMSNorm forward.  [P1] rms_norm_forward(in, gamma, out, row_rms, rows, cols, eps).
 *   rms_i = sqrt(mean_j x_ij^2 + eps),  out_ij = gamma_j * x_ij / rms_i,
 *   row_rms_i = rms_i (the cached statistic).
 * x, out: rows x cols; gamma: cols; row_rms: rows.  cols == 0, eps < 0 or
 * non-finite eps are ROWOPS_ERR_SHAPE.  Outputs must not overlap inputs or each
 * other.
 */
int rowops_rmsnorm_fwd(const float *x, const float *gamma, float *out, float *row_rms, int64_t rows,
                       int64_t cols, float eps, rowops_stream stream);

/*
 * RMSNorm backward.  [P1] rms_norm_backward(grad_out, gamma, in, row_rms,
 * grad_in, gamma_terms, rows, cols).
 *   g'_ij = dy_ij * gamma_j,  dx_ij = (g'_ij - x_ij * mean_k(g'_ik x_ik) / rms_i^2) / rms_i,
 *   gamma_terms_ij = dy_ij * x_ij / rms_i
 * (gamma's gradient is rowops_column_sums(gamma_terms), as [P1] intends).
 * dy, x, dx, gamma_terms: rows x cols; gamma: cols; row_rms: rows.  cols == 0 is
 * ROWOPS_ERR_SHAPE.  Outputs must not overlap inputs or each other.
 */
int rowops_rmsnorm_bwd(const float *dy, const float *gamma, const float *x, const float *row_rms,
                       float *dx, float *gamma_terms, int64_t rows, int64_t cols,
                       rowops_stream stream);

/*
 * Column sums.  [P1] column_sums(in, out, rows, cols, beta).
 *   out_j = beta * out_j + sum_i in_ij;  beta == 0 does not read out.
 * in: rows x cols; out: cols.  Deterministic: fixed blocks of consecutive rows
 * are added in row order, then the blocks in block order (no workspace: a
 * thread-block cluster per 32-column tile).  Exception to the common contract:
 * rows == 0 still applies beta.  Non-finite beta is ROWOPS_ERR_SHAPE; out must not
 * overlap in ([P1]).
 */
int rowops_column_sums(const float *in, float *out, int64_t rows, int64_t cols, float beta,
                       rowops_stream stream);

/*
 * Hard-masked softmax with a floating-point mask.  [P3] hard-masked softmax: an
 * entry is allowed when its mask value is not zero (mask != 0.0f: -0.0 blocks,
 * NaN allows); otherwise exactly rowops_masked_softmax.  mask: rows x cols fp32.
 * y may be exactly x; any other overlap is ROWOPS_ERR_ALIAS.
 */
int rowops_masked_softmax_fmask(const float *x, const float *mask, float *y, int64_t rows,
                                int64_t cols, rowops_stream stream);

/*
 * Softmax relevance rule.  [P1] lrp_softmax_rows(x, y, r, r_in, rows, cols):
 *   r_in_ij = x_ij * (r_ij - y_ij * sum_k r_ik).
 * x, y, r, r_in: rows x cols (y is the softmax output).  r_in must not overlap the
 * inputs.  cols == 0 is a no-op.
 */
int rowops_lrp_softmax_rows(const float *x, const float *y, const float *r, float *r_in,
                            int64_t rows, int64_t cols, rowops_stream stream);

/*
 * First-max one-hot.  [P3]: 1.0f at the first maximal coordinate of each
 * nonempty row and 0.0f elsewhere (the input dtype).  A coordinate is maximal
 * when no entry is larger than it, so a NaN is maximal and, without NaN, this is
 * the first index of the maximum.  x, out: rows x cols; out must not overlap x.
 * cols == 0 is a no-op (empty rows give an empty result).
 */
int rowops_argmax_onehot(const float *x, float *out, int64_t rows, int64_t cols,
                         rowops_stream stream);

/*
 * Weighted-logits (soft-target) cross-entropy.  [P3] mean weighted-logits
 * cross-entropy, read as cross-entropy against a weight row, with every
 * log-probability taken from the original logits (x - lse) so that a weighted
 * term whose probability underflows stays finite:
 *   loss_i = sum_j w_ij (lse_i - x_ij),  *mean_loss = (1/rows) sum_i loss_i,
 *   grad_ij = grad_scale * (softmax(x_i)_j * sum_k w_ik - w_ij).
 * A one-hot w gives rowops_softmax_ce.  logits, weights, grad: rows x cols;
 * row_loss: rows; mean_loss: one device double.  cols == 0 or non-finite
 * grad_scale is ROWOPS_ERR_SHAPE; outputs must not overlap inputs or each other.
 */
int rowops_soft_ce(const float *logits, const float *weights, float *grad, float *row_loss,
                   double *mean_loss, int64_t rows, int64_t cols, float grad_scale,
                   rowops_stream stream);

/*
 * Fixed-teacher cross-entropy and the student gradient.  [P3] fixed-teacher mean
 * cross-entropy, or its student gradient: q = softmax(teacher) is a constant,
 *   loss_i = sum_j q_ij (lse(student)_i - student_ij),  mean over rows,
 *   grad_ij = grad_scale * (softmax(student_i)_j - q_ij)   (written when grad != NULL).
 * Shapes and rules as rowops_soft_ce; grad may be NULL (loss only).
 */
int rowops_teacher_ce(const float *student, const float *teacher, float *grad, float *row_loss,
                      double *mean_loss, int64_t rows, int64_t cols, float grad_scale,
                      rowops_stream stream);

/*
 * The mixture-of-experts layer behind the router: the plan that groups
 * (token, choice) pairs by expert, the rows moved to their experts and back,
 * and the experts' matrix products.  The pages have no counterpart; these
 * entry points take what rowops_top_k_rows and rowops_router_masked_topk
 * answer.  Beyond the common contract:
 *   - Matrices marked `void` hold the element type that their rowops_dtype
 *     argument names.  An argument that names no type, or one that the entry
 *     point does not take, is ROWOPS_ERR_SHAPE.  Sums are fp32; each result is
 *     rounded once, to nearest even.
 *   - `slots` (rows of a matrix grouped by expert) and rows * k are at most
 *     2^30, experts is 1..1024 and k at least 1, else ROWOPS_ERR_SHAPE.
 *   - offsets, slot and indices are device data that no host check sees.  Their
 *     use is checked on the device: a slot outside [0, slots) is skipped, and
 *     offsets are clamped to 0..slots with no group ending before it starts.
 *     Results do not depend on rows that no group or slot names (the products may
 *     read them), and output rows that none names are left as they were.
 */
typedef enum {
    ROWOPS_F32 = 0,
    ROWOPS_F16 = 1,
    ROWOPS_BF16 = 2,
    ROWOPS_E4M3 = 3, /* with one scale for each 128 columns: answers only */
    ROWOPS_E2M1 = 4  /* with a power of two for each 32 columns: answers only */
} rowops_dtype;

/* Bytes of device workspace rowops_expert_plan needs (a function of the sizes
 * and the current device's SM count; 0 for up to 2048 pairs and for sizes that
 * the call refuses). */
size_t rowops_expert_plan_workspace(int64_t rows, int64_t k, int64_t experts);

/*
 * Plan of a routed batch: the pairs p = t * k + j (token t, choice j) sorted by
 * expert, in the order of p within an expert.
 *   e_p = trunc(indices_p); pair p takes part when 0 <= indices_p < experts and
 *         values is NULL or values_p != 0 (NaN takes part)
 *   offsets_e = number of pairs of the experts before e  (offsets[experts]: all)
 *   slot_p  = the pair's rank in the sorted order, -1 for a pair left out
 *   order_s = the pair at rank s, -1 for s >= offsets[experts]
 * indices, values: rows x k fp32 as rowops_top_k_rows writes them on
 * probabilities (a masked expert has probability +0.0, so a token whose mask
 * leaves fewer than k experts, or none, loses those pairs); offsets: experts + 1;
 * order, slot: rows * k.  rows == 0 writes offsets (all 0).  `workspace` holds at
 * least rowops_expert_plan_workspace(...) bytes, 16-byte aligned; concurrent
 * calls need separate workspaces.  No output may overlap another buffer.
 */
int rowops_expert_plan(const float *indices, const float *values, int32_t *offsets, int32_t *order,
                       int32_t *slot, int64_t rows, int64_t k, int64_t experts, void *workspace,
                       size_t workspace_bytes, rowops_stream stream);

/*
 * Token rows to their experts' slots: out[slot[t][j]] = x[t], rounded to
 * out_type.  x: rows x cols of x_type; slot: rows x k; out: slots x cols.  No plan
 * names a slot twice; where the caller's does, each value of that row of out is of
 * one of the rows, which one may differ from value to value and from call to call.
 * The gradient is rowops_expert_combine of the slots' gradients with weights NULL.
 * cols == 0 is a no-op.
 */
int rowops_expert_gather(const void *x, const int32_t *slot, void *out, int64_t rows, int64_t k,
                         int64_t cols, int64_t slots, int x_type, int out_type,
                         rowops_stream stream);

/*
 * Expert rows back to their tokens: out[t] = sum_j w[t][j] * y[slot[t][j]], the
 * choices in order, skipped slots adding nothing; a token with none is all +0.0.
 * y: slots x cols of y_type; slot, weights: rows x k (weights NULL: all 1);
 * out: rows x cols of out_type.  cols == 0 is a no-op.
 */
int rowops_expert_combine(const void *y, const int32_t *slot, const float *weights, void *out,
                          int64_t rows, int64_t k, int64_t cols, int64_t slots, int y_type,
                          int out_type, rowops_stream stream);

/*
 * Backward of rowops_expert_combine.
 *   dy[slot[t][j]] = w[t][j] * dout[t]
 *   dweights[t][j] = sum_c dout[t][c] * y[slot[t][j]][c]   (0 for a skipped slot)
 * dout: rows x cols of out_type; y, dy: slots x cols of y_type; slot, weights,
 * dweights: rows x k.  A row of dy that two pairs name holds, value by value, one of
 * theirs and not their sum, as for rowops_expert_gather.  cols == 0 writes dweights
 * (all 0).
 */
int rowops_expert_combine_bwd(const void *dout, const void *y, const int32_t *slot,
                              const float *weights, void *dy, float *dweights, int64_t rows,
                              int64_t k, int64_t cols, int64_t slots, int out_type, int y_type,
                              rowops_stream stream);

/*
 * Matrix product of each expert's rows with its weights.
 *   y[s][n] = sum_k x[s][k] * w[e][n][k]     for offsets[e] <= s < offsets[e + 1]
 *             (transposed != 0: w[e][k][n])
 * x: slots x in_cols; w: experts x out_cols x in_cols (transposed: experts x
 * in_cols x out_cols); y: slots x out_cols; all of `dtype`, ROWOPS_F16 or
 * ROWOPS_BF16.  offsets: experts + 1, or NULL with experts == 1 for one dense
 * product.  The gradient with respect to x is the same call on dy with the
 * other `transposed`.  in_cols == 0 or out_cols == 0 is ROWOPS_ERR_SHAPE.
 * The tensor cores' kernel reads matrices whose first value and rows lie on
 * 16-byte boundaries.  For others give a workspace: they are copied there first
 * (rowops_expert_matmul_workspace(...) bytes cover row widths that are no multiple
 * of 8 values, and are 0 where all are; a matrix with whole rows that starts off a
 * 16-byte boundary needs its own bytes and 512 more on top).  Without one, or with
 * too little, a slower kernel takes them as they are (6 to 16 times), so NULL and 0
 * are always allowed; a workspace that is not 16-byte aligned is
 * ROWOPS_ERR_WORKSPACE.  Concurrent calls need separate workspaces.
 * Waits of the pipelined kernel are bounded: one that runs out (a defect) leaves
 * y incomplete and counts one timeout, see rowops_pipeline_timeouts().
 */
size_t rowops_expert_matmul_workspace(int64_t slots, int64_t in_cols, int64_t out_cols,
                                      int64_t experts, int transposed);
int rowops_expert_matmul(const void *x, const void *w, const int32_t *offsets, void *y,
                         int64_t slots, int64_t in_cols, int64_t out_cols, int64_t experts,
                         int transposed, int dtype, void *workspace, size_t workspace_bytes,
                         rowops_stream stream);

/*
 * Gradient of rowops_expert_matmul with respect to the weights.
 *   dw[e][n][k] = sum_{s of expert e} dy[s][n] * x[s][k]   (overwritten; an
 *   expert without rows gets zeros)
 * dy: slots x out_cols; x: slots x in_cols; both of `dtype` (ROWOPS_F16 or
 * ROWOPS_BF16); dw: experts x out_cols x in_cols of `dw_type`, which is `dtype`
 * or ROWOPS_F32.  For transposed weights swap dy and x (and their widths).
 * slots == 0 writes zeros.  Workspace and timeouts as for rowops_expert_matmul.
 */
size_t rowops_expert_matmul_wgrad_workspace(int64_t slots, int64_t in_cols, int64_t out_cols);
int rowops_expert_matmul_wgrad(const void *dy, const void *x, const int32_t *offsets, void *dw,
                               int64_t slots, int64_t in_cols, int64_t out_cols, int64_t experts,
                               int dtype, int dw_type, void *workspace, size_t workspace_bytes,
                               rowops_stream stream);

/*
 * Quantises to e4m3 (four exponent bits, no infinity, largest value 448) with
 * one scale for each block of 128 columns of a row (block_rows == 1) or of 128
 * rows by 128 columns (block_rows == 128); the last blocks may be smaller.
 *   a = max(max |x| over the block's finite x, 2^-100)
 *   scale = a / 448,  q = e4m3(448 * x / a)      (ties to even)
 * so that x is about q * scale.  An infinite or NaN x becomes e4m3 NaN.
 * x: batches x rows x cols of x_type; q: the same shape, one byte a value;
 * scale: batches x ceil(rows / block_rows) x ceil(cols / 128).  Blocks do not
 * cross matrices.  Any other block_rows is ROWOPS_ERR_SHAPE; cols == 0 is a no-op.
 */
int rowops_quantize_blocks(const void *x, uint8_t *q, float *scale, int64_t batches, int64_t rows,
                           int64_t cols, int64_t block_rows, int x_type, rowops_stream stream);

/*
 * rowops_expert_matmul (not transposed) on e4m3 operands with a scale for each
 * block of 128.
 *   y[s][n] = sum_b xs[s][b] * ws[e][n / 128][b] * sum_{k in block b} xq[s][k] * wq[e][n][k]
 * xq: slots x in_cols with xs: slots x ceil(in_cols / 128); wq: experts x
 * out_cols x in_cols with ws: experts x ceil(out_cols / 128) x ceil(in_cols / 128),
 * as rowops_quantize_blocks writes them with block_rows 1 and 128; y: slots x
 * out_cols of y_type.  offsets, workspace (for in_cols that are no multiple of 16)
 * and timeouts as for rowops_expert_matmul.
 * A block's two scales are multiplied first, in fp32: where their product leaves the
 * range of normal numbers (2^-126 .. 2^128) it loses bits or becomes 0 or infinite,
 * and y with it.
 * The gradient with respect to x is this call on dy, quantised by rows, with the
 * bytes of wq and the scales ws transposed within each expert (blocks of 128 x 128
 * stay blocks, so nothing is quantised again).  The gradient with respect to the
 * weights sums over rows, across which these scales differ: take
 * rowops_expert_matmul_wgrad on fp16 or bf16 rows.
 */
size_t rowops_expert_matmul_fp8_workspace(int64_t slots, int64_t in_cols, int64_t out_cols,
                                          int64_t experts);
int rowops_expert_matmul_fp8(const uint8_t *xq, const float *xs, const uint8_t *wq,
                             const float *ws, const int32_t *offsets, void *y, int64_t slots,
                             int64_t in_cols, int64_t out_cols, int64_t experts, int y_type,
                             void *workspace, size_t workspace_bytes, rowops_stream stream);

/*
 * Quantises to microscaled 4-bit values (OCP Microscaling Formats 1.0, MXFP4):
 * e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with a power of two for each
 * block of 32 columns of a row; the last block may be smaller.
 *   e = max(floor(log2(max |x| over the block)) - 2, -127)
 *   scale = e + 127 (one byte),  q = e2m1(x / 2^e)   (ties to even, at most 6)
 * so that x is about q * 2^(scale - 127).  A block with an infinite or NaN x has
 * scale 255, which stands for NaN, and q = 0.
 * x: rows x cols of x_type; q: rows x ceil(cols / 2) bytes, the lower column in the
 * lower four bits, and 0 in the upper bits behind an odd row's end; scale: rows x
 * ceil(cols / 32) bytes.  cols > 2^31 - 257 is ROWOPS_ERR_SHAPE; cols == 0 is a no-op.
 */
int rowops_quantize_mx4(const void *x, uint8_t *q, uint8_t *scale, int64_t rows, int64_t cols,
                        int x_type, rowops_stream stream);

/*
 * rowops_expert_matmul (not transposed) on microscaled 4-bit operands.
 *   y[s][n] = sum_b 2^(xs[s][b] + ws[e][n][b] - 254) * sum_{k in block b} xq[s][k] * wq[e][n][k]
 * with blocks of 32; a scale of 255 makes its products NaN.  xq: slots x in_cols / 2
 * bytes with xs: slots x ceil(in_cols / 32); wq: experts x out_cols x in_cols / 2 with
 * ws: experts x out_cols x ceil(in_cols / 32), as rowops_quantize_mx4 writes them; y:
 * slots x out_cols of y_type.  in_cols is even (else ROWOPS_ERR_SHAPE): an odd row
 * counts the four bits behind its end, which are 0.  offsets, workspace (for in_cols
 * that are no multiple of 32) and timeouts as for rowops_expert_matmul.
 * The gradient with respect to x is this call on dy, quantised by rows, with the
 * weights transposed within each expert and quantised from their own values (blocks
 * run along the sum, so these bytes cannot be transposed): in_cols is then out_cols,
 * or out_cols + 1 where that is odd, for both operands' rows end in four bits of 0, and
 * out_cols is in_cols.  The gradient with respect to the weights is
 * rowops_expert_matmul_wgrad on fp16 or bf16 rows.
 */
size_t rowops_expert_matmul_mx4_workspace(int64_t slots, int64_t in_cols, int64_t out_cols,
                                          int64_t experts);
int rowops_expert_matmul_mx4(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                             const uint8_t *ws, const int32_t *offsets, void *y, int64_t slots,
                             int64_t in_cols, int64_t out_cols, int64_t experts, int y_type,
                             void *workspace, size_t workspace_bytes, rowops_stream stream);

/*
 * Between two sublayers' products: dropout, the residual's addition and its
 * root-mean-square norm.  The pages have no counterpart beyond rms_norm_forward and
 * rms_norm_backward.  `void` matrices, types and roundings as for the expert
 * operators; cols > 2^31 - 257 is ROWOPS_ERR_SHAPE.
 *
 * Dropout drops with probability p, 0 <= p <= 1 (else ROWOPS_ERR_SHAPE), rounded to
 * t / 65536, and multiplies what stays by 65536 / (65536 - t) (p == 1: nothing stays).
 * What drops is +0.0, whatever it was.  The mask is not stored: value (i, c) drops
 * when u < t, where u is the 16-bit half c mod 8 (the lower half of a word first) of
 * the 128 bits that Philox4x32-10 gives for the key rng[0] and the counter (block,
 * rng[1]), both low word first, and block = i * ceil(cols / 8) + c / 8.  So the same
 * rng, rows and cols give the same mask.  rng: two 64-bit numbers in device memory,
 * 8-byte aligned, read when the call runs: a captured graph whose replays shall drop
 * anew advances rng[1] in the graph.  rng may be NULL where t is 0 or 65536.
 */

/*
 * y = residual + drop(x).  x: rows x cols of x_type; residual (NULL: none) and y:
 * rows x cols of y_type, any two types.  The gradient with respect to x is this call
 * on dy without a residual; that of the residual is dy.  y may be exactly residual, or
 * exactly x where the types are the same; any other overlap is ROWOPS_ERR_ALIAS.
 * cols == 0 is a no-op.
 */
int rowops_dropout(const void *x, const void *residual, const uint64_t *rng, void *y, int64_t rows,
                   int64_t cols, float p, int x_type, int y_type, rowops_stream stream);

/*
 * Residual addition and RMSNorm.
 *   h = residual + drop(x),  rms_i = sqrt(mean_j h_ij^2 + eps),  y_ij = gamma_j * h_ij / rms_i
 * x: rows x cols of x_type; residual (NULL: none) and h (NULL: not wanted): rows x cols
 * of h_type, which is x_type or ROWOPS_F32; gamma: cols fp32; row_rms (NULL: not
 * wanted): rows fp32.  The norm is of the sum before it is rounded to h_type.
 * out holds y, rows x cols, by out_type:
 *   x_type        y; scale is not used
 *   ROWOPS_E4M3   as rowops_quantize_blocks with block_rows 1 writes it, the scales
 *                 (fp32, rows x ceil(cols / 128)) in scale
 *   ROWOPS_E2M1   as rowops_quantize_mx4 writes it, the scales (bytes, rows x
 *                 ceil(cols / 32)) in scale
 * so that the quantised rows are operands of rowops_expert_matmul_fp8 and
 * rowops_expert_matmul_mx4.  h may be exactly residual; any other overlap of an
 * output is ROWOPS_ERR_ALIAS.  cols == 0, eps < 0 and non-finite eps are
 * ROWOPS_ERR_SHAPE.
 */
int rowops_add_rmsnorm_fwd(const void *x, const void *residual, const float *gamma,
                           const uint64_t *rng, void *h, void *out, void *scale, float *row_rms,
                           int64_t rows, int64_t cols, float eps, float p, int x_type, int h_type,
                           int out_type, rowops_stream stream);

/* Bytes of device workspace rowops_add_rmsnorm_bwd needs (a function of the sizes and
 * the current device's SM count; 0 for sizes that need none or that it refuses). */
size_t rowops_add_rmsnorm_bwd_workspace(int64_t rows, int64_t cols);

/*
 * Backward of rowops_add_rmsnorm_fwd (of y itself, whatever it was quantised to).
 *   n = h / rms,  g = dy * gamma,  t = dh + (g - n * mean_j(g_j n_j)) / rms
 *   dresidual = t,  dx = drop(t),  dgamma_j = sum_i dy_ij n_ij   (overwritten)
 * dy, dx: rows x cols of x_type; h, dh, dresidual: rows x cols of h_type; gamma,
 * dgamma: cols; row_rms: rows.  dh is the gradient that arrives at h from elsewhere
 * (the residual stream; NULL: none).  dresidual and dx may be NULL where they are not
 * wanted, and rng without dx; without dropout and with one type they are the same
 * values.  dresidual may
 * be exactly dh, and dx exactly dy; any other overlap of an output is
 * ROWOPS_ERR_ALIAS.  Rows of 8193 to 65536 values share a cluster, whose waits are
 * bounded as rowops_pipeline_timeouts says.  dgamma is summed in a fixed order, through `workspace`: at least
 * rowops_add_rmsnorm_bwd_workspace(rows, cols) bytes, 16-byte aligned, with
 * concurrent calls in separate ones.  cols == 0 is ROWOPS_ERR_SHAPE; rows == 0 writes
 * zeros to dgamma.
 */
int rowops_add_rmsnorm_bwd(const void *dy, const float *gamma, const void *h, const float *row_rms,
                           const void *dh, const uint64_t *rng, void *dresidual, void *dx,
                           float *dgamma, int64_t rows, int64_t cols, float p, int x_type,
                           int h_type, void *workspace, size_t workspace_bytes,
                           rowops_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* ROWOPS_H */
