/*
 * residual_rms_norm.h -- C ABI of the RMS norms before and after a model's block,
 * with the block's gate and residual scale, on GB300 (sm_103a), in the same
 * library as linear_logp.h.
 *
 * The end of one block and the start of the next, in one pass over the rows.  With
 * b the block's output, x the residual stream before it:
 *
 *     post_rstd[n] = 1 / sqrt(sum_d b[n, d]^2 / D + eps)
 *     m[n, d]      = b[n, d] * post_rstd[n] * post_weight[d]      (b without post_weight)
 *     s[n, d]      = x[n, d] + scale * gate[n, d] * m[n, d]       (x without a branch)
 *     rstd[n]      = 1 / sqrt(sum_d s[n, d]^2 / D + eps)
 *     h[n, d]      = s[n, d] * rstd[n] * weight[d]                (only with weight)
 *
 * gate is one value per column ([D]), one per element ([N, D]), or left out (1).
 * Without a branch this is the plain RMS norm of x.  The gradient, from s, with
 * c = s * rstd and a = grad_h * weight:
 *
 *     G             = grad_s + rstd * (a - c * sum_d(a c) / D)        = grad_x
 *     grad_weight   = sum_n grad_h * c
 *     grad_gate     = scale * G * m           (summed over n where gate is [D])
 *     e             = scale * gate * G,   k = b * post_rstd
 *     grad_post_weight = sum_n e * k
 *     grad_b        = post_rstd * (e post_weight - k * sum_d(e post_weight k) / D)
 *                     (e without post_weight)
 *
 * Sums and statistics are fp32, every output is rounded once; h and rstd come from
 * the unrounded s, the gradient from the s it is given.  The order of a row's sums
 * depends on D, the types and the gate's kind alone, the order of the sums over rows on these and
 * N: rows are bitwise the same for any batch, and all results in every run.
 *
 * Conventions as in linear_logp.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, arguments checked before anything is enqueued, the same
 * LLP_* status codes.  Rows and their gradients are bf16 (dtype 0), fp32 (dtype 1)
 * or fp16 (dtype 2); weight, post_weight, a gate per column and their gradients
 * have param_dtype: the same as dtype, or fp32.  Input rows start row_stride
 * elements apart (D when contiguous; 0 repeats one row); outputs are contiguous.
 * Element alignment suffices; 16-byte aligned rows move fastest.  N < 2^31,
 * 1 <= D < 2^22.
 */
#ifndef RESIDUAL_RMS_NORM_H_
#define RESIDUAL_RMS_NORM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RESIDUAL_RMS_NORM_GATE_NONE 0
#define RESIDUAL_RMS_NORM_GATE_COLUMNS 1
#define RESIDUAL_RMS_NORM_GATE_ROWS 2

/* Forward.  branch, post_weight and weight may be NULL as above; gate_kind NONE
 * goes with a NULL gate.  s [N, D] is required with a branch and must be NULL
 * without one; h [N, D] and rstd [N] go with weight, post_rstd [N] with
 * post_weight (NULL otherwise).  Outputs overlap no input.  N == 0 is a no-op. */
int residual_rms_norm_fwd(const void* x, int64_t x_row_stride, const void* branch, int64_t branch_row_stride,
                          const void* gate, int64_t gate_row_stride, int gate_kind, const void* post_weight,
                          const void* weight, int dtype, int param_dtype, int64_t N, int64_t D, float scale, float eps,
                          void* s, void* h, float* post_rstd, float* rstd, void* stream);

/* Bytes of workspace residual_rms_norm_bwd needs (0 when N == 0 or a size is
 * invalid); enough for any choice. */
size_t residual_rms_norm_bwd_workspace_bytes(int64_t N, int64_t D);

/* Backward.  s is the forward's (x itself without a branch).  grad_s may be NULL (no
 * gradient comes from the stream); grad_h and rstd go with weight.  grad_x, grad_b
 * [N, D], grad_gate ([D] or [N, D]), grad_post_weight and grad_weight [D] may each
 * be NULL to skip it; those given are overwritten.  N == 0 writes zeros into the
 * [D] gradients.  The workspace needs no clearing and must be 16-byte aligned. */
int residual_rms_norm_bwd(const void* grad_s, int64_t grad_s_row_stride, const void* grad_h, int64_t grad_h_row_stride,
                          const void* s, int64_t s_row_stride, const void* branch, int64_t branch_row_stride,
                          const void* gate, int64_t gate_row_stride, int gate_kind, const void* post_weight,
                          const void* weight, const float* post_rstd, const float* rstd, int dtype, int param_dtype,
                          int64_t N, int64_t D, float scale, void* grad_x, void* grad_b, void* grad_gate,
                          void* grad_post_weight, void* grad_weight, void* workspace, size_t workspace_bytes,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RESIDUAL_RMS_NORM_H_ */
