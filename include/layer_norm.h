/*
 * layer_norm.h -- C ABI of layer norm over the last dimension on GB300
 * (sm_103a), in the same library as linear_logp.h.
 *
 *     mean[n] = sum_d x[n, d] / D
 *     rstd[n] = 1 / sqrt(sum_d (x[n, d] - mean[n])^2 / D + eps)
 *     h[n, d] = (x[n, d] - mean[n]) * rstd[n]
 *     y[n, d] = h[n, d] * weight[d] + bias[d]
 *
 * and, with a = grad_y * weight,
 *
 *     grad_x[n, :]   = rstd[n] * (a - sum_d a / D - h * (sum_d a h) / D)
 *     grad_weight[d] = sum_n grad_y[n, d] * h[n, d]
 *     grad_bias[d]   = sum_n grad_y[n, d]
 *
 * Sums and statistics are fp32 (the variance from the centred values), each
 * output is rounded once.  The order of a row's sums depends on D and the types
 * alone, so y, mean, rstd and grad_x rows are bitwise the same for any batch,
 * layout and run; the order of grad_weight / grad_bias's sums depends on N, D
 * and the types, so they are bitwise the same in every run.
 *
 * Conventions as in linear_logp.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, arguments checked before anything is enqueued, the
 * same LLP_* status codes.  x, grad_y, y and grad_x are bf16 (dtype 0), fp32
 * (dtype 1) or fp16 (dtype 2); weight, bias and their gradients have
 * param_dtype: the same as dtype, or fp32.  weight and bias may each be NULL
 * (1 and 0).  The rows of x and grad_y start row_stride elements apart (D when
 * contiguous; 0 repeats one row); outputs are contiguous.  Element alignment
 * suffices; 16-byte aligned rows move fastest.  N < 2^31, 1 <= D < 2^22.
 */
#ifndef LAYER_NORM_H_
#define LAYER_NORM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LAYER_NORM_DTYPE_BF16 0
#define LAYER_NORM_DTYPE_F32 1
#define LAYER_NORM_DTYPE_F16 2

/* Forward.  y [N, D]; mean, rstd fp32 [N] (all required, overwritten); eps >= 0
 * and finite.  N == 0 is a no-op. */
int layer_norm_fwd(const void* x, int64_t x_row_stride, int dtype, int64_t N, int64_t D, const void* weight,
                   const void* bias, int param_dtype, float eps, void* y, float* mean, float* rstd, void* stream);

/* Bytes of workspace layer_norm_bwd needs when grad_weight or grad_bias is
 * asked for (0 when N == 0 or a size is invalid); enough for any choice. */
size_t layer_norm_bwd_workspace_bytes(int64_t N, int64_t D);

/* Backward, with mean and rstd of the forward on the same x.  grad_x [N, D],
 * grad_weight [D] and grad_bias [D] may each be NULL to skip it; those given are
 * overwritten.  N == 0 writes zeros into grad_weight and grad_bias.  The
 * workspace needs no clearing, must be 16-byte aligned, and may be NULL when
 * only grad_x is asked for. */
int layer_norm_bwd(const void* grad_y, int64_t grad_y_row_stride, const void* x, int64_t x_row_stride, int dtype,
                   int64_t N, int64_t D, const float* mean, const float* rstd, const void* weight, int param_dtype,
                   void* grad_x, void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                   void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYER_NORM_H_ */
