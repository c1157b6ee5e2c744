/*
 * gated_linear.h -- C ABI of the gated linear layer, the first half of a gated
 * feed-forward block, on GB300 (sm_103a), in the same library as linear_logp.h.
 *
 *     gate[n, f] = sum_d x[n, d] * w_gate[f, d],   up[n, f] = sum_d x[n, d] * w_up[f, d]
 *     y[n, f]    = act(gate[n, f]) * up[n, f]
 *
 * and, from the projections that the forward kept,
 *
 *     dG = grad_y * up * act'(gate),   dU = grad_y * act(gate)
 *     grad_x = dG . w_gate + dU . w_up,   grad_w_gate = dG^T . x,   grad_w_up = dU^T . x
 *
 * act: 0 silu z / (1 + exp(-z)); 1 gelu z Phi(z), Phi the normal distribution
 * function; 2 its tanh form z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2.
 *
 * All sums are fp32 on the tensor cores; y is formed from the fp32 projections
 * and rounded once.  The kept projections, dG and dU (the backward's matrix
 * operands) are rounded to the tensors' type.  Every sum runs in an order that
 * depends on the sizes alone, so results are bitwise the same in every run.
 *
 * Conventions as in linear_logp.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, arguments checked before anything is enqueued, the
 * same LLP_* status codes.  All tensors are bf16 (dtype 0) or fp16 (dtype 2),
 * contiguous and 16-byte aligned.  D and F are multiples of 8; N < 2^31,
 * D, F < 2^30.
 */
#ifndef GATED_LINEAR_H_
#define GATED_LINEAR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GATED_LINEAR_SILU 0
#define GATED_LINEAR_GELU 1
#define GATED_LINEAR_GELU_TANH 2

/* Forward.  x [N, D]; w_gate, w_up [F, D]; y [N, F]; pre [2, N, F] receives gate
 * and up for the backward, or is NULL.  N == 0 is a no-op. */
int gated_linear_fwd(const void* x, const void* w_gate, const void* w_up, int dtype, int act, int64_t N, int64_t D,
                     int64_t F, void* y, void* pre, void* stream);

/* Bytes of workspace gated_linear_bwd needs (0 when N == 0 or a size is invalid). */
size_t gated_linear_bwd_workspace_bytes(int64_t N, int64_t D, int64_t F);

/* Backward.  grad_y [N, F], pre of the forward; grad_x [N, D], grad_w_gate and
 * grad_w_up [F, D] may each be NULL to skip it; those given are overwritten.
 * N == 0 writes zeros into the weights' gradients.  The workspace needs no
 * clearing and must be 16-byte aligned. */
int gated_linear_bwd(const void* grad_y, const void* pre, const void* x, const void* w_gate, const void* w_up,
                     int dtype, int act, int64_t N, int64_t D, int64_t F, void* grad_x, void* grad_w_gate,
                     void* grad_w_up, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GATED_LINEAR_H_ */
