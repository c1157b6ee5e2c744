/*
 * adamw.h -- C ABI of the AdamW step over many tensors at once on GB300
 * (sm_103a), in the same library as linear_logp.h.
 *
 * For every element, with t = step (+ *device_step), rate = lr (* *device_lr) and
 * g = grad (* *grad_scale):
 *
 *     m = beta1 m + (1 - beta1) g
 *     v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - rate decay) - rate / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * in fp32, from the fp32 master copy where there is one (which is then updated,
 * and the parameter is its rounding), else from the parameter itself.
 * Decay and update are summed and subtracted from the parameter in one rounding, so
 * that a small rate times decay keeps its digits.
 *
 * States in 32 bits are fp32.  States in 8 bits are e4m3 values (one sign, four
 * exponent and three fraction bits) times a scale that ADAMW_BLOCK consecutive
 * elements of a tensor share: m, and the root of v, whose range is half as many
 * binades.  The step computes with the fp32 values and stores
 *
 *     scale = max |m| * (1 / 448),   code = e4m3(m / scale)         (all 0 where max |m| is 0)
 *
 * and the same of sqrt(v), of which no value above 0 is stored as 0: at an element
 * whose gradients are far below its block's largest, a step divides by no less than
 * the smallest code (2^-9 scale).  The moments and the scales are rounded operation
 * by operation, so that the codes are those of the formulas in fp32, next to the
 * border between two codes too.  A gradient that is not finite spoils its
 * element, in 8 bits its block.
 *
 * Conventions as in linear_logp.h: device pointers in host arrays of `count`
 * entries, read before the call returns; work enqueued on `stream`, arguments
 * checked before anything is enqueued, the same LLP_* status codes.  Parameters are
 * bf16 (0), fp32 (1) or fp16 (2), gradients of the same type or fp32, each tensor
 * its own.  Element alignment suffices; tensors whose arrays reach a 16-byte
 * boundary at the same element move fastest.  No tensor may be listed twice or
 * overlap another.  Results do not depend on how tensors are listed, and are
 * bitwise the same in every run.
 */
#ifndef ADAMW_H_
#define ADAMW_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ADAMW_BLOCK 256

/* One step.  Entry i is a tensor of sizes[i] elements (0 is skipped).
 * state_bits: 32 (exp_avg, exp_avg_sq fp32; the scale arrays NULL) or 8 (codes, with
 * exp_avg_scale[i], exp_avg_sq_scale[i] fp32 of ceil(sizes[i] / ADAMW_BLOCK)).
 * masters: NULL, or fp32 arrays, NULL entries without one.  weight_decay: one per
 * tensor.  0 <= beta1, beta2 < 1; eps, lr, weight_decay finite, eps >= 0.  step >= 1,
 * or step >= 0 beside device_step (int64 on the device; the sum counts from 1);
 * device_lr and grad_scale
 * (fp32 on the device) may be NULL.  The three are read when the kernel runs, so that
 * a captured graph can advance them. */
int adamw_step(int64_t count, void* const* params, const void* const* grads, void* const* exp_avg,
               void* const* exp_avg_sq, float* const* exp_avg_scale, float* const* exp_avg_sq_scale,
               float* const* masters, const int64_t* sizes, const int32_t* param_dtypes, const int32_t* grad_dtypes,
               const double* weight_decay, int state_bits, double lr, double beta1, double beta2, double eps,
               int64_t step, const int64_t* device_step, const float* device_lr, const float* grad_scale,
               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_H_ */
