/*
 * dropout.h -- C ABI of dropout from a counter-based generator on GB300
 * (sm_103a), in the same library as linear_logp.h.  The mask is never stored:
 * forward and backward draw it again from (seed, offset, element index).
 *
 *     T    = floor(p * 65536 + 1/2)
 *     y[e] = (r(e) >= T ? x[e] * 65536 / (65536 - T) : 0) + residual[e]
 *
 * r(e) is a 16-bit number: lane e % 8 (low half of word 0, high half of word
 * 0, low half of word 1, ...) of the Philox4x32-10 block ("Parallel random
 * numbers: as easy as 1, 2, 3", Salmon et al. 2011) with the 64-bit seed as
 * its key and the counter (e / 8, offset), low words first.  So the
 * probability has steps of 2^-16, and the scale uses the rounded one: kept
 * values average to x exactly.  Elements are numbered row-major over the whole
 * tensor; the same (seed, offset) gives the same mask on every device and in
 * every run, another offset gives an independent one (one per layer and step).
 * A dropped element is 0 whatever x holds, NaN and infinities included; T =
 * 65536 drops everything.
 *
 * Conventions as in linear_logp.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, arguments checked before anything is enqueued, the
 * same LLP_* status codes.  Tensors are contiguous, `count` elements of bf16
 * (dtype 0), fp32 (dtype 1) or fp16 (dtype 2), rounded once from fp32; count <=
 * 2^40.  Element alignment suffices; 16-byte aligned tensors move fastest.  y
 * may be x or residual itself.  count == 0 is a no-op.
 */
#ifndef DROPOUT_H_
#define DROPOUT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DROPOUT_DTYPE_BF16 0
#define DROPOUT_DTYPE_F32 1
#define DROPOUT_DTYPE_F16 2

/* residual may be NULL.  device_offset (NULL, or one int64 on the device) is
 * added to offset when the kernel runs: a captured graph that advances it
 * draws a new mask at each replay.  0 <= p <= 1. */
int dropout_fwd(const void* x, const void* residual, int dtype, int64_t count, double p, uint64_t seed,
                uint64_t offset, const int64_t* device_offset, void* y, void* stream);

/* grad_x[e] = (r(e) >= T ? grad_y[e] * 65536 / (65536 - T) : 0), with the
 * forward's p, seed and offset; the residual's gradient is grad_y itself. */
int dropout_bwd(const void* grad_y, int dtype, int64_t count, double p, uint64_t seed, uint64_t offset,
                const int64_t* device_offset, void* grad_x, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DROPOUT_H_ */
