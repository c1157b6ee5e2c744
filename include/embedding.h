/*
 * embedding.h -- C ABI of the token embedding on GB300 (sm_103a), in the same
 * library as linear_logp.h.
 *
 *     out[n, :]         = scale * weight[t_n, :]
 *     grad_weight[v, :] = scale * sum_{n : t_n = v} grad_out[n, :]
 *
 * A token that equals ignore_index or lies outside [0, V) is invalid: its
 * output row is zero, it adds nothing to any gradient, and neither the table
 * nor its grad_out row is read for it.
 *
 * The gradient sorts the tokens and sums each table row's tokens in ascending
 * token order in fp32, with one rounding to the table's type.  A row named
 * more than 32 times is summed in pieces, and groups of pieces, whose lengths
 * depend on that count alone, joined in ascending order.  A row of the gradient therefore depends
 * on its own tokens only, and is bitwise the same in every run.
 *
 * Conventions as in linear_logp.h: device pointers, caller-owned buffers, work
 * enqueued on `stream`, arguments checked before anything is enqueued, the
 * same LLP_* status codes.  tokens is int64 [N]; weight, grad_weight [V, D] and
 * out [N, D] are contiguous row-major in bf16 (dtype 0), fp32 (dtype 1) or
 * fp16 (dtype 2); any D >= 1.  Element alignment suffices; 16-byte aligned
 * tensors with rows of a multiple of 16 bytes move fastest.  scale is rounded
 * to fp32 by the caller; one that is not finite is refused (LLP_ERR_BAD_SHAPE).
 * N, V < 2^31, D < 2^22, N * D <= 2^42.
 */
#ifndef EMBEDDING_H_
#define EMBEDDING_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define EMBEDDING_DTYPE_BF16 0
#define EMBEDDING_DTYPE_F32 1
#define EMBEDDING_DTYPE_F16 2

/* Lookup.  out is overwritten; N == 0 is a no-op (tokens and out may be NULL). */
int embedding_fwd(const int64_t* tokens, const void* weight, int dtype, int64_t N, int64_t V, int64_t D, float scale,
                  int64_t ignore_index, void* out, void* stream);

/* Bytes of workspace embedding_bwd needs (0 when N == 0 or a size is invalid). */
size_t embedding_bwd_workspace_bytes(int64_t N, int64_t V, int64_t D);

/* Gradient of the table.  grad_out's rows start grad_out_row_stride < 2^31
 * elements apart (D when contiguous; 0 repeats one row).
 *   accumulate == 0: every row of grad_weight is overwritten (zero where no
 *     token names it); N == 0 writes zeros.
 *   accumulate != 0: the tokens' sums are added to the rows they name, in fp32
 *     with one rounding, and no other row is read or written -- for a table
 *     tied to the LM head whose gradient is there already; N == 0 is a no-op.
 * The workspace needs no clearing, and must be 16-byte aligned. */
int embedding_bwd(const int64_t* tokens, const void* grad_out, int64_t grad_out_row_stride, int dtype, int64_t N,
                  int64_t V, int64_t D, float scale, int64_t ignore_index, int accumulate, void* grad_weight,
                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EMBEDDING_H_ */
