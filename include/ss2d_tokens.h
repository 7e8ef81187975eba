/*
 * ss2d_tokens.h -- C ABI of libss2d.so's token-sequence operators: what a
 * language model's layer runs next to the scans of ss2d.h.
 *   linear attention with a decay per head   the state recurrence of the scans
 *       with one decay for a head's whole state: forward over prompts, its
 *       gradients, and one token per row over a cache of states;
 *   root-mean-square norm                    with the residual's addition, in the
 *       storage type or in 8 bits with scales, and its gradients;
 *   8-bit matrix product                     e4m3 values with a scale per block
 *       of 128, what the norm's 8-bit output is projected with.
 *
 * Status codes, the storage types (ss2d_dtype) and the error texts are those of
 * ss2d.h.  Every tensor pointer is DEVICE memory owned by the caller.  Arguments
 * are validated before any device work; on SS2D_OK the work has been enqueued
 * asynchronously on `stream` (a hipStream_t of the current device, NULL = the
 * default stream).  Nothing is printed, thrown or aborted, and the calls keep
 * nothing between them: they are thread-safe, and may run under graph capture.
 * None allocates: where a call needs a temporary the caller passes a workspace of
 * the size that the matching *_workspace function returns, aligned to 16 bytes.
 * Its contents need not be initialised and mean nothing after the call; calls
 * that may run at the same time (two streams, two captured graphs) need one each.
 * Pointers need the alignment of their elements.
 */
#ifndef SS2D_TOKENS_H_
#define SS2D_TOKENS_H_

#include <stdint.h>

#include "ss2d.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Sizes and strides of linear attention.  Strides are in elements, for each of
 * sequence, token and head, at least 0 (0 repeats one value along that axis) and
 * for tokens below 2^24; the innermost axis (key_dim or value_dim) is dense.  With
 * packed sequences the sequence stride is unused.  do_stride is used by the backward
 * only.
 */
typedef struct {
  int64_t sequences;  /* >= 1                                                        */
  int64_t tokens;     /* of all sequences together, >= 1; without cu_seqlens a        */
                      /* multiple of `sequences` (each then has tokens/sequences)    */
  int64_t groups;     /* heads of q and k; divides `heads`: value head h reads        */
                      /* group h / (heads / groups)                                  */
  int64_t heads;      /* heads of v, the decay, the states and the output             */
  int64_t key_dim;    /* 1..256                                                      */
  int64_t value_dim;  /* 1..1024                                                     */
  int64_t q_stride[3], k_stride[3], v_stride[3], decay_stride[3], do_stride[3];
} ss2d_attention_sizes;

/*
 * ss2d_linear_attention -- linear attention with a decay per head, over prompts:
 *     h_t = exp(g_t) h_{t-1} + k_t v_t',   o_t = scale h_t' q_t,
 * h a key_dim x value_dim state per sequence and head.
 *   q, k       [tokens, groups, key_dim]   dtype   strided as `sizes` says
 *   v          [tokens, heads, value_dim]  dtype   strided
 *   log_decay  [tokens, heads]             fp32    strided; g, usually <= 0.  Values
 *              under -104 (exp of them is 0 in fp32), -Inf too, count as a decay to 0;
 *              sums over 88 within 64 tokens (exp of them is Inf) may give NaN.
 *   state_in   [sequences, heads, key_dim, value_dim] fp32, or NULL for 0
 *   cu_seqlens [sequences + 1] int32, or NULL: sequence s is the tokens
 *              cu_seqlens[s] .. cu_seqlens[s+1]-1 (none: an empty sequence, whose final
 *              state is its initial one).  Must not decrease; values are clamped to
 *              0..tokens on the device, so wrong ones give wrong results but no access
 *              out of range.  Tokens before the first and behind the last sequence are
 *              not read and their outputs are left as they were.
 *   o          [tokens, heads, value_dim]  dtype   out, dense
 *   state_out  [sequences, heads, key_dim, value_dim] fp32, out, or NULL; may be
 *              state_in itself
 * Outputs must not overlap inputs otherwise (SS2D_ERR_ALIAS).  States, decays and
 * sums are fp32 (decays summed in fp64).  For bf16 the masked scores and the state
 * are rounded to bf16 for their products into o, whose own rounding is as large; what
 * the state itself is made of keeps all its bits.  NaN and Inf propagate: from a token to its
 * sequence's outputs from up to 63 tokens before it on (tokens are taken in chunks as
 * matrix products), so padding behind a sequence's end has to be finite, or left out
 * by cu_seqlens.  Results do not depend on the
 * workspace, other sequences or streams: no atomics, sums in a fixed order.
 * SS2D_ERR_SHAPE for sizes outside the ranges above, token strides of 2^24 and more,
 * and over 2^30 tiles of 64 value columns of all heads and segments (a sequence has one
 * or more) or blocks of 256 entries of all states.
 */
int ss2d_linear_attention(const void* q, const void* k, const void* v, const float* log_decay,
                          const float* state_in, const int32_t* cu_seqlens, void* o, float* state_out,
                          const ss2d_attention_sizes* sizes, float scale, int dtype, void* workspace,
                          int64_t workspace_bytes, void* stream);

/* Bytes of workspace ss2d_linear_attention needs (0: none), or a negative status.
 * packed: 1 if it will be given cu_seqlens, else 0. */
int64_t ss2d_linear_attention_workspace(const ss2d_attention_sizes* sizes, int packed, int dtype);

/*
 * ss2d_linear_attention_backward -- the gradients of ss2d_linear_attention.
 *   inputs  q, k, v, log_decay, state_in, cu_seqlens as for the forward;
 *           d_o         [tokens, heads, value_dim] dtype, strided
 *           dstate_out  gradient of state_out, fp32, dense, or NULL for 0
 *   outputs dq, dk      [tokens, groups, key_dim] dtype, dense, summed over a group's
 *                       heads in a fixed order
 *           dv          [tokens, heads, value_dim] dtype, dense
 *           dlog_decay  [tokens, heads] fp32, dense (a decay repeated by stride 0 gets
 *                       the gradient of each of its uses)
 *           dstate_in   [sequences, heads, key_dim, value_dim] fp32 or NULL
 * Outputs are overwritten, not added to; tokens outside the sequences keep what they
 * were.  Outputs must not overlap inputs or each other.  Rounding, validation and the
 * rest as for the forward.
 */
int ss2d_linear_attention_backward(const void* q, const void* k, const void* v, const float* log_decay,
                                   const float* state_in, const int32_t* cu_seqlens, const void* d_o,
                                   const float* dstate_out, void* dq, void* dk, void* dv, float* dlog_decay,
                                   float* dstate_in, const ss2d_attention_sizes* sizes, float scale, int dtype,
                                   void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace ss2d_linear_attention_backward needs, or a negative status. */
int64_t ss2d_linear_attention_backward_workspace(const ss2d_attention_sizes* sizes, int packed, int dtype);

/*
 * ss2d_linear_attention_step -- one token for each row, over a cache of states:
 *     h = exp(g) h + k v',   o = scale h' q,
 * the state updated in place.
 *   q, k       [rows, groups, key_dim]  dtype, dense inside a row; rows are
 *   v          [rows, heads, value_dim] dtype  q_row, k_row and v_row elements apart
 *   log_decay  [rows, heads] fp32, dense
 *   state      [slots, heads, key_dim, value_dim] fp32, in and out
 *   index      [rows] int32, the row's slot, or NULL: row i has slot i (rows <= slots).
 *              A row whose index is outside 0..slots-1 is padding: its output is 0 and
 *              no state is read or written for it.  Rows of one slot are consecutive
 *              tokens of one sequence, in the order of the rows.
 *   o          [rows, heads, value_dim] dtype, dense
 * key_dim 1..256, value_dim 1..1024, rows and slots >= 1, rows at most 65535
 * (SS2D_ERR_SHAPE otherwise).  One kernel, no workspace; all arithmetic is fp32.
 */
int ss2d_linear_attention_step(const void* q, const void* k, const void* v, const float* log_decay, float* state,
                               const int32_t* index, void* o, int64_t rows, int64_t slots, int64_t groups,
                               int64_t heads, int64_t key_dim, int64_t value_dim, int64_t q_row, int64_t k_row,
                               int64_t v_row, float scale, int dtype, void* stream);

/*
 * ss2d_rms_norm -- root-mean-square norm of rows, with the residual's addition:
 *     r = x + residual,   y = r / sqrt(mean(r^2) + eps) * weight.
 *   x            [rows, dim] dtype
 *   residual     [rows, dim] dtype, or NULL (r = x)
 *   weight       [dim] fp32, or NULL for 1
 *   residual_out [rows, dim] dtype: r, rounded once; NULL if not wanted; may be x or
 *                residual itself
 *   y            [rows, dim]: dtype if scales is NULL, rounded once (may then be x or
 *                residual itself, but not residual_out); with scales, e4m3 (one byte):
 *   scales       [rows, ceil(dim/128)] fp32 or NULL: per 128 channels (the last block
 *                may be shorter) s = max(max|y| / 448, 2^-126), and the stored value is
 *                y / s rounded to nearest even; NaN stays NaN
 * y is formed from the unrounded fp32 sum; squares are summed in fp32, so a row with
 * values over 2^63 gives 0.  rows 1..2^31-1, dim 1..16384; eps >= 0 and
 * finite (SS2D_ERR_SHAPE otherwise).  One kernel, no workspace.
 */
int ss2d_rms_norm(const void* x, const void* residual, const float* weight, float eps, void* residual_out, void* y,
                  float* scales, int64_t rows, int64_t dim, int dtype, void* stream);

/*
 * ss2d_rms_norm_backward -- the gradients of y = r / sqrt(mean(r^2) + eps) * weight:
 *     dx = dresidual + rstd (weight dy - xhat mean(weight dy xhat)),   xhat = r rstd,
 *     dweight = sum over rows of dy xhat.
 *   r            [rows, dim] dtype: residual_out of the forward (x without a residual);
 *                dx is the gradient of both x and the residual
 *   dy           [rows, dim] dtype
 *   dresidual    [rows, dim] dtype: gradient of residual_out, or NULL for 0
 *   dx           [rows, dim] dtype, may be dy or dresidual itself
 *   dweight      [dim] fp32, or NULL if not wanted (always so without a weight)
 *   workspace    only with dweight; sums run in a fixed order
 */
int ss2d_rms_norm_backward(const void* r, const float* weight, const void* dy, const void* dresidual, float eps,
                           void* dx, float* dweight, int64_t rows, int64_t dim, int dtype, void* workspace,
                           int64_t workspace_bytes, void* stream);
int64_t ss2d_rms_norm_backward_workspace(int64_t rows, int64_t dim, int dtype);

/*
 * ss2d_matmul_fp8 -- out = a b', both in e4m3 with scales:
 *     out[m, n] = sum_j a_scales[m, j] b_scales[n / 128, j] sum_{k in block j} a[m, k] b[n, k],
 * block j the inner indices 128 j .. 128 j + 127 (the last may be shorter).
 *   a         [m, k] e4m3         a_scales  [m, ceil(k/128)] fp32
 *   b         [n, k] e4m3         b_scales  [ceil(n/128), ceil(k/128)] fp32
 *   out       [m, n] dtype (fp32 or bf16, rounded once)
 * All dense; out must not overlap an input.  The two scales' product is formed in fp32
 * (under 2^-126 it loses bits).  Sums are fp32 on the matrix cores, in a
 * fixed order.  For a bf16 output the products run in 8 bits, where the instruction
 * drops, in each group of eight inner indices, what lies below 2^-13 of the group's
 * largest product; for an fp32 output they run in bf16 (exact values), all bits kept.
 * m, n 1..2^30, at most 2^31-1 tiles of 16 x 16 in out, k 1..2^20 (SS2D_ERR_SHAPE
 * otherwise).  One kernel, no
 * workspace; any k and any addresses, fastest with k a multiple of 16 and a and b
 * aligned to 16 bytes.
 */
int ss2d_matmul_fp8(const void* a, const float* a_scales, const void* b, const float* b_scales, void* out, int64_t m,
                    int64_t n, int64_t k, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SS2D_TOKENS_H_ */
