/*
 * ss2d_delta_rule.h -- C ABI of libss2d.so's gated delta rule and of the norms that
 * its queries and keys come from; token-sequence operators beside those of
 * ss2d_tokens.h.
 *   gated delta rule     linear attention whose state replaces what it holds for a
 *       key instead of adding to it: forward over prompts, its gradients, and one
 *       token per row over a cache of states;
 *   query and key norms  the root-mean-square norm of each head's query and key with
 *       the rotation by the token's position in the same pass, and its gradients.
 *
 * Status codes, storage types, memory, streams, workspaces and threads as in
 * ss2d_tokens.h.
 */
#ifndef SS2D_DELTA_RULE_H_
#define SS2D_DELTA_RULE_H_

#include <stdint.h>

#include "ss2d_tokens.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes and strides of the delta rule: linear attention's, and beta's strides. */
typedef struct {
  ss2d_attention_sizes a;
  int64_t beta_stride[3];
} ss2d_delta_sizes;

/*
 * ss2d_delta_rule -- the gated delta rule over prompts:
 *     h_t = exp(g_t) h_{t-1} + beta_t k_t (v_t - exp(g_t) h_{t-1}' k_t)',
 *     o_t = scale h_t' q_t,
 * h a key_dim x value_dim state per sequence and head.
 *   q, k, v, log_decay, state_in, cu_seqlens, o, state_out  as in ss2d_linear_attention
 *   beta       [tokens, heads] fp32    strided; the share of a key's old value that is
 *              replaced, usually in [0, 1].  With keys of unit length (a weight of
 *              key_dim^-0.5 in ss2d_qk_norm) the state stays bounded for beta in [0, 2];
 *              where beta |k|^2 is over 2 it grows from token to token, and results lose
 *              precision with it.
 * Outputs must not overlap inputs, but state_out may be state_in itself
 * (SS2D_ERR_ALIAS).  States, decays, sums and the triangular systems of 64 tokens
 * (32 in fp32) are fp32, decays summed in fp64, and what enters a product keeps 24 bits
 * in either type: an output in bf16 shows its own rounding alone.  NaN and Inf
 * propagate: from a token to its sequence's outputs from up to 63 tokens before it on, so
 * padding behind a sequence's end has to be finite, or left out by cu_seqlens.
 * Results do not depend on the workspace, streams, or other sequences' values.  Where
 * long sequences are cut goes by the sizes of the call, so another packing of the same
 * sequence may round differently.
 * SS2D_ERR_SHAPE for sizes out of ss2d_linear_attention's ranges, and over 2^30
 * workgroups: chunks of 64 (32) tokens times heads, or segments times heads times tiles
 * of 64 value and key columns.
 */
int ss2d_delta_rule(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                    const float* state_in, const int32_t* cu_seqlens, void* o, float* state_out,
                    const ss2d_delta_sizes* sizes, float scale, int dtype, void* workspace, int64_t workspace_bytes,
                    void* stream);

/* Bytes of workspace ss2d_delta_rule needs, or a negative status.  packed: 1 if it will
 * be given cu_seqlens, else 0.  24 KiB per 64 tokens and head (8 KiB per 32 in fp32),
 * each packed sequence's last chunk counted whole; and where long sequences of few heads
 * are cut, packed ones too that might be long, a state and a key_dim x key_dim map per
 * segment and head: at most about 2048 / tiles of 64 value columns of these, however many
 * sequences there are. */
int64_t ss2d_delta_rule_workspace(const ss2d_delta_sizes* sizes, int packed, int dtype);

/*
 * ss2d_delta_rule_backward -- the gradients of ss2d_delta_rule.
 *   inputs  q, k, v, log_decay, beta, state_in, cu_seqlens as for the forward;
 *           d_o         [tokens, heads, value_dim] dtype, strided (do_stride)
 *           dstate_out  gradient of state_out, fp32, dense, or NULL for 0
 *   outputs dq, dk      [tokens, groups, key_dim] dtype, dense, summed over a group's
 *                       heads in a fixed order
 *           dv          [tokens, heads, value_dim] dtype, dense
 *           dlog_decay, dbeta  [tokens, heads] fp32, dense (where stride 0 repeats a
 *                       value, the gradient of each of its uses)
 *           dstate_in   [sequences, heads, key_dim, value_dim] fp32 or NULL
 * Outputs are overwritten, not added to; tokens outside the sequences keep what they
 * were.  Outputs must not overlap inputs or each other.  What enters a product keeps 24
 * bits in either type, so dq, dk and dv in bf16 show their own rounding alone.
 * dlog_decay sums terms of its chunk that cancel, q.dq - dv.v of the tokens behind it and
 * the state with its gradient, and its error is fp32's relative to those terms' sizes: the
 * gradient of a token that forgets nearly everything, near exp(g), may have no correct
 * digits.
 */
int ss2d_delta_rule_backward(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                             const float* state_in, const int32_t* cu_seqlens, const void* d_o,
                             const float* dstate_out, void* dq, void* dk, void* dv, float* dlog_decay, float* dbeta,
                             float* dstate_in, const ss2d_delta_sizes* sizes, float scale, int dtype, void* workspace,
                             int64_t workspace_bytes, void* stream);

/* Bytes of workspace ss2d_delta_rule_backward needs, or a negative status: two states
 * per chunk of 64 (32) tokens and head, among others. */
int64_t ss2d_delta_rule_backward_workspace(const ss2d_delta_sizes* sizes, int packed, int dtype);

/*
 * ss2d_delta_rule_step -- one token for each row, over a cache of states updated in
 * place:  h <- exp(g) h,  u = beta (v - h' k),  h <- h + k u',  o = scale h' q.
 *   beta       [rows, heads] fp32, dense; all else, ranges too, as in
 *              ss2d_linear_attention_step (index, padding rows, rows of one slot)
 * One kernel, no workspace; all arithmetic is fp32.
 */
int ss2d_delta_rule_step(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                         float* state, const int32_t* index, void* o, int64_t rows, int64_t slots, int64_t groups,
                         int64_t heads, int64_t key_dim, int64_t value_dim, int64_t q_row, int64_t k_row,
                         int64_t v_row, float scale, int dtype, void* stream);

/*
 * Sizes and strides of the query and key norms.  Strides are in elements, for each of
 * sequence, token and head, at least 0; the innermost axis (dim) is dense.  q_out_stride
 * and k_out_stride are those of the outputs, for gradients of the outputs' gradients;
 * an output's elements must be apart (SS2D_ERR_SHAPE otherwise).
 */
typedef struct {
  int64_t sequences;      /* >= 1                                                     */
  int64_t tokens;         /* of one sequence, >= 1                                    */
  int64_t q_heads, k_heads;  /* >= 1                                                  */
  int64_t dim;            /* 1..256                                                   */
  int64_t rotated;        /* channels that rotate, the first of each head: even, at    */
                          /* most dim; 0 if and only if there is no rotation table    */
  int64_t table_rows;     /* positions in the table; unused without one               */
  int64_t q_stride[3], k_stride[3], q_out_stride[3], k_out_stride[3];
} ss2d_qk_sizes;

/*
 * ss2d_qk_norm -- for each token and head, x a query or key:
 *     y = R(x / sqrt(mean(x^2) + eps) * weight),
 * R turning pairs of channels by the angles of the token's position.
 *   q          [sequences, tokens, q_heads, dim] dtype, strided
 *   k          [sequences, tokens, k_heads, dim] dtype, strided
 *   q_weight, k_weight  [dim] fp32, or NULL for 1.  A weight of dim^-0.5 gives unit
 *              length (up to eps)
 *   rotation   [table_rows, rotated] fp32: for each position the cosines of its
 *              rotated / 2 angles, then the sines; or NULL for no rotation
 *   positions  [sequences, tokens] int32: each token's row of the table; or NULL: its
 *              number in its sequence.  Clamped to 0..table_rows-1 on the device
 *   interleaved  0: channels i and i + rotated / 2 are a pair (i < rotated / 2);
 *              1: channels 2 i and 2 i + 1
 *   q_out, k_out  as q and k, strided; each may be its own input (the same strides), and
 *              the two sides may lie in one tensor in any layout that leaves them no
 *              address in common: slices of a projection's rows, q, k and v side by side
 *              for each head, heads or planes before tokens (SS2D_ERR_ALIAS otherwise)
 * All arithmetic is fp32, each output rounded once.  A head with squares that overflow
 * fp32 (values over 2^63) gives 0, a head of zeros 0 too, but NaN if eps is 0.  At most 2^31-1 tokens times heads, dim 1..256,
 * eps >= 0 and finite (SS2D_ERR_SHAPE otherwise).  One kernel, no workspace.
 */
int ss2d_qk_norm(const void* q, const void* k, const float* q_weight, const float* k_weight, const float* rotation,
                 const int32_t* positions, void* q_out, void* k_out, const ss2d_qk_sizes* sizes, float eps,
                 int interleaved, int dtype, void* stream);

/*
 * ss2d_qk_norm_backward -- the gradients of ss2d_qk_norm with respect to q, k and the
 * weights.
 *   inputs  q, k, weights, rotation, positions as for the forward; dq_out, dk_out the
 *           gradients of its outputs, strided (q_out_stride, k_out_stride; a stride of 0
 *           repeats a value)
 *   outputs dq, dk  as q and k, dense; must not overlap inputs
 *           dq_weight, dk_weight  [dim] fp32, NULL if not wanted (always so without the
 *           weight); sums in fp32 in a fixed order
 *   workspace    only with a weight's gradient
 */
int ss2d_qk_norm_backward(const void* q, const void* k, const float* q_weight, const float* k_weight,
                          const float* rotation, const int32_t* positions, const void* dq_out, const void* dk_out,
                          void* dq, void* dk, float* dq_weight, float* dk_weight, const ss2d_qk_sizes* sizes,
                          float eps, int interleaved, int dtype, void* workspace, int64_t workspace_bytes,
                          void* stream);
int64_t ss2d_qk_norm_backward_workspace(const ss2d_qk_sizes* sizes, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* SS2D_DELTA_RULE_H_ */
