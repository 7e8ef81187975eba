// C ABI of the token-sequence operators: argument validation and launch.  The
// declarations and their contract are in include/ss2d_tokens.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ss2d.h"
#include "ss2d_api_checks.h"
#include "ss2d_attention.h"
#include "ss2d_token_ops.h"
#include "ss2d_tokens.h"

namespace {

using namespace ss2d::checks;

// ------------------------------------------------------------------ norm
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

int check_norm(const void* x, const void* y, const float* weight, float eps, int64_t rows, int64_t dim, int dtype) {
  if (!x || !y) return SS2D_ERR_NULL;
  if (rows < 1 || rows > kMaxRows || dim < 1 || dim > ss2d::kMaxNormDim) return SS2D_ERR_SHAPE;
  if (!(eps >= 0.f && eps < __builtin_inff())) return SS2D_ERR_SHAPE;  // also rejects NaN
  if (!dtype_ok(dtype)) return SS2D_ERR_DTYPE;
  if (misaligned(weight, 4)) return SS2D_ERR_ALIGN;
  return SS2D_OK;
}

// ------------------------------------------------------------------ attention
ss2d::AttentionPlan plan_of(const ss2d_attention_sizes* z, bool packed, int dtype) {
  return ss2d::plan_attention(z->sequences, z->tokens, z->heads, z->key_dim, z->value_dim, packed, dtype);
}

ss2d::AttentionPlan backward_plan_of(const ss2d_attention_sizes* z, bool packed, int dtype) {
  return ss2d::plan_attention_backward(z->sequences, z->tokens, z->heads, z->key_dim, z->value_dim, packed, dtype);
}

// Whether a plan's launches fit a grid: two passes' segments in tiles of 64 value
// columns, two passes' state entries.
bool grid_ok(const ss2d::AttentionPlan& pl, const ss2d_attention_sizes& z) {
  return pl.slots * z.heads * pl.vtiles * (pl.vt / 64) <= INT32_MAX / 2 &&
         z.sequences * z.heads * ((z.key_dim * z.value_dim + 255) / 256) <= INT32_MAX / 2;
}
// The same with the sums of dq's, dk's and the decay's parts.
bool backward_grid_ok(const ss2d::AttentionPlan& pl, const ss2d_attention_sizes& z) {
  return grid_ok(pl, z) && z.tokens * z.groups * z.key_dim / 256 < INT32_MAX && z.tokens * z.heads / 256 < INT32_MAX;
}

}  // namespace

extern "C" {

int64_t ss2d_linear_attention_backward_workspace(const ss2d_attention_sizes* sizes, int packed, int dtype) {
  const int rc = check_attention_sizes(sizes, packed != 0, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d::AttentionPlan pl = backward_plan_of(sizes, packed != 0, dtype);
  if (!backward_grid_ok(pl, *sizes)) return SS2D_ERR_SHAPE;
  return (int64_t)ss2d::attention_backward_workspace_bytes(pl, sizes->tokens, sizes->groups, sizes->heads,
                                                           sizes->key_dim, sizes->value_dim);
}

int ss2d_linear_attention_backward(const void* q, const void* k, const void* v, const float* log_decay,
                                   const float* state_in, const int32_t* cu_seqlens, const void* d_o,
                                   const float* dstate_out, void* dq, void* dk, void* dv, float* dlog_decay,
                                   float* dstate_in, const ss2d_attention_sizes* sizes, float scale, int dtype,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv || !dlog_decay || !sizes) return SS2D_ERR_NULL;
  const bool packed = cu_seqlens != nullptr;
  int rc = check_attention_sizes(sizes, packed, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d_attention_sizes& z = *sizes;
  const int64_t e = elem_bytes(dtype), st = z.sequences * z.heads * z.key_dim * z.value_dim * 4;
  const Range in[8] = {{q, extent(z.q_stride, z.sequences, z.tokens, z.groups, z.key_dim, packed, e)},
                       {k, extent(z.k_stride, z.sequences, z.tokens, z.groups, z.key_dim, packed, e)},
                       {v, extent(z.v_stride, z.sequences, z.tokens, z.heads, z.value_dim, packed, e)},
                       {log_decay, extent(z.decay_stride, z.sequences, z.tokens, z.heads, 1, packed, 4)},
                       {d_o, extent(z.do_stride, z.sequences, z.tokens, z.heads, z.value_dim, packed, e)},
                       {cu_seqlens, (z.sequences + 1) * 4},
                       {state_in, st},
                       {dstate_out, st}};
  for (const Range& r : in)
    if (r.bytes < 0) return SS2D_ERR_SHAPE;
  const ss2d::AttentionPlan pl = backward_plan_of(sizes, packed, dtype);
  if (!backward_grid_ok(pl, z)) return SS2D_ERR_SHAPE;
  const int64_t need = (int64_t)ss2d::attention_backward_workspace_bytes(pl, z.tokens, z.groups, z.heads, z.key_dim,
                                                                         z.value_dim);
  const Range out[6] = {{dq, z.tokens * z.groups * z.key_dim * e},   {dk, z.tokens * z.groups * z.key_dim * e},
                        {dv, z.tokens * z.heads * z.value_dim * e},  {dlog_decay, z.tokens * z.heads * 4},
                        {dstate_in, st},                             {need > 0 ? workspace : nullptr, need}};
  for (int i = 0; i < 6; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return SS2D_ERR_ALIAS;
    for (int j = i + 1; j < 6; ++j)
      if (overlap(out[i], out[j])) return SS2D_ERR_ALIAS;
  }
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(d_o, e) || misaligned(dq, e) ||
      misaligned(dk, e) || misaligned(dv, e) || misaligned(log_decay, 4) || misaligned(dlog_decay, 4) ||
      misaligned(state_in, 4) || misaligned(dstate_out, 4) || misaligned(dstate_in, 4) || misaligned(cu_seqlens, 4))
    return SS2D_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != SS2D_OK) return rc;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  ss2d::AttentionBackwardArgs a{};
  a.f = attention_args(q, k, v, log_decay, state_in, cu_seqlens, nullptr, nullptr, z, scale, dtype, workspace, stream);
  a.d_o = d_o;
  for (int i = 0; i < 3; ++i) a.do_stride[i] = z.do_stride[i];
  a.dstate_out = dstate_out;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dlog_decay = dlog_decay;
  a.dstate_in = dstate_in;
  return finish(ss2d::launch_attention_backward(a, pl));
}

int64_t ss2d_linear_attention_workspace(const ss2d_attention_sizes* sizes, int packed, int dtype) {
  const int rc = check_attention_sizes(sizes, packed != 0, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d::AttentionPlan pl = plan_of(sizes, packed != 0, dtype);
  if (!grid_ok(pl, *sizes)) return SS2D_ERR_SHAPE;
  return (int64_t)ss2d::attention_workspace_bytes(pl, sizes->heads, sizes->key_dim, sizes->value_dim);
}

int ss2d_linear_attention(const void* q, const void* k, const void* v, const float* log_decay, const float* state_in,
                          const int32_t* cu_seqlens, void* o, float* state_out, const ss2d_attention_sizes* sizes,
                          float scale, int dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !log_decay || !o || !sizes) return SS2D_ERR_NULL;
  const bool packed = cu_seqlens != nullptr;
  int rc = check_attention_sizes(sizes, packed, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d_attention_sizes& z = *sizes;
  const int64_t e = elem_bytes(dtype);
  const Range in[6] = {{q, extent(z.q_stride, z.sequences, z.tokens, z.groups, z.key_dim, packed, e)},
                       {k, extent(z.k_stride, z.sequences, z.tokens, z.groups, z.key_dim, packed, e)},
                       {v, extent(z.v_stride, z.sequences, z.tokens, z.heads, z.value_dim, packed, e)},
                       {log_decay, extent(z.decay_stride, z.sequences, z.tokens, z.heads, 1, packed, 4)},
                       {cu_seqlens, (z.sequences + 1) * 4},
                       {state_in, z.sequences * z.heads * z.key_dim * z.value_dim * 4}};
  for (const Range& r : in)
    if (r.bytes < 0) return SS2D_ERR_SHAPE;
  const Range ro{o, z.tokens * z.heads * z.value_dim * e}, rs{state_out, in[5].bytes};
  const ss2d::AttentionPlan pl = plan_of(sizes, packed, dtype);
  if (!grid_ok(pl, z)) return SS2D_ERR_SHAPE;
  const int64_t need = (int64_t)ss2d::attention_workspace_bytes(pl, z.heads, z.key_dim, z.value_dim);
  const Range rw{need > 0 ? workspace : nullptr, need};
  for (int i = 0; i < 6; ++i)
    if (overlap(ro, in[i]) || overlap(rw, in[i]) || (i < 5 ? overlap(rs, in[i]) : partly(rs, in[i])))
      return SS2D_ERR_ALIAS;
  if (overlap(ro, rs) || overlap(ro, rw) || overlap(rs, rw)) return SS2D_ERR_ALIAS;
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(o, e) || misaligned(log_decay, 4) ||
      misaligned(state_in, 4) || misaligned(state_out, 4) || misaligned(cu_seqlens, 4))
    return SS2D_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != SS2D_OK) return rc;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  const ss2d::AttentionArgs a = attention_args(q, k, v, log_decay, state_in, cu_seqlens, o, state_out, z, scale, dtype,
                                               workspace, stream);
  return finish(ss2d::launch_attention(a, pl));
}

int ss2d_linear_attention_step(const void* q, const void* k, const void* v, const float* log_decay, float* state,
                               const int32_t* index, void* o, int64_t rows, int64_t slots, int64_t groups,
                               int64_t heads, int64_t key_dim, int64_t value_dim, int64_t q_row, int64_t k_row,
                               int64_t v_row, float scale, int dtype, void* stream) {
  ss2d::StepArgs a{};
  int rc = check_step(q, k, v, log_decay, state, index, o, rows, slots, groups, heads, key_dim, value_dim, q_row, k_row,
                      v_row, scale, dtype, stream, a);
  if (rc != SS2D_OK) return rc;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  return finish(ss2d::launch_attention_step(a));
}

int ss2d_rms_norm(const void* x, const void* residual, const float* weight, float eps, void* residual_out, void* y,
                  float* scales, int64_t rows, int64_t dim, int dtype, void* stream) {
  int rc = check_norm(x, y, weight, eps, rows, dim, dtype);
  if (rc != SS2D_OK) return rc;
  const int64_t e = elem_bytes(dtype), n = rows * dim;
  const Range rx{x, n * e}, rr{residual, n * e}, rw{weight, dim * 4}, ro{residual_out, n * e},
      ry{y, n * (scales ? 1 : e)}, rs{scales, rows * ((dim + 127) / 128) * 4};
  if (overlap(ro, ry) || overlap(ro, rw) || overlap(ry, rw) || partly(ro, rx) || partly(ro, rr) ||
      overlap(rs, rx) || overlap(rs, rr) || overlap(rs, rw) || overlap(rs, ro) || overlap(rs, ry))
    return SS2D_ERR_ALIAS;
  if (scales ? overlap(ry, rx) || overlap(ry, rr) : partly(ry, rx) || partly(ry, rr)) return SS2D_ERR_ALIAS;
  if (misaligned(x, e) || misaligned(residual, e) || misaligned(residual_out, e) || misaligned(y, scales ? 1 : e) ||
      misaligned(scales, 4))
    return SS2D_ERR_ALIGN;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  const ss2d::NormArgs a{x,    residual, weight, residual_out, y, scales, eps, rows, dim, dtype,
                         static_cast<hipStream_t>(stream)};
  return finish(ss2d::launch_rms_norm(a));
}

int64_t ss2d_rms_norm_backward_workspace(int64_t rows, int64_t dim, int dtype) {
  if (rows < 1 || rows > kMaxRows || dim < 1 || dim > ss2d::kMaxNormDim) return SS2D_ERR_SHAPE;
  if (!dtype_ok(dtype)) return SS2D_ERR_DTYPE;
  return ss2d::norm_backward_blocks(rows, dim) * dim * 4;
}

int ss2d_rms_norm_backward(const void* r, const float* weight, const void* dy, const void* dresidual, float eps,
                           void* dx, float* dweight, int64_t rows, int64_t dim, int dtype, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  if (!dy) return SS2D_ERR_NULL;
  int rc = check_norm(r, dx, weight, eps, rows, dim, dtype);
  if (rc != SS2D_OK) return rc;
  const int64_t e = elem_bytes(dtype), n = rows * dim;
  const int64_t need = dweight ? ss2d_rms_norm_backward_workspace(rows, dim, dtype) : 0;
  const Range rr{r, n * e}, rw{weight, dim * 4}, ry{dy, n * e}, rd{dresidual, n * e}, rx{dx, n * e},
      rg{dweight, dim * 4}, rt{need > 0 ? workspace : nullptr, need};
  if (overlap(rx, rr) || overlap(rx, rw) || partly(rx, ry) || partly(rx, rd) || overlap(rx, rg)) return SS2D_ERR_ALIAS;
  for (const Range& q : {rr, rw, ry, rd})
    if (overlap(rg, q) || overlap(rt, q)) return SS2D_ERR_ALIAS;
  if (overlap(rt, rx) || overlap(rt, rg)) return SS2D_ERR_ALIAS;
  if (misaligned(r, e) || misaligned(dy, e) || misaligned(dresidual, e) || misaligned(dx, e) || misaligned(dweight, 4))
    return SS2D_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != SS2D_OK) return rc;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  const ss2d::NormBackwardArgs a{r,    weight, dy,  dresidual, dx, dweight, static_cast<float*>(workspace), eps,
                                 rows, dim,    dtype, static_cast<hipStream_t>(stream)};
  return finish(ss2d::launch_rms_norm_backward(a));
}

int ss2d_matmul_fp8(const void* a, const float* a_scales, const void* b, const float* b_scales, void* out, int64_t m,
                    int64_t n, int64_t k, int dtype, void* stream) {
  if (!a || !a_scales || !b || !b_scales || !out) return SS2D_ERR_NULL;
  constexpr int64_t most = (int64_t)1 << 30;
  if (m < 1 || m > most || n < 1 || n > most || k < 1 || k > (1 << 20)) return SS2D_ERR_SHAPE;
  if (((m + 15) / 16) * ((n + 15) / 16) > INT32_MAX) return SS2D_ERR_SHAPE;  // workgroups
  if (!dtype_ok(dtype)) return SS2D_ERR_DTYPE;
  const int64_t e = elem_bytes(dtype), kb = (k + 127) / 128;
  const Range ro{out, m * n * e};
  for (const Range& r : {Range{a, m * k}, Range{b, n * k}, Range{a_scales, m * kb * 4},
                         Range{b_scales, (n + 127) / 128 * kb * 4}})
    if (overlap(ro, r)) return SS2D_ERR_ALIAS;
  if (misaligned(out, e) || misaligned(a_scales, 4) || misaligned(b_scales, 4)) return SS2D_ERR_ALIGN;
  const int rc = check_device();
  if (rc != SS2D_OK) return rc;
  const ss2d::MatmulArgs x{a, a_scales, b, b_scales, out, m, n, k, dtype, static_cast<hipStream_t>(stream)};
  return finish(ss2d::launch_matmul_fp8(x));
}

}  // extern "C"
