// Argument checks that the C entry points of the token-sequence operators share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ss2d.h"
#include "ss2d_attention.h"
#include "ss2d_internal.h"
#include "ss2d_tokens.h"

namespace ss2d {
namespace checks {

inline int finish(hipError_t e) {
  if (e == hipSuccess) return SS2D_OK;
  ss2d::remember_hip_error(e);
  return SS2D_ERR_HIP;
}

inline int check_device() {
  int dev = -1;
  const hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess && dev >= 0) return SS2D_OK;
  if (e != hipSuccess) ss2d::remember_hip_error(e);
  return SS2D_ERR_NO_DEVICE;
}

inline bool dtype_ok(int dtype) { return dtype == SS2D_F32 || dtype == SS2D_BF16; }
inline int64_t elem_bytes(int dtype) { return dtype == SS2D_BF16 ? 2 : 4; }

// A range of bytes an argument occupies.
struct Range {
  const void* p;
  int64_t bytes;
};

inline bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

inline bool misaligned(const void* p, int64_t to) { return ((uintptr_t)p & (uintptr_t)(to - 1)) != 0; }

// Bytes of a workspace argument that holds `need`, checked.
inline int check_workspace(const void* workspace, int64_t bytes, int64_t need) {
  if (need > 0 && (!workspace || bytes < need || misaligned(workspace, 16))) return SS2D_ERR_WORKSPACE;
  return SS2D_OK;
}

// Overlap other than being the very same tensor.
inline bool partly(const Range& a, const Range& b) { return a.p != b.p && overlap(a, b); }

// Bytes from a strided tensor's first to behind its last element; -1 if they do
// not fit.  Axes: sequence (unused when packed), token (at most `far` apart), head,
// and `inner` dense.
inline int64_t extent(const int64_t* stride, int64_t sequences, int64_t tokens, int64_t heads, int64_t inner, bool packed,
               int64_t elem, int64_t far = ss2d::kMaxTokenStride) {
  const int64_t n[3] = {packed ? 1 : sequences, packed ? tokens : tokens / sequences, heads};
  int64_t last = 0;
  for (int i = 0; i < 3; ++i) {
    int64_t part;
    if (n[i] == 1) continue;
    if (stride[i] < 0 || (i == 1 && stride[i] > far) || __builtin_mul_overflow(n[i] - 1, stride[i], &part) ||
        __builtin_add_overflow(last, part, &last))
      return -1;
  }
  if (last > INT64_MAX / 16 - inner) return -1;
  return (last + inner) * elem;
}

inline int check_attention_sizes(const ss2d_attention_sizes* z, bool packed, int dtype) {
  if (!z) return SS2D_ERR_NULL;
  if (z->sequences < 1 || z->sequences > (1 << 24) || z->tokens < 1 || z->tokens > INT32_MAX || z->heads < 1 ||
      z->heads > 65536 || z->groups < 1 || z->heads % z->groups != 0 || z->key_dim < 1 ||
      z->key_dim > ss2d::kMaxKeyDim || z->value_dim < 1 || z->value_dim > ss2d::kMaxValueDim)
    return SS2D_ERR_SHAPE;
  if (!packed && z->tokens % z->sequences != 0) return SS2D_ERR_SHAPE;
  if (!dtype_ok(dtype)) return SS2D_ERR_DTYPE;
  return SS2D_OK;
}

inline ss2d::AttentionArgs attention_args(const void* q, const void* k, const void* v, const float* log_decay,
                                   const float* state_in, const int32_t* cu_seqlens, void* o, float* state_out,
                                   const ss2d_attention_sizes& z, float scale, int dtype, void* workspace,
                                   void* stream) {
  ss2d::AttentionArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.log_decay = log_decay;
  a.state_in = state_in;
  a.cu = cu_seqlens;
  a.o = o;
  a.state_out = state_out;
  a.sequences = z.sequences;
  a.tokens = z.tokens;
  a.groups = z.groups;
  a.heads = z.heads;
  a.key_dim = z.key_dim;
  a.value_dim = z.value_dim;
  for (int i = 0; i < 3; ++i) {
    a.q_stride[i] = z.q_stride[i];
    a.k_stride[i] = z.k_stride[i];
    a.v_stride[i] = z.v_stride[i];
    a.g_stride[i] = z.decay_stride[i];
  }
  a.scale = scale;
  a.dtype = dtype;
  a.workspace = workspace;
  a.stream = static_cast<hipStream_t>(stream);
  return a;
}

// The arguments of one token per row over a cache of states, checked, as `a`.
inline int check_step(const void* q, const void* k, const void* v, const float* log_decay, float* state,
                      const int32_t* index, void* o, int64_t rows, int64_t slots, int64_t groups, int64_t heads,
                      int64_t key_dim, int64_t value_dim, int64_t q_row, int64_t k_row, int64_t v_row, float scale,
                      int dtype, void* stream, ss2d::StepArgs& a) {
  if (!q || !k || !v || !log_decay || !state || !o) return SS2D_ERR_NULL;
  if (rows < 1 || rows > 65535 || slots < 1 || slots > INT32_MAX || (!index && rows > slots) || groups < 1 ||
      heads < 1 || heads > 65536 || heads % groups != 0 || key_dim < 1 || key_dim > ss2d::kMaxKeyDim ||
      value_dim < 1 || value_dim > ss2d::kMaxValueDim)
    return SS2D_ERR_SHAPE;
  if (!dtype_ok(dtype)) return SS2D_ERR_DTYPE;
  const int64_t e = elem_bytes(dtype);
  const int64_t strides[3][3] = {{0, q_row, 0}, {0, k_row, 0}, {0, v_row, 0}};
  const Range in[5] = {{q, extent(strides[0], 1, rows, 1, groups * key_dim, true, e, INT64_MAX)},
                       {k, extent(strides[1], 1, rows, 1, groups * key_dim, true, e, INT64_MAX)},
                       {v, extent(strides[2], 1, rows, 1, heads * value_dim, true, e, INT64_MAX)},
                       {log_decay, rows * heads * 4},
                       {index, rows * 4}};
  for (const Range& r : in)
    if (r.bytes < 0) return SS2D_ERR_SHAPE;
  if (rows * heads * ((value_dim + 15) / 16) > INT32_MAX || slots > INT64_MAX / 4 / (heads * key_dim * value_dim))
    return SS2D_ERR_SHAPE;
  const Range rs{state, slots * heads * key_dim * value_dim * 4}, ro{o, rows * heads * value_dim * e};
  for (const Range& r : in)
    if (overlap(ro, r) || overlap(rs, r)) return SS2D_ERR_ALIAS;
  if (overlap(ro, rs)) return SS2D_ERR_ALIAS;
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(o, e) || misaligned(log_decay, 4) ||
      misaligned(state, 4) || misaligned(index, 4))
    return SS2D_ERR_ALIGN;
  a = ss2d::StepArgs{q,     k,         v,     log_decay, state, index, o,     rows,  slots,
                         groups, heads,    key_dim, value_dim, q_row, k_row, v_row, scale, dtype,
                         static_cast<hipStream_t>(stream)};
  return SS2D_OK;
}

}  // namespace checks
}  // namespace ss2d
