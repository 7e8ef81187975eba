// C ABI of the gated delta rule and of the query and key norms: argument validation and
// launch.  The declarations and their contract are in include/ss2d_delta_rule.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ss2d_api_checks.h"
#include "ss2d_delta.h"
#include "ss2d_delta_rule.h"
#include "ss2d_qk_norm.h"

namespace {

using namespace ss2d::checks;

// ------------------------------------------------------------------ delta rule
ss2d::DeltaPlan plan_of(const ss2d_attention_sizes& z, bool packed, int dtype, bool backward) {
  return ss2d::plan_delta(z.sequences, z.tokens, z.heads, z.key_dim, z.value_dim, packed, dtype, backward);
}

constexpr int64_t kMostBlocks = (int64_t)1 << 30;
bool grid_ok(const ss2d::DeltaPlan& pl, const ss2d_attention_sizes& z) {
  return ss2d::delta_blocks(pl, z.sequences, z.heads, z.value_dim) <= kMostBlocks;
}
// The same with the sums of dq's and dk's parts.
bool backward_grid_ok(const ss2d::DeltaPlan& pl, const ss2d_attention_sizes& z) {
  return grid_ok(pl, z) && z.tokens * z.groups * z.key_dim / 256 < INT32_MAX;
}

ss2d::DeltaArgs delta_args(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                           const float* state_in, const int32_t* cu, void* o, float* state_out,
                           const ss2d_delta_sizes& z, float scale, int dtype, void* workspace, void* stream) {
  ss2d::DeltaArgs a{};
  a.f = attention_args(q, k, v, log_decay, state_in, cu, o, state_out, z.a, scale, dtype, workspace, stream);
  a.beta = beta;
  for (int i = 0; i < 3; ++i) a.beta_stride[i] = z.beta_stride[i];
  return a;
}

// ------------------------------------------------------------------ query and key norms
constexpr int64_t kMaxQkDim = 256;

// A strided tensor (sequence, token, head; `dim` dense) as its bytes.
struct Rows {
  const void* p;
  const int64_t* stride;
  int64_t heads;
};
int64_t bytes_of(const Rows& r, const ss2d_qk_sizes& z, int64_t e) {
  return extent(r.stride, z.sequences, z.sequences * z.tokens, r.heads, z.dim, false, e, INT64_MAX);
}
bool same(const Rows& a, const Rows& b, const ss2d_qk_sizes& z) {
  if (a.p != b.p || a.heads != b.heads) return false;
  const int64_t n[3] = {z.sequences, z.tokens, a.heads};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && a.stride[i] != b.stride[i]) return false;
  return true;
}
// Whether no two elements share an address: each axis steps over all that the narrower ones span.
bool apart(const Rows& r, const ss2d_qk_sizes& z) {
  int64_t n[3] = {z.sequences, z.tokens, r.heads}, s[3] = {r.stride[0], r.stride[1], r.stride[2]};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (s[j] > s[j + 1]) {
        const int64_t a = s[j], b = n[j];
        s[j] = s[j + 1];
        n[j] = n[j + 1];
        s[j + 1] = a;
        n[j + 1] = b;
      }
  int64_t span = z.dim;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (s[i] < span) return false;
    span += (n[i] - 1) * s[i];
  }
  return true;
}
// Whether x + sum of c s lies within `width` of 0 for some whole c in lo .. hi of each step; steps descend.  A step that is
// as wide as all that follow span leaves two or three c to look at; where steps mix so that there would be many, true.
struct Step {
  int64_t s, lo, hi;
};
bool meets(const Step* at, const Step* end, int64_t x, int64_t width, int& tries) {
  if (at == end) return x < width && -x < width;
  if (--tries < 0) return true;
  int64_t low = 1 - width, high = width - 1;  // what the others leave to come within reach
  for (const Step* i = at + 1; i < end; ++i) {
    low -= i->hi * i->s;
    high -= i->lo * i->s;
  }
  const int64_t from = low - x, to = high - x;
  int64_t c = from / at->s + (from % at->s > 0), last = to / at->s - (to % at->s < 0);
  if (c < at->lo) c = at->lo;
  if (last > at->hi) last = at->hi;
  for (; c <= last; ++c)
    if (meets(at + 1, end, x + c * at->s, width, tries)) return true;
  return false;
}
// Whether two tensors have no address in common, whatever the order of their axes in memory.
bool disjoint(const Rows& a, const Rows& b, const ss2d_qk_sizes& z, int64_t e) {
  if (!overlap(Range{a.p, bytes_of(a, z, e)}, Range{b.p, bytes_of(b, z, e)})) return true;
  const int64_t na[3] = {z.sequences, z.tokens, a.heads}, nb[3] = {z.sequences, z.tokens, b.heads};
  Step steps[6];
  int n = 0;
  auto add = [&](int64_t stride, int64_t lo, int64_t hi) {
    if (stride == 0 || lo == hi) return;
    int i = n++;
    for (; i > 0 && steps[i - 1].s < stride * e; --i) steps[i] = steps[i - 1];
    steps[i] = Step{stride * e, lo, hi};
  };
  for (int i = 0; i < 3; ++i) {
    if (a.stride[i] == b.stride[i]) {  // one step: the difference of the places
      add(a.stride[i], 1 - na[i], nb[i] - 1);
    } else {
      add(na[i] > 1 ? a.stride[i] : 0, 1 - na[i], 0);
      add(nb[i] > 1 ? b.stride[i] : 0, 0, nb[i] - 1);
    }
  }
  int tries = 1 << 12;
  return !meets(steps, steps + n, (int64_t)((uintptr_t)b.p - (uintptr_t)a.p), z.dim * e, tries);
}

int check_qk(const void* q, const void* k, const float* qw, const float* kw, const float* table,
             const int32_t* positions, const ss2d_qk_sizes* z, float eps, int dtype) {
  if (!q || !k || !z) return SS2D_ERR_NULL;
  constexpr int64_t most = INT32_MAX;
  if (z->sequences < 1 || z->sequences > most || z->tokens < 1 || z->tokens > most || z->q_heads < 1 ||
      z->q_heads > 65536 || z->k_heads < 1 || z->k_heads > 65536 || z->dim < 1 || z->dim > kMaxQkDim)
    return SS2D_ERR_SHAPE;
  if (z->sequences * z->tokens > most / (z->q_heads + z->k_heads)) return SS2D_ERR_SHAPE;
  if (z->rotated < 0 || z->rotated > z->dim || z->rotated % 2 != 0 || (z->rotated > 0) != (table != nullptr))
    return SS2D_ERR_SHAPE;
  if (table && (z->table_rows < 1 || z->table_rows > most)) return SS2D_ERR_SHAPE;
  if (!(eps >= 0.f && eps < __builtin_inff())) return SS2D_ERR_SHAPE;  // also rejects NaN
  if (!dtype_ok(dtype)) return SS2D_ERR_DTYPE;
  const int64_t e = elem_bytes(dtype);
  for (const Rows& r : {Rows{q, z->q_stride, z->q_heads}, Rows{k, z->k_stride, z->k_heads},
                        Rows{q, z->q_out_stride, z->q_heads}, Rows{k, z->k_out_stride, z->k_heads}})
    if (bytes_of(r, *z, e) < 0) return SS2D_ERR_SHAPE;
  if (misaligned(q, e) || misaligned(k, e) || misaligned(qw, 4) || misaligned(kw, 4) || misaligned(table, 4) ||
      misaligned(positions, 4))
    return SS2D_ERR_ALIGN;
  return SS2D_OK;
}

ss2d::QkArgs qk_args(const ss2d_qk_sizes& z, const void* q, const void* k, const float* qw, const float* kw,
                     const float* table, const int32_t* positions, float eps, int interleaved, int dtype,
                     void* stream) {
  ss2d::QkArgs a{};
  a.side[0].x = q;
  a.side[1].x = k;
  a.side[0].weight = qw;
  a.side[1].weight = kw;
  for (int i = 0; i < 3; ++i) {
    a.side[0].x_stride[i] = z.q_stride[i];
    a.side[1].x_stride[i] = z.k_stride[i];
    a.side[0].y_stride[i] = z.q_out_stride[i];
    a.side[1].y_stride[i] = z.k_out_stride[i];
  }
  a.table = table;
  a.positions = positions;
  a.sequences = z.sequences;
  a.length = z.tokens;
  a.heads[0] = z.q_heads;
  a.heads[1] = z.k_heads;
  a.dim = z.dim;
  a.rotated = z.rotated;
  a.table_rows = z.table_rows;
  a.interleaved = interleaved != 0;
  a.eps = eps;
  a.dtype = dtype;
  a.stream = static_cast<hipStream_t>(stream);
  return a;
}

// The inputs of the norms other than q and k.
struct Others {
  Range r[4];
};
Others others(const float* qw, const float* kw, const float* table, const int32_t* positions, const ss2d_qk_sizes& z) {
  return Others{{{qw, z.dim * 4}, {kw, z.dim * 4}, {table, z.table_rows * z.rotated * 4},
                 {positions, z.sequences * z.tokens * 4}}};
}

}  // namespace

extern "C" {

int64_t ss2d_delta_rule_workspace(const ss2d_delta_sizes* sizes, int packed, int dtype) {
  const int rc = check_attention_sizes(sizes ? &sizes->a : nullptr, packed != 0, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d::DeltaPlan pl = plan_of(sizes->a, packed != 0, dtype, false);
  if (!grid_ok(pl, sizes->a)) return SS2D_ERR_SHAPE;
  return (int64_t)ss2d::delta_workspace_bytes(pl, sizes->a.heads, sizes->a.key_dim, sizes->a.value_dim, dtype);
}

int ss2d_delta_rule(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                    const float* state_in, const int32_t* cu_seqlens, void* o, float* state_out,
                    const ss2d_delta_sizes* sizes, float scale, int dtype, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  if (!q || !k || !v || !log_decay || !beta || !o || !sizes) return SS2D_ERR_NULL;
  const bool packed = cu_seqlens != nullptr;
  int rc = check_attention_sizes(&sizes->a, packed, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d_attention_sizes& z = sizes->a;
  const int64_t e = elem_bytes(dtype);
  const Range in[7] = {{q, extent(z.q_stride, z.sequences, z.tokens, z.groups, z.key_dim, packed, e)},
                       {k, extent(z.k_stride, z.sequences, z.tokens, z.groups, z.key_dim, packed, e)},
                       {v, extent(z.v_stride, z.sequences, z.tokens, z.heads, z.value_dim, packed, e)},
                       {log_decay, extent(z.decay_stride, z.sequences, z.tokens, z.heads, 1, packed, 4)},
                       {beta, extent(sizes->beta_stride, z.sequences, z.tokens, z.heads, 1, packed, 4)},
                       {cu_seqlens, (z.sequences + 1) * 4},
                       {state_in, z.sequences * z.heads * z.key_dim * z.value_dim * 4}};
  for (const Range& r : in)
    if (r.bytes < 0) return SS2D_ERR_SHAPE;
  const Range ro{o, z.tokens * z.heads * z.value_dim * e}, rs{state_out, in[6].bytes};
  const ss2d::DeltaPlan pl = plan_of(z, packed, dtype, false);
  if (!grid_ok(pl, z)) return SS2D_ERR_SHAPE;
  const int64_t need = (int64_t)ss2d::delta_workspace_bytes(pl, z.heads, z.key_dim, z.value_dim, dtype);
  const Range rw{workspace, need};
  for (int i = 0; i < 7; ++i)
    if (overlap(ro, in[i]) || overlap(rw, in[i]) || (i < 6 ? overlap(rs, in[i]) : partly(rs, in[i])))
      return SS2D_ERR_ALIAS;
  if (overlap(ro, rs) || overlap(ro, rw) || overlap(rs, rw)) return SS2D_ERR_ALIAS;
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(o, e) || misaligned(log_decay, 4) ||
      misaligned(beta, 4) || misaligned(state_in, 4) || misaligned(state_out, 4) || misaligned(cu_seqlens, 4))
    return SS2D_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != SS2D_OK) return rc;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  return finish(ss2d::launch_delta(delta_args(q, k, v, log_decay, beta, state_in, cu_seqlens, o, state_out, *sizes,
                                              scale, dtype, workspace, stream),
                                   pl));
}

int64_t ss2d_delta_rule_backward_workspace(const ss2d_delta_sizes* sizes, int packed, int dtype) {
  const int rc = check_attention_sizes(sizes ? &sizes->a : nullptr, packed != 0, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d_attention_sizes& z = sizes->a;
  const ss2d::DeltaPlan pl = plan_of(z, packed != 0, dtype, true);
  if (!backward_grid_ok(pl, z)) return SS2D_ERR_SHAPE;
  return (int64_t)ss2d::delta_backward_workspace_bytes(pl, z.tokens, z.groups, z.heads, z.key_dim, z.value_dim, dtype);
}

int ss2d_delta_rule_backward(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                             const float* state_in, const int32_t* cu_seqlens, const void* d_o,
                             const float* dstate_out, void* dq, void* dk, void* dv, float* dlog_decay, float* dbeta,
                             float* dstate_in, const ss2d_delta_sizes* sizes, float scale, int dtype, void* workspace,
                             int64_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !log_decay || !beta || !d_o || !dq || !dk || !dv || !dlog_decay || !dbeta || !sizes)
    return SS2D_ERR_NULL;
  const bool packed = cu_seqlens != nullptr;
  int rc = check_attention_sizes(&sizes->a, packed, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d_attention_sizes& z = sizes->a;
  const int64_t e = elem_bytes(dtype), st = z.sequences * z.heads * z.key_dim * z.value_dim * 4;
  const Range in[9] = {{q, extent(z.q_stride, z.sequences, z.tokens, z.groups, z.key_dim, packed, e)},
                       {k, extent(z.k_stride, z.sequences, z.tokens, z.groups, z.key_dim, packed, e)},
                       {v, extent(z.v_stride, z.sequences, z.tokens, z.heads, z.value_dim, packed, e)},
                       {log_decay, extent(z.decay_stride, z.sequences, z.tokens, z.heads, 1, packed, 4)},
                       {beta, extent(sizes->beta_stride, z.sequences, z.tokens, z.heads, 1, packed, 4)},
                       {d_o, extent(z.do_stride, z.sequences, z.tokens, z.heads, z.value_dim, packed, e)},
                       {cu_seqlens, (z.sequences + 1) * 4},
                       {state_in, st},
                       {dstate_out, st}};
  for (const Range& r : in)
    if (r.bytes < 0) return SS2D_ERR_SHAPE;
  const ss2d::DeltaPlan pl = plan_of(z, packed, dtype, true);
  if (!backward_grid_ok(pl, z)) return SS2D_ERR_SHAPE;
  const int64_t need = (int64_t)ss2d::delta_backward_workspace_bytes(pl, z.tokens, z.groups, z.heads, z.key_dim,
                                                                     z.value_dim, dtype);
  const Range out[7] = {{dq, z.tokens * z.groups * z.key_dim * e},
                        {dk, z.tokens * z.groups * z.key_dim * e},
                        {dv, z.tokens * z.heads * z.value_dim * e},
                        {dlog_decay, z.tokens * z.heads * 4},
                        {dbeta, z.tokens * z.heads * 4},
                        {dstate_in, st},
                        {workspace, need}};
  for (int i = 0; i < 7; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return SS2D_ERR_ALIAS;
    for (int j = i + 1; j < 7; ++j)
      if (overlap(out[i], out[j])) return SS2D_ERR_ALIAS;
  }
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(d_o, e) || misaligned(dq, e) ||
      misaligned(dk, e) || misaligned(dv, e) || misaligned(log_decay, 4) || misaligned(beta, 4) ||
      misaligned(dlog_decay, 4) || misaligned(dbeta, 4) || misaligned(state_in, 4) || misaligned(dstate_out, 4) ||
      misaligned(dstate_in, 4) || misaligned(cu_seqlens, 4))
    return SS2D_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != SS2D_OK) return rc;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  ss2d::DeltaBackwardArgs a{};
  a.d = delta_args(q, k, v, log_decay, beta, state_in, cu_seqlens, nullptr, nullptr, *sizes, scale, dtype, workspace,
                   stream);
  a.d_o = d_o;
  for (int i = 0; i < 3; ++i) a.do_stride[i] = z.do_stride[i];
  a.dstate_out = dstate_out;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dlog_decay = dlog_decay;
  a.dbeta = dbeta;
  a.dstate_in = dstate_in;
  return finish(ss2d::launch_delta_backward(a, pl));
}

int ss2d_delta_rule_step(const void* q, const void* k, const void* v, const float* log_decay, const float* beta,
                         float* state, const int32_t* index, void* o, int64_t rows, int64_t slots, int64_t groups,
                         int64_t heads, int64_t key_dim, int64_t value_dim, int64_t q_row, int64_t k_row,
                         int64_t v_row, float scale, int dtype, void* stream) {
  if (!beta) return SS2D_ERR_NULL;
  ss2d::StepArgs s{};
  int rc = check_step(q, k, v, log_decay, state, index, o, rows, slots, groups, heads, key_dim, value_dim, q_row, k_row,
                      v_row, scale, dtype, stream, s);
  if (rc != SS2D_OK) return rc;
  const Range rb{beta, rows * heads * 4};
  if (overlap(rb, Range{state, slots * heads * key_dim * value_dim * 4}) ||
      overlap(rb, Range{o, rows * heads * value_dim * elem_bytes(dtype)}))
    return SS2D_ERR_ALIAS;
  if (misaligned(beta, 4)) return SS2D_ERR_ALIGN;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  return finish(ss2d::launch_delta_step(ss2d::DeltaStepArgs{s, beta}));
}

int ss2d_qk_norm(const void* q, const void* k, const float* q_weight, const float* k_weight, const float* rotation,
                 const int32_t* positions, void* q_out, void* k_out, const ss2d_qk_sizes* sizes, float eps,
                 int interleaved, int dtype, void* stream) {
  if (!q_out || !k_out) return SS2D_ERR_NULL;
  int rc = check_qk(q, k, q_weight, k_weight, rotation, positions, sizes, eps, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d_qk_sizes& z = *sizes;
  const int64_t e = elem_bytes(dtype);
  if (misaligned(q_out, e) || misaligned(k_out, e)) return SS2D_ERR_ALIGN;
  const Rows in[2] = {{q, z.q_stride, z.q_heads}, {k, z.k_stride, z.k_heads}};
  const Rows out[2] = {{q_out, z.q_out_stride, z.q_heads}, {k_out, z.k_out_stride, z.k_heads}};
  for (const Rows& o : out)
    if (!apart(o, z)) return SS2D_ERR_SHAPE;
  if (!disjoint(out[0], out[1], z, e)) return SS2D_ERR_ALIAS;
  for (int i = 0; i < 2; ++i) {
    if (!same(out[i], in[i], z) && !disjoint(out[i], in[i], z, e)) return SS2D_ERR_ALIAS;
    if (!disjoint(out[i], in[1 - i], z, e)) return SS2D_ERR_ALIAS;
    for (const Range& r : others(q_weight, k_weight, rotation, positions, z).r)
      if (overlap(Range{out[i].p, bytes_of(out[i], z, e)}, r)) return SS2D_ERR_ALIAS;
  }
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  ss2d::QkArgs a = qk_args(z, q, k, q_weight, k_weight, rotation, positions, eps, interleaved, dtype, stream);
  a.side[0].y = q_out;
  a.side[1].y = k_out;
  return finish(ss2d::launch_qk_norm(a));
}

int64_t ss2d_qk_norm_backward_workspace(const ss2d_qk_sizes* sizes, int dtype) {
  if (!sizes) return SS2D_ERR_NULL;
  static const float one = 1.f;
  const int rc = check_qk(&one, &one, nullptr, nullptr, sizes->rotated > 0 ? &one : nullptr, nullptr, sizes, 0.f, dtype);
  if (rc != SS2D_OK) return rc;
  const int64_t heads[2] = {sizes->q_heads, sizes->k_heads};
  return (int64_t)ss2d::qk_norm_backward_workspace_bytes(sizes->sequences * sizes->tokens, heads, sizes->dim,
                                                         sizes->rotated);
}

int ss2d_qk_norm_backward(const void* q, const void* k, const float* q_weight, const float* k_weight,
                          const float* rotation, const int32_t* positions, const void* dq_out, const void* dk_out,
                          void* dq, void* dk, float* dq_weight, float* dk_weight, const ss2d_qk_sizes* sizes,
                          float eps, int interleaved, int dtype, void* workspace, int64_t workspace_bytes,
                          void* stream) {
  if (!dq_out || !dk_out || !dq || !dk || (dq_weight && !q_weight) || (dk_weight && !k_weight)) return SS2D_ERR_NULL;
  int rc = check_qk(q, k, q_weight, k_weight, rotation, positions, sizes, eps, dtype);
  if (rc != SS2D_OK) return rc;
  const ss2d_qk_sizes& z = *sizes;
  const int64_t e = elem_bytes(dtype), tokens = z.sequences * z.tokens;
  const int64_t need = dq_weight || dk_weight ? ss2d_qk_norm_backward_workspace(sizes, dtype) : 0;
  const Rows in[4] = {{q, z.q_stride, z.q_heads},
                      {k, z.k_stride, z.k_heads},
                      {dq_out, z.q_out_stride, z.q_heads},
                      {dk_out, z.k_out_stride, z.k_heads}};
  const Range out[5] = {{dq, tokens * z.q_heads * z.dim * e},
                        {dk, tokens * z.k_heads * z.dim * e},
                        {dq_weight, z.dim * 4},
                        {dk_weight, z.dim * 4},
                        {need > 0 ? workspace : nullptr, need}};
  const Others more = others(q_weight, k_weight, rotation, positions, z);
  for (int i = 0; i < 5; ++i) {
    for (const Rows& r : in)
      if (overlap(out[i], Range{r.p, bytes_of(r, z, e)})) return SS2D_ERR_ALIAS;
    for (const Range& r : more.r)
      if (overlap(out[i], r)) return SS2D_ERR_ALIAS;
    for (int j = i + 1; j < 5; ++j)
      if (overlap(out[i], out[j])) return SS2D_ERR_ALIAS;
  }
  if (misaligned(dq_out, e) || misaligned(dk_out, e) || misaligned(dq, e) || misaligned(dk, e) ||
      misaligned(dq_weight, 4) || misaligned(dk_weight, 4))
    return SS2D_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, need);
  if (rc != SS2D_OK) return rc;
  rc = check_device();
  if (rc != SS2D_OK) return rc;
  ss2d::QkArgs a = qk_args(z, q, k, q_weight, k_weight, rotation, positions, eps, interleaved, dtype, stream);
  a.side[0].dy = dq_out;
  a.side[1].dy = dk_out;
  a.side[0].y = dq;
  a.side[1].y = dk;
  a.side[0].dweight = dq_weight;
  a.side[1].dweight = dk_weight;
  a.partial = static_cast<float*>(workspace);
  return finish(ss2d::launch_qk_norm_backward(a));
}

}  // extern "C"
