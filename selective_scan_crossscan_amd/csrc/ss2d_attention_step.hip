// Linear attention with a decay per head, one token per row over a cache of
// states:  h = exp(g) h + k v',  o = scale h' q,  h (key_dim x value_dim) fp32.
//
// Bound by memory: a row's states are read and written once (8 bytes per entry
// and nothing else of that size), so one workgroup owns a tile of VT value
// columns of one head, holds all its key rows in registers (16 bytes along the
// value axis per thread and key row), and every load is issued before the first
// is used.  192 rows of 16 heads of 128 x 128 take 94 us (4.3 TB/s) among states
// that no cache holds, one row 5.4 us by itself and 4.2 after another in a graph, the
// latency of its loads and stores.
//
// Rows of one slot are consecutive tokens: the workgroups of the first such row
// run the later ones too, in order, on the state they hold; the others' leave.
#include "ss2d_token_ops.h"

namespace ss2d {
namespace {

using namespace tok;

constexpr int kStepThreads = 256;

struct StepParams {
  const void *q, *k, *v;
  const float* log_decay;
  float* state;
  const int32_t* index;
  void* o;
  int64_t q_row, k_row, v_row, slots;
  int rows, groups, heads, K, V, vtiles;
  float scale;
};

struct __attribute__((packed, aligned(4))) Float4u {
  float x[4];
};

// KP: key_dim rounded up to 64, 128 or 256.
template <typename S, int KP, int VT>
__global__ __launch_bounds__(kStepThreads) void attention_step_kernel(StepParams p) {
  constexpr int TV = VT / 4;               // threads along the value axis
  constexpr int KG = kStepThreads / TV;    // key rows per pass
  constexpr int NK = (KP + KG - 1) / KG;   // passes: key rows per thread
  constexpr int GW = 64 / TV;              // key rows per pass of one wave
  __shared__ float qs[KP], ks[KP];
  __shared__ float part[4][VT];
  __shared__ int next_row;
  const int t = threadIdx.x, tv = t % TV, kg = t / TV;
  const uint32_t block = (uint32_t)block_id(), rest = block / p.vtiles;
  const int vt = block % p.vtiles, head = rest % p.heads, row0 = rest / p.heads;
  if (row0 >= p.rows) return;  // behind the last workgroup
  const int v0 = vt * VT + tv * 4, nv = p.V - v0;  // this thread's columns, and how many exist
  const int group = head / (p.heads / p.groups);
  const int64_t slot = p.index ? p.index[row0] : row0;
  const int64_t head_at = (int64_t)head * p.V + v0;
  if (slot < 0 || slot >= p.slots) {  // padding
    if (kg == 0)
      for (int i = 0; i < 4 && i < nv; ++i)
        store1(static_cast<S*>(p.o) + (int64_t)row0 * p.heads * p.V + head_at + i, 0.f);
    return;
  }
  float* hp = p.state + (slot * p.heads + head) * (int64_t)p.K * p.V + v0;
  float h[NK][4];
#pragma unroll
  for (int j = 0; j < NK; ++j) {
    const int kk = kg + j * KG;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[j][i] = 0.f;
    if (kk < p.K) {
      if (nv >= 4) {
        const Float4u u = *reinterpret_cast<const Float4u*>(hp + (int64_t)kk * p.V);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[j][i] = u.x[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < nv) h[j][i] = hp[(int64_t)kk * p.V + i];
      }
    }
  }
  bool later = false;
  if (p.index) {
    bool earlier = false;
    for (int r = t; r < p.rows; r += kStepThreads) {
      const bool same = p.index[r] == (int32_t)slot;
      earlier |= same && r < row0;
      later |= same && r > row0;
    }
    if (__syncthreads_or(earlier)) return;  // the first row of this slot does them all
    later = __syncthreads_or(later);
  }
  for (int row = row0;;) {
    const S* qrow = static_cast<const S*>(p.q) + row * p.q_row + (int64_t)group * p.K;
    const S* krow = static_cast<const S*>(p.k) + row * p.k_row + (int64_t)group * p.K;
    if (t < KP) {
      qs[t] = t < p.K ? load1(qrow + t) : 0.f;
      ks[t] = t < p.K ? load1(krow + t) : 0.f;
    }
    const S* vrow = static_cast<const S*>(p.v) + row * p.v_row + head_at;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < nv ? load1(vrow + i) : 0.f;
    const float a = expf(clamp_log_decay(p.log_decay[(int64_t)row * p.heads + head]));
    __syncthreads();
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int kk = kg + j * KG;
      const float kv = kk < KP ? ks[kk < KP ? kk : 0] : 0.f, qv = kk < KP ? qs[kk < KP ? kk : 0] : 0.f;
      if (kk < p.K) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[j][i] = fmaf(a, h[j][i], kv * v[i]);
          o[i] = fmaf(qv, h[j][i], o[i]);
        }
      }
    }
    // sum over the key rows: lanes TV apart, then the four waves
#pragma unroll
    for (int m = TV; m < 64; m <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], m);
    if ((t & 63) < TV)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[t >> 6][tv * 4 + i] = o[i];
    __syncthreads();
    if (t < VT && vt * VT + t < p.V) {
      const float s = (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]);
      store1(static_cast<S*>(p.o) + ((int64_t)row * p.heads + head) * p.V + vt * VT + t, s * p.scale);
    }
    if (!later) break;
    if (t == 0) next_row = p.rows;
    __syncthreads();
    for (int r = row + 1 + t; r < p.rows; r += kStepThreads)
      if (p.index[r] == (int32_t)slot) {
        atomicMin(&next_row, r);
        break;
      }
    __syncthreads();
    row = next_row;
    __syncthreads();  // next_row and the sums have been read
    if (row >= p.rows) break;
  }
  static_assert(GW >= 1, "a wave holds whole key rows");
#pragma unroll
  for (int j = 0; j < NK; ++j) {
    const int kk = kg + j * KG;
    if (kk < p.K) {
      if (nv >= 4) {
        Float4u u;
#pragma unroll
        for (int i = 0; i < 4; ++i) u.x[i] = h[j][i];
        *reinterpret_cast<Float4u*>(hp + (int64_t)kk * p.V) = u;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < nv) hp[(int64_t)kk * p.V + i] = h[j][i];
      }
    }
  }
}

template <typename S, int VT>
void launch_step_v(const StepArgs& a, StepParams p) {
  p.vtiles = (int)((a.value_dim + VT - 1) / VT);
  const dim3 grid = grid_of(a.rows * a.heads * p.vtiles, kStepThreads), block(kStepThreads);
  if (a.key_dim <= 64)
    attention_step_kernel<S, 64, VT><<<grid, block, 0, a.stream>>>(p);
  else if (a.key_dim <= 128)
    attention_step_kernel<S, 128, VT><<<grid, block, 0, a.stream>>>(p);
  else
    attention_step_kernel<S, 256, VT><<<grid, block, 0, a.stream>>>(p);
}

template <typename S>
hipError_t launch_step_s(const StepArgs& a) {
  StepParams p{a.q,     a.k,     a.v,       a.log_decay,  a.state,       a.index,        a.o,
               a.q_row, a.k_row, a.v_row,   a.slots,      (int)a.rows,   (int)a.groups,  (int)a.heads,
               (int)a.key_dim,   (int)a.value_dim, 0,     a.scale};
  // Tiles of 16 columns spread a few rows over four times as many CUs, tiles of 64 read 256 bytes at once.  16 heads
  // of 128 x 128, one launch after another in a graph, tiles of 16 against 64: one row 4.2 us (5.0), two 4.9 (5.1), four 6.9 (5.8), 192 134 (95).
  if (a.rows * a.heads * ((a.value_dim + 63) / 64) < 128)
    launch_step_v<S, 16>(a, p);
  else
    launch_step_v<S, 64>(a, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_step(const StepArgs& a) {
  return a.dtype == 1 ? launch_step_s<uint16_t>(a) : launch_step_s<float>(a);
}

}  // namespace ss2d
