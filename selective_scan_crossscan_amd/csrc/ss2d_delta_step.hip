// The gated delta rule, one token per row over a cache of states (key_dim x value_dim, fp32):
//   h <- a h,   u = b (v - h' k),   h <- h + k u',   o = scale h' q.
//
// Bound by memory: a row's states are read and written once, so one workgroup owns a tile of VT value columns of one
// head and holds all its key rows in registers, 16 bytes along the value axis per thread and key row, every load issued
// before the first is used.  The output needs no second sum over the keys after the update: h' q and h' k are summed
// together before it, and o = scale (h' q + (q . k) u).  192 rows of 16 heads of 128 x 128 take 96 us, 4.2 TB/s.
//
// Rows of one slot are consecutive tokens: the workgroups of the first such row run the later ones too, in order, on
// the state they hold; the others' leave.
#include "ss2d_delta.h"

namespace ss2d {
namespace {

using namespace tok;

// (Tiles of 16 columns, four times the workgroups, are no faster for few rows either: one row of 16 heads of 128 6.6 us,
// 6.3 with 64; 8 rows 12.4 and 7.9.)
constexpr int kStepThreads = 256, kStepColumns = 64;

struct StepParams {
  const void *q, *k, *v;
  const float *log_decay, *beta;
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
template <typename S, int KP>
__global__ __launch_bounds__(kStepThreads) void delta_step_kernel(StepParams p) {
  constexpr int VT = kStepColumns, TV = VT / 4;               // threads along the value axis
  constexpr int KG = kStepThreads / TV;    // key rows per pass
  constexpr int NK = (KP + KG - 1) / KG;   // passes: key rows per thread
  __shared__ float qs[KP], ks[KP];
  __shared__ __attribute__((aligned(16))) float seen[4][VT], asked[4][VT];  // h' k, h' q by wave
  __shared__ float both[4];                                                  // q . k by wave
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
    const float b = p.beta[(int64_t)row * p.heads + head];
    __syncthreads();
    float hk[4] = {0.f, 0.f, 0.f, 0.f}, hq[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int kk = kg + j * KG;
      const float kv = kk < KP ? ks[kk < KP ? kk : 0] : 0.f, qv = kk < KP ? qs[kk < KP ? kk : 0] : 0.f;
      qk = fmaf(qv, kv, qk);
      if (kk < p.K)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[j][i] *= a;
          hk[i] = fmaf(kv, h[j][i], hk[i]);
          hq[i] = fmaf(qv, h[j][i], hq[i]);
        }
    }
    // sums over the key rows: lanes TV apart, then the four waves
#pragma unroll
    for (int m = TV; m < 64; m <<= 1) {
      qk += __shfl_xor(qk, m);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hk[i] += __shfl_xor(hk[i], m);
        hq[i] += __shfl_xor(hq[i], m);
      }
    }
    if ((t & 63) < TV) {
      *reinterpret_cast<f32x4*>(&seen[t >> 6][tv * 4]) = f32x4{hk[0], hk[1], hk[2], hk[3]};
      *reinterpret_cast<f32x4*>(&asked[t >> 6][tv * 4]) = f32x4{hq[0], hq[1], hq[2], hq[3]};
    }
    if ((t & 63) == 0) both[t >> 6] = qk;
    __syncthreads();
    f32x4 s = *reinterpret_cast<const f32x4*>(&seen[0][tv * 4]);
#pragma unroll
    for (int w = 1; w < 4; ++w) s += *reinterpret_cast<const f32x4*>(&seen[w][tv * 4]);
    float u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = b * (v[i] - s[i]);
    if (kg == 0) {
      f32x4 o = *reinterpret_cast<const f32x4*>(&asked[0][tv * 4]);
#pragma unroll
      for (int w = 1; w < 4; ++w) o += *reinterpret_cast<const f32x4*>(&asked[w][tv * 4]);
      const float all = (both[0] + both[1]) + (both[2] + both[3]);
      S* to = static_cast<S*>(p.o) + (int64_t)row * p.heads * p.V + head_at;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < nv) store1(to + i, p.scale * fmaf(all, u[i], o[i]));
    }
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int kk = kg + j * KG;
      const float kv = kk < KP ? ks[kk < KP ? kk : 0] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = fmaf(kv, u[i], h[j][i]);
    }
    if (!later) break;
    if (t == 0) next_row = p.rows;
    __syncthreads();  // also: keys, queries and sums have been read
    for (int r = row + 1 + t; r < p.rows; r += kStepThreads)
      if (p.index[r] == (int32_t)slot) {
        atomicMin(&next_row, r);
        break;
      }
    __syncthreads();
    row = next_row;
    __syncthreads();  // next_row has been read
    if (row >= p.rows) break;
  }
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

template <typename S>
hipError_t launch_step_s(const DeltaStepArgs& x) {
  const StepArgs& a = x.s;
  const StepParams p{a.q,     a.k,     a.v,     a.log_decay, x.beta,        a.state,          a.index,
                     a.o,     a.q_row, a.k_row, a.v_row,     a.slots,       (int)a.rows,      (int)a.groups,
                     (int)a.heads, (int)a.key_dim, (int)a.value_dim,
                     (int)((a.value_dim + kStepColumns - 1) / kStepColumns), a.scale};
  const dim3 grid = grid_of(a.rows * a.heads * p.vtiles, kStepThreads), block(kStepThreads);
  if (a.key_dim <= 64)
    delta_step_kernel<S, 64><<<grid, block, 0, a.stream>>>(p);
  else if (a.key_dim <= 128)
    delta_step_kernel<S, 128><<<grid, block, 0, a.stream>>>(p);
  else
    delta_step_kernel<S, 256><<<grid, block, 0, a.stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& x) {
  return x.s.dtype == 1 ? launch_step_s<uint16_t>(x) : launch_step_s<float>(x);
}

}  // namespace ss2d
