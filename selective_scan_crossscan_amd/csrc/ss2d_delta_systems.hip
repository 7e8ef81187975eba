// The gated delta rule: the systems of all chunks, which do not depend on the state.
//
// With L_ij = exp(G_i - G_j) k_i . k_j for j < i, b = beta and P_ij = scale exp(G_i - G_j) q_i . k_j for j <= i, per
// chunk of C tokens and head
//   forward    N = (1 + L diag(b))^-1 - 1 and P;
//   gradients  the same N, and ((1 + diag(b) L)^-1)' - 1 and P',
// in fp32, as fragments in the order in which the walks read them, the ones on the diagonal left to those.  The walks take
// all 24 bits in three bf16 parts: with two of an inverse states were up to 1.6e-6 off where elementary fp32 operations are
// 1.8e-7; with two of P, of the replaced values and of the state towards an output bf16 outputs were 1.1e-4 from those of
// elementary fp32 operations in the norm, with three 3.8e-5.
//
// A triangle is inverted in blocks of 16.  A diagonal block by substitution: a lane holds one row of the inverse and
// the block's entries are read by all lanes at once; as stable as the system is, where a series of powers would cancel
// (keys that repeat: powers up to 6435 of entries up to 1).  The other blocks X_tw = -X_tt sum_c Z_tc X_cw on the
// matrix cores in fp32 (16x16x4), one block column per wave: a result tile is the next product's second operand as it
// lies.
//
// Bound by memory: 16 x 2048 tokens, 16 heads of 128 in bf16, take 90 us: 32 KiB read and 24 KiB written per chunk and
// head at 5.2 TB/s.
#include <type_traits>

#include "ss2d_delta.h"

namespace ss2d {
namespace {

using namespace tok;

template <int C>
struct Triangle {
  static constexpr int kStride = C + 4, kDiagStride = 20;  // rows of 16 bytes, spread over the banks
  __attribute__((aligned(16))) float z[C * kStride];
  __attribute__((aligned(16))) float d[C / 16][16 * kDiagStride];
};

// The inverse X of 1 + Z, Z the strictly upper (lower) triangle of m.z: x[t] gets the rows 16 t + 4 g + r of column
// 16 w + l, w this wave.  Barriers inside: all waves call it, after m.z is written.
template <int C, bool UPPER>
__device__ __forceinline__ void invert(Triangle<C>& m, int w, f32x4 (&x)[C / 16]) {
  constexpr int NI = C / 16;
  const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  __syncthreads();
  {
    // lane l's row of the diagonal block's inverse: x_q + sum_c x_c Z_cq = (q == l), columns in order
    float row[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) row[q] = q == l ? 1.f : 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      const int c = UPPER ? s : 15 - s;
      const float* zc = &m.z[(w * 16 + c) * m.kStride + w * 16];
#pragma unroll
      for (int q = 0; q < 16; q += 4) {
        if (UPPER ? q + 3 > c : q < c) {
          const f32x4 z = *reinterpret_cast<const f32x4*>(zc + q);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (UPPER ? q + r > c : q + r < c) row[q + r] = fmaf(-row[c], z[r], row[q + r]);
        }
      }
    }
    if (g == 0)
#pragma unroll
      for (int q = 0; q < 16; q += 4)
        *reinterpret_cast<f32x4*>(&m.d[w][l * m.kDiagStride + q]) = f32x4{row[q], row[q + 1], row[q + 2], row[q + 3]};
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NI; ++t) x[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // block column w: its diagonal block, then outwards
#pragma unroll
  for (int s = 0; s < NI; ++s) {
    const int t = UPPER ? NI - 1 - s : s;  // x is indexed by constants
    if (t == w) {
#pragma unroll
      for (int r = 0; r < 4; ++r) x[t][r] = m.d[t][(4 * g + r) * m.kDiagStride + l];
    } else if (UPPER ? t < w : t > w) {
      f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NI; ++c)
        if (UPPER ? c > t && c <= w : c < t && c >= w) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(&m.z[(t * 16 + l) * m.kStride + c * 16 + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) y = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], x[c][r], y, 0, 0, 0);
        }
      const f32x4 a = *reinterpret_cast<const f32x4*>(&m.d[t][l * m.kDiagStride + 4 * g]);
      f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 4; ++r) v = __builtin_amdgcn_mfma_f32_16x16x4f32(-a[r], y[r], v, 0, 0, 0);
      x[t] = v;
    }
  }
}

// The diagonal's ones are the walks'.
template <int NI>
__device__ __forceinline__ void drop_ones(int w, f32x4 (&x)[NI]) {
  const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
#pragma unroll
  for (int t = 0; t < NI; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) x[t][r] = t == w && 4 * g + r == l ? 0.f : x[t][r];
}

// Two stacked tiles to memory as fragment `at`.
__device__ __forceinline__ void put_frag(char* out, int at, const f32x4& a, const f32x4& b) {
  f32x4* to = reinterpret_cast<f32x4*>(out) + (at * 64 + (threadIdx.x & 63)) * 2;
  to[0] = a;
  to[1] = b;
}

// exp(G_i - G_j) for i .. i + 3
template <int C>
__device__ __forceinline__ f32x4 to4(const Decays<C>& d, int i, int j) {
  const f32x4 w = *reinterpret_cast<const f32x4*>(&d.whole[i]), f = *reinterpret_cast<const f32x4*>(&d.frac[i]);
  const float wj = d.whole[j], fj = d.frac[j];
  f32x4 e;
#pragma unroll
  for (int r = 0; r < 4; ++r) e[r] = __builtin_amdgcn_exp2f((w[r] - wj) + (f[r] - fj));
  return e;
}

template <typename E, int C, int KP, bool BACK, bool TINY>
__global__ __launch_bounds__(C * 4) void delta_systems(DeltaParams p) {
  constexpr int NI = C / 16, THREADS = NI * 64;
  using S = Systems<E, C>;
  __shared__ Tile<E, C, KP> ks;
  __shared__ union Rest {  // the queries are done with before the triangle is written
    Tile<E, C, KP> qs;
    Triangle<C> m;
    __device__ Rest() {}
  } rest;
  auto& qs = rest.qs;
  auto& m = rest.m;
  __shared__ Decays<C> dec;
  __shared__ float bs[C];
  const int w = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const uint32_t block = (uint32_t)block_id();
  if (block >= p.blocks) return;
  const int head = block % p.heads;
  const int64_t chunk = block / p.heads;
  Segment seg;
  if (!find_segment(p.chunk_map, chunk, seg)) return;
  const int n = (int)(seg.end - seg.begin);
  if (n == 0) return;
  const int group = head / (p.heads / p.groups);
  const int64_t token0 = (p.map.cu ? seg.start : 0) + seg.begin, sq = p.map.cu ? 0 : seg.s;
  {
    TileLoad<E, C, KP, 16, THREADS, TINY> q, k;
    q.load(static_cast<const E*>(p.q) + sq * p.q_stride[0] + token0 * p.q_stride[1] + group * p.q_stride[2], p.q_stride[1], n, p.K);
    k.load(static_cast<const E*>(p.k) + sq * p.k_stride[0] + token0 * p.k_stride[1] + group * p.k_stride[2], p.k_stride[1], n, p.K);
    if (w == 0) {
      const int64_t t = token0 + min(lane, n - 1);
      const float x = p.g[sq * p.g_stride[0] + t * p.g_stride[1] + head * p.g_stride[2]];
      const float b = p.beta[sq * p.b_stride[0] + t * p.b_stride[1] + head * p.b_stride[2]];
      if (lane < C) bs[lane] = lane < n ? b : 0.f;
      scan_decays<C>(lane < n ? x : 0.f, dec);
    }
    q.store(qs, n, p.K);
    k.store(ks, n, p.K);
  }
  __syncthreads();
  char* out = p.systems + (int64_t)block * (BACK ? S::kBackward : S::kForward);
  const int i0 = w * 16 + l;

  // P by tiles: rows j of column i in tile column w, for gradients rows i of column j in tile column w
  {
    f32x4 s[NI];
#pragma unroll
    for (int t = 0; t < NI; ++t) {
      s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (BACK ? t >= w : t <= w) {
#pragma unroll
        for (int c = 0; c < KP; c += 32)
          s[t] = BACK ? mma(frag_row(qs, t * 16 + l, c), frag_row(ks, i0, c), s[t])
                      : mma(frag_row(ks, t * 16 + l, c), frag_row(qs, i0, c), s[t]);
        const f32x4 e = BACK ? to4(dec, t * 16 + 4 * g, i0) : dec.between4(i0, t * 16 + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = t * 16 + 4 * g + r;
          const float v = s[t][r] * (p.scale * e[r]);
          s[t][r] = (BACK ? at >= i0 : at <= i0) ? v : 0.f;
        }
      }
    }
#pragma unroll
    for (int pair = 0; pair < NI / 2; ++pair)
      if (BACK ? pair >= w / 2 : pair <= w / 2) {
        if (BACK)
          put_frag(out + 2 * S::kOne, S::upper(w, pair), s[2 * pair], s[2 * pair + 1]);
        else
          put_frag(out + S::kOne, S::lower(w, pair), s[2 * pair], s[2 * pair + 1]);
      }
  }
  __syncthreads();  // the queries have been read
  // (1 + L diag(b))^-1 transposed, an upper triangle: rows j, columns i
#pragma unroll
  for (int t = 0; t < NI; ++t)
    if (t <= w) {
      f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KP; c += 32) s = mma(frag_row(ks, i0, c), frag_row(ks, t * 16 + l, c), s);
      const f32x4 e = to4(dec, w * 16 + 4 * g, t * 16 + l);
      const float b = bs[t * 16 + l];
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] *= e[r] * b;
      *reinterpret_cast<f32x4*>(&m.z[(t * 16 + l) * m.kStride + w * 16 + 4 * g]) = s;
    }
  f32x4 x[NI];
  invert<C, true>(m, w, x);
  drop_ones(w, x);
#pragma unroll
  for (int pair = 0; pair < NI / 2; ++pair)
    if (pair <= w / 2)
      put_frag(out, S::lower(w, pair), x[2 * pair], x[2 * pair + 1]);
  if (!BACK) return;
  // (1 + diag(b) L)^-1, a lower triangle: rows i, columns j
  __syncthreads();  // the first triangle has been read
#pragma unroll
  for (int t = 0; t < NI; ++t)
    if (t <= w) {
      f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KP; c += 32) s = mma(frag_row(ks, t * 16 + l, c), frag_row(ks, i0, c), s);
      const f32x4 e = dec.between4(i0, t * 16 + 4 * g);
      const float b = bs[i0];
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] *= e[r] * b;
      *reinterpret_cast<f32x4*>(&m.z[i0 * m.kStride + t * 16 + 4 * g]) = s;
    }
  invert<C, false>(m, w, x);
  drop_ones(w, x);
#pragma unroll
  for (int pair = 0; pair < NI / 2; ++pair)
    if (pair >= w / 2)
      put_frag(out + S::kOne, S::upper(w, pair), x[2 * pair], x[2 * pair + 1]);
}

template <typename E, int C, bool BACK>
void launch(const DeltaParams& p, const DeltaPlan& pl, hipStream_t st) {
  const dim3 grid = grid_of(p.blocks, C * 4), block(C * 4);
  if (pl.a.tiny && pl.a.kp == 32)
    delta_systems<E, C, 32, BACK, true><<<grid, block, 0, st>>>(p);  // keys of 16 bytes or more need no care here
  else if (pl.a.kp == 32)
    delta_systems<E, C, 32, BACK, false><<<grid, block, 0, st>>>(p);
  else if (pl.a.kp == 64)
    delta_systems<E, C, 64, BACK, false><<<grid, block, 0, st>>>(p);
  else if (pl.a.kp == 128)
    delta_systems<E, C, 128, BACK, false><<<grid, block, 0, st>>>(p);
  else
    delta_systems<E, C, 256, BACK, false><<<grid, block, 0, st>>>(p);
}

}  // namespace

int64_t system_bytes(const DeltaPlan& pl, int dtype) {
  if (dtype == 1) return pl.backward ? Systems<uint16_t, 64>::kBackward : Systems<uint16_t, 64>::kForward;
  return pl.backward ? Systems<float, 32>::kBackward : Systems<float, 32>::kForward;
}

hipError_t launch_delta_systems(const DeltaParams& q, const DeltaPlan& pl, int dtype, hipStream_t st) {
  DeltaParams p = q;
  p.blocks = (uint32_t)(pl.a.chunks * p.heads);
  if (dtype == 1)
    pl.backward ? launch<uint16_t, 64, true>(p, pl, st) : launch<uint16_t, 64, false>(p, pl, st);
  else
    pl.backward ? launch<float, 32, true>(p, pl, st) : launch<float, 32, false>(p, pl, st);
  return hipGetLastError();
}

}  // namespace ss2d
