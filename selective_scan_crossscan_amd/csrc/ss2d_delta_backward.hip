// The gated delta rule: the gradients (notation of ss2d_delta.h).
//
// With D the gradient of the state behind a chunk:
//   dU = P' dO + w K D,   dF = ((1 + diag(b) L)^-1)' dU,   dV = dZ = b dF,   db_j = E_j . dF_j,
//   D <- exp(G_last) D + Q' (scale exp(G) dO) - K' (exp(G) dZ)   (the chunk before's D);
// with the states H before the chunk, X = scale exp(G_i - G_j) (do_i . u_j) for j <= i and
// Y = -exp(G_i - G_j) (dz_i . u_j) for j < i:
//   dq_i = scale exp(G_i) H do_i + sum_j X_ij k_j,
//   dk_i = w_i D u_i - exp(G_i) H dz_i + sum_j X_ji q_j + sum_j (Y_ij + Y_ji) k_j.
// The decay's gradient: a decay before token t scales everything that passes from before t to t or behind it, and
// scaling o, v and the state together changes nothing, so inside a chunk
//   dg_t = sum_{i >= t} (q_i . dq_i - dv_i . v_i) + <H_next, D>,
//   <H_next, D> = exp(G_last) <H, D> + sum_j u_j . (w K D)_j,
// formed anew in every chunk: summed on to the sequence's end, each token's own terms, which cancel, would leave their
// errors to all tokens before.
//
// Three steps.  The states before all chunks and the errors E by the forward's walk; D behind all chunks and dF by a
// walk backwards, which is the same kind of recurrence (a wave owns value columns and needs nothing from other waves);
// all else chunk by chunk, in any order, with no walk to wait for.  A segment's map of D is the transpose of its map of
// the state, so cut sequences' maps are formed once.
#include <type_traits>

#include "ss2d_delta.h"

namespace ss2d {
namespace {

using namespace tok;

struct BackParams {
  DeltaParams d;
  const void* d_o;
  int64_t do_stride[3];
  const float* dstate_out;  // or null
  float* seg_dstate;        // (slot, head, K, V): what a segment adds, after the carry the gradient behind it
  float* chunk_dstate;      // (chunk, head, K, V): D behind every chunk
  float* df;                // (token, head, V)
  float* inner;             // (chunk, head, 16-column tile): parts of sum_j u_j . (w K D)_j
  void *dq, *dk, *dv;
  float *dq_part, *dk_part;  // (part, token, group, K), or null: dq and dk themselves
  float *dg, *dbeta;
  float* dstate_in;         // or null
  int columns;              // 16-column tiles of `inner`
  uint32_t blocks;
};

// ------------------------------------------------------------------ the walk backwards
template <typename E, int C, int KP, int VT, bool SUM, bool TINY>
__global__ __launch_bounds__(VT * 4, VT == 64 ? 1 : 2) void delta_walk_back(BackParams b) {
  const DeltaParams& p = b.d;
  constexpr int NW = VT / 16, THREADS = NW * 64, NI = C / 16, NK = KP / 16, PF = kFullParts<E>;
  using S = Systems<E, C>;
  constexpr int PN = S::kParts;
  constexpr int kSystem = S::kBackward - S::kInverse;  // the transposed inverse and P'
  constexpr int kPieces = (kSystem / 16 + THREADS - 1) / THREADS;
  __shared__ Tile<E, C, KP, 32> qs, ks;
  __shared__ Tile<E, C, VT, 32> ds;
  __shared__ __attribute__((aligned(16))) char sys[kSystem];
  __shared__ Rates<C> rates;

  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  uint32_t unit, tile;
  if (!spread((uint32_t)block_id(), b.blocks, p.vtiles, unit, tile)) return;
  const int vt = tile, head = unit % p.heads;
  const int64_t slot = unit / p.heads;
  Segment seg;
  if (!find_segment(p.map, slot, seg)) return;
  if (SUM && seg.begin == 0) return;  // of no use
  const int group = head / (p.heads / p.groups);
  const int K = p.K, v0 = vt * VT, nv = min(p.V - v0, VT), v = wave * 16 + l;
  const bool active = wave * 16 < nv;
  const int64_t token0 = p.map.cu ? seg.start : 0, sq = p.map.cu ? 0 : seg.s;
  const E* qb = static_cast<const E*>(p.q) + sq * p.q_stride[0] + token0 * p.q_stride[1] + group * p.q_stride[2];
  const E* kb = static_cast<const E*>(p.k) + sq * p.k_stride[0] + token0 * p.k_stride[1] + group * p.k_stride[2];
  const E* db = static_cast<const E*>(b.d_o) + sq * b.do_stride[0] + token0 * b.do_stride[1] + head * b.do_stride[2] + v0;
  const float* gb = p.g + sq * p.g_stride[0] + token0 * p.g_stride[1] + head * p.g_stride[2];
  const float* bb = p.beta + sq * p.b_stride[0] + token0 * p.b_stride[1] + head * p.b_stride[2];
  const int64_t chunk0 = chunk_number<C>(p.map, seg, seg.begin);
  const char* sb = p.systems + (chunk0 * p.heads + head) * p.system_stride + S::kInverse;
  const int64_t sstep = p.heads * p.system_stride;

  struct Chunk {
    TileLoad<E, C, KP, 32, THREADS, TINY> q, k;
    TileLoad<E, C, VT, 32, THREADS, TINY> d;
    uint4 s[kPieces];
    float g, b;
  };
  auto fetch = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.q.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    x.d.load(db + at * b.do_stride[1], b.do_stride[1], n, nv);
    const char* from = sb + (at - seg.begin) / C * sstep;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      x.s[i] = *reinterpret_cast<const uint4*>(from + min((int)threadIdx.x + i * THREADS, kSystem / 16 - 1) * 16);
    const int64_t t = at + min(lane, n - 1);
    x.g = gb[t * p.g_stride[1]];
    x.b = bb[t * p.b_stride[1]];
  };
  auto land = [&](const Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.q.store(qs, n, K);
    x.k.store(ks, n, K);
    x.d.store(ds, n, nv);
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (kSystem / 16 % THREADS == 0 || threadIdx.x + i * THREADS < kSystem / 16)
        *reinterpret_cast<uint4*>(sys + (threadIdx.x + i * THREADS) * 16) = x.s[i];
    if (wave == 0) scan_rates<C>(lane < n ? x.g : 0.f, lane < n ? x.b : 0.f, rates);
  };
  const int64_t chunks = (seg.end - seg.begin + C - 1) / C;
  Chunk first;  // on its way while the gradient is read
  if (chunks > 0) fetch(first, seg.begin + (chunks - 1) * C);

  // D: rows 16 kt + 4 g + r, column v
  f32x4 d[NK];
  const int64_t kv = (int64_t)K * p.V, sh = (slot * p.heads + head) * kv, qh = ((int64_t)seg.s * p.heads + head) * kv;
  const float* from = SUM ? nullptr : !seg.last ? b.seg_dstate + sh : b.dstate_out ? b.dstate_out + qh : nullptr;
#pragma unroll
  for (int kt = 0; kt < NK; ++kt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int k = kt * 16 + 4 * g + r;
      const float x = from ? from[(int64_t)min(k, K - 1) * p.V + v0 + min(v, nv - 1)] : 0.f;
      d[kt][r] = k < K && v < nv ? x : 0.f;
    }
  if (chunks > 0) land(first, seg.begin + (chunks - 1) * C);
  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int64_t at = seg.begin + c * C;
    const int n = (int)min((int64_t)C, seg.end - at);
    __syncthreads();  // the chunk has landed
    Chunk next;  // as in the forward
    const int64_t ahead = c > 0 ? at - C : at;
    fetch(next, ahead);
    const int64_t chunk = (chunk0 + c) * p.heads + head;
    if (active) {
      const uint32_t step = (uint32_t)(p.heads * p.V);
      const int64_t rows = ((seg.start + at) * p.heads + head) * p.V + v0;
      f32x4 e[NI];
      if (!SUM) {
        float* to = b.chunk_dstate + chunk * kv + v0;
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int k = kt * 16 + 4 * g + r;
            if (k < K && v < nv) to[k * p.V + v] = d[kt][r];
          }
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            e[x][r] = p.errors[rows + (uint32_t)min(x * 16 + 4 * g + r, n - 1) * step + min(v, nv - 1)];
      }
      // dU = w K D + P' dO
      f32x4 u[NI];
#pragma unroll
      for (int x = 0; x < NI; ++x) u[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int a = 0; a < NK; a += 2) {
        Frag<E> f[PF];
        float y[8];
        stack(d[a], d[a + 1], y);
        split_parts(y, f);
        Frag<E> k[NI];
#pragma unroll
        for (int x = 0; x < NI; ++x) k[x] = frag_row_split(ks, x * 16 + l, a * 16);
#pragma unroll
        for (int q = PF - 1; q >= 0; --q)  // independent products next to each other
#pragma unroll
          for (int x = 0; x < NI; ++x) u[x] = mma(k[x], f[q], u[x]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int x = 0; x < NI; ++x) u[x] *= rates.four(&rates.left[x * 16 + 4 * g]);
      if (!SUM) {
        float s = 0.f;  // errors behind the end and outside the columns meet a 0
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const f32x4 be = rates.four(&rates.beta[x * 16 + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) s = x * 16 + 4 * g + r < n && v < nv ? fmaf(be[r] * e[x][r], u[x][r], s) : s;
        }
        s = wave_sum(s);
        if (lane == 0) b.inner[chunk * b.columns + vt * NW + wave] = s;
      }
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const Frag<E> f = frag_col_split(ds, j * 16, wave * 16);
#pragma unroll
        for (int q = PF - 1; q >= 0; --q)
#pragma unroll
          for (int x = 0; x < j + 2; ++x)
            u[x] = mma(system_frag<E>(sys + S::kInverse + (S::upper(x, j / 2) * PF + q) * S::kFragBytes), f, u[x]);
      }
      __builtin_amdgcn_sched_barrier(0);
      // dF = dU + N' dU
      f32x4 z[NI];
#pragma unroll
      for (int x = 0; x < NI; ++x) z[x] = u[x];
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> f[PN], a[NI][PN];
        float y[8];
#pragma unroll
        for (int x = 0; x < j + 2; ++x)
#pragma unroll
          for (int q = 0; q < PN; ++q) a[x][q] = system_frag<E>(sys + (S::upper(x, j / 2) * PN + q) * S::kFragBytes);
        stack(u[j], u[j + 1], y);
        split_parts(y, f);
        j == 0 ? mma_parts<0, 2>(a, f, z) : mma_parts<0, NI>(a, f, z);
      }
      if (!SUM) {
        float* to = b.df + rows;
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = x * 16 + 4 * g + r;
            if (i < n && v < nv) to[(uint32_t)i * step + v] = z[x][r];
          }
      }
      __builtin_amdgcn_sched_barrier(0);
      // D for the chunk before
      const float all = rates.since[C - 1];
#pragma unroll
      for (int kt = 0; kt < NK; ++kt) d[kt] *= all;
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const f32x4 f0 = rates.four(&rates.since[j * 16 + 4 * g]), f1 = rates.four(&rates.since[j * 16 + 16 + 4 * g]);
        Frag<E> fo[PF], fz[PF];
        float y[8];
        frag_values(frag_col_split(ds, j * 16, wave * 16), y);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          y[r] *= p.scale * f0[r];
          y[4 + r] *= p.scale * f1[r];
        }
        split_parts(y, fo);
        const f32x4 b0 = rates.four(&rates.beta[j * 16 + 4 * g]), b1 = rates.four(&rates.beta[j * 16 + 16 + 4 * g]);
        stack(z[j] * (b0 * -f0), z[j + 1] * (b1 * -f1), y);
        split_parts(y, fz);
#pragma unroll
        for (int kt = 0; kt < NK; kt += 2) {
          Frag<E> q[2], k[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            q[i] = frag_col_split(qs, j * 16, (kt + i) * 16);
            k[i] = frag_col_split(ks, j * 16, (kt + i) * 16);
          }
#pragma unroll
          for (int n = PF - 1; n >= 0; --n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) d[kt + i] = mma(q[i], fo[n], d[kt + i]);
#pragma unroll
            for (int i = 0; i < 2; ++i) d[kt + i] = mma(k[i], fz[n], d[kt + i]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else if (!SUM && lane == 0) {
      b.inner[chunk * b.columns + vt * NW + wave] = 0.f;
    }
    __syncthreads();  // the chunk has been read
    land(next, ahead);
  }
  float* to = SUM ? b.seg_dstate + sh : seg.begin == 0 && b.dstate_in ? b.dstate_in + qh : nullptr;
  if (to)
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = kt * 16 + 4 * g + r;
        if (k < K && v < nv) to[(int64_t)k * p.V + v0 + v] = d[kt][r];
      }
}

// ------------------------------------------------------------------ chunk by chunk
// Four values into N LDS tiles' rows, in parts.
template <int N, int R, int CC, int PAD>
__device__ __forceinline__ void put4_parts(Tile<uint16_t, R, CC, PAD> (&m)[N], int at, f32x4 x) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t w[2] = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    __builtin_memcpy(__builtin_assume_aligned(&m[n].e[at], 8), w, 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] -= __uint_as_float(w[i] << 16);
      x[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <int R, int CC, int PAD>
__device__ __forceinline__ void put4_parts(Tile<float, R, CC, PAD> (&m)[1], int at, f32x4 x) {
  put4(&m[0].e[at], x);
}

// One workgroup per chunk and head; a wave owns key columns wave, wave + NW, ... by 16 and their dq and dk, transposed
// (rows k, columns token); the values are gone through in tiles of 64 columns.
template <typename E, int C, int KP, int NW, bool TINY>
__global__ __launch_bounds__(NW * 64) void delta_gradients(BackParams b) {
  const DeltaParams& p = b.d;
  constexpr int THREADS = NW * 64, NI = C / 16, NK = KP / 16, VT = 64, NV = VT / 16, PF = kFullParts<E>;
  constexpr int OK = (NK + NW - 1) / NW;
  constexpr int PB = PF > 1 ? 2 : 1;  // parts of U and dZ towards dk, whose products round one operand only
  constexpr int JS = NW / NI < NI ? NW / NI : NI;  // waves that share 16 tokens' scores
  constexpr int TT = THREADS / C, PC = VT / TT;    // threads per token, each with PC columns of values
  static_assert(NW >= NI && PC % 4 == 0, "score tiles and columns are dealt evenly");
  struct Values {
    Tile<E, C, VT> d, z[PB], u[PF];
  };
  struct Scores {
    Tile<E, C, C, 32> x[PF], y;
  };
  __shared__ Tile<E, C, KP, 32> qs, ks;
  __shared__ union {
    Values v;
    Scores s;
  } m;
  __shared__ Decays<C> dec;
  __shared__ float bs[C], vd[C], fs[NW][C], xs[NW];

  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const uint32_t block = (uint32_t)block_id();
  if (block >= b.blocks) return;
  const int head = block % p.heads;
  Segment seg;
  if (!find_segment(p.chunk_map, block / p.heads, seg)) return;
  const int n = (int)(seg.end - seg.begin);
  if (n == 0) return;
  const int rep = p.heads / p.groups, group = head / rep, K = p.K;
  const int64_t at = (p.map.cu ? seg.start : 0) + seg.begin, sq = p.map.cu ? 0 : seg.s, token = seg.start + seg.begin;
  const int64_t kv = (int64_t)K * p.V;
  const float *hb = p.chunk_state + block * kv, *db = b.chunk_dstate + block * kv;
  {
    TileLoad<E, C, KP, 32, THREADS, TINY> q, k;
    q.load(static_cast<const E*>(p.q) + sq * p.q_stride[0] + at * p.q_stride[1] + group * p.q_stride[2], p.q_stride[1], n, K);
    k.load(static_cast<const E*>(p.k) + sq * p.k_stride[0] + at * p.k_stride[1] + group * p.k_stride[2], p.k_stride[1], n, K);
    if (wave == 0) {
      const int64_t t = at + min(lane, n - 1);
      const float x = p.g[sq * p.g_stride[0] + t * p.g_stride[1] + head * p.g_stride[2]];
      const float y = p.beta[sq * p.b_stride[0] + t * p.b_stride[1] + head * p.b_stride[2]];
      if (lane < C) bs[lane] = lane < n ? y : 0.f;
      scan_decays<C>(lane < n ? x : 0.f, dec);
    }
    q.store(qs, n, K);
    k.store(ks, n, K);
  }
  const E* vb = static_cast<const E*>(p.v) + sq * p.v_stride[0] + at * p.v_stride[1] + head * p.v_stride[2];
  const E* ob = static_cast<const E*>(b.d_o) + sq * b.do_stride[0] + at * b.do_stride[1] + head * b.do_stride[2];

  f32x4 dq[OK][1][NI], dk[OK][1][NI], dz[OK][NI], sx[NI], sy[NI];
#pragma unroll
  for (int x = 0; x < NI; ++x) {
    sx[x] = sy[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int a = 0; a < OK; ++a) dq[a][0][x] = dk[a][0][x] = dz[a][x] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  float xsum = 0.f, bsum = 0.f, vsum = 0.f;
  const int ti = threadIdx.x / TT, tc = threadIdx.x % TT * PC;  // this thread's token and columns
  const int it = wave % NI, share = wave / NI, i0 = it * 16 + l;
  for (int v0 = 0; v0 < p.V; v0 += VT) {
    const int nv = min(p.V - v0, VT);
    __syncthreads();  // the tiles before have been read, the decays are there
    {
      TileLoad<E, C, VT, 16, THREADS, TINY> d;
      d.load(ob + v0, b.do_stride[1], n, nv);
      const float be = bs[ti];
      const int64_t row = ((token + min(ti, n - 1)) * p.heads + head) * p.V + v0 + tc;
#pragma unroll
      for (int c = 0; c < PC; c += 4) {
        const int left = ti < n ? nv - tc - c : 0;
        const f32x4 e = load4(p.errors + row + c, left), f = load4(b.df + row + c, left);
        const f32x4 v = load4(vb + min(ti, n - 1) * p.v_stride[1] + v0 + tc + c, left), z = f * be;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          bsum = fmaf(e[r], f[r], bsum);
          vsum = fmaf(z[r], v[r], vsum);
        }
        put4_parts(m.v.u, ti * m.v.u[0].stride + tc + c, e * be);
        put4_parts(m.v.z, ti * m.v.z[0].stride + tc + c, z);
        if (left > 0) store4(static_cast<E*>(b.dv) + row + c, left, z);
      }
      d.store(m.v.d, n, nv);
    }
    __syncthreads();
    // (do . u) and (dz . u), transposed: rows j, columns i
#pragma unroll
    for (int jt = 0; jt < NI; ++jt)
      if (share < JS && jt % JS == share && jt <= it)
#pragma unroll
        for (int c = 0; c < VT; c += 32) {
          const Frag<E> fd = frag_row(m.v.d, i0, c);
          Frag<E> fu[PF], fz[PB];
#pragma unroll
          for (int q = 0; q < PF; ++q) fu[q] = frag_row(m.v.u[q], jt * 16 + l, c);
#pragma unroll
          for (int q = 0; q < PB; ++q) fz[q] = frag_row(m.v.z[q], i0, c);
#pragma unroll
          for (int q = PF - 1; q >= 0; --q) sx[jt] = mma(fu[q], fd, sx[jt]);
#pragma unroll
          for (int s = PB - 1; s >= 0; --s)
#pragma unroll
            for (int q = 0; q <= s; ++q) sy[jt] = mma(fu[q], fz[s - q], sy[jt]);
        }
#pragma unroll
    for (int a = 0; a < OK; ++a)
      if (wave + a * NW < NK) {
        const int k = (wave + a * NW) * 16 + l;
#pragma unroll
        for (int c = 0; c < NV; c += 2) {
          const int64_t row = (int64_t)min(k, K - 1) * p.V + v0;
          const int c0 = c * 16 + 4 * g, c1 = c0 + 16;
          const int n0 = k < K ? nv - c0 : 0, n1 = k < K ? nv - c1 : 0;
          float h[8], d[8];
          stack(load4(hb + row + c0, n0), load4(hb + row + c1, n1), h);
          stack(load4(db + row + c0, n0), load4(db + row + c1, n1), d);
#pragma unroll
          for (int r = 0; r < 8; ++r) xsum = fmaf(h[r], d[r], xsum);
          Frag<E> fh[PF], fd[1];
          split_parts(h, fh);
          split_parts(d, fd);
#pragma unroll
          for (int x = 0; x < NI; ++x) {
            const Frag<E> o = frag_row_split(m.v.d, x * 16 + l, c * 16);
#pragma unroll
            for (int q = PF - 1; q >= 0; --q) dq[a][0][x] = mma(fh[q], o, dq[a][0][x]);
#pragma unroll
            for (int q = PB - 1; q >= 0; --q) {
              dk[a][0][x] = mma(fd[0], frag_row_split(m.v.u[q], x * 16 + l, c * 16), dk[a][0][x]);
              dz[a][x] = mma(fh[0], frag_row_split(m.v.z[q], x * 16 + l, c * 16), dz[a][x]);
            }
          }
        }
      }
  }
  // sums over a token's threads
#pragma unroll
  for (int s = 1; s < TT; s <<= 1) {
    bsum += __shfl_xor(bsum, s);
    vsum += __shfl_xor(vsum, s);
  }
  if (threadIdx.x % TT == 0) {
    vd[ti] = vsum;
    if (ti < n) b.dbeta[(token + ti) * p.heads + head] = bsum;
  }
  __syncthreads();  // the last values have been read
#pragma unroll
  for (int jt = 0; jt < NI; ++jt)
    if (share < JS && jt % JS == share && jt <= (it | 1)) {  // the last may be all masked: pairs are read
      const f32x4 e = dec.between4(i0, jt * 16 + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = jt * 16 + 4 * g + r;
        const float x = sx[jt][r] * (p.scale * e[r]), y = -sy[jt][r] * e[r];
        sx[jt][r] = j <= i0 ? x : 0.f;
        sy[jt][r] = j < i0 ? y : 0.f;
      }
      put4_parts(m.s.x, i0 * m.s.x[0].stride + jt * 16 + 4 * g, sx[jt]);
      put4(&m.s.y.e[i0 * m.s.y.stride + jt * 16 + 4 * g], sy[jt]);
    }
  __syncthreads();
  float fsum[NI];
#pragma unroll
  for (int x = 0; x < NI; ++x) fsum[x] = 0.f;
#pragma unroll
  for (int a = 0; a < OK; ++a)
    if (wave + a * NW < NK) {
      const int k0 = (wave + a * NW) * 16;
#pragma unroll
      for (int x = 0; x < NI; ++x) {
        const int i = x * 16 + l;
        const float since = __builtin_amdgcn_exp2f(dec.whole[i] + dec.frac[i]);
        dq[a][0][x] *= p.scale * since;
        dk[a][0][x] = dk[a][0][x] * dec.between(C - 1, i) - dz[a][x] * since;
      }
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const Frag<E> fk = frag_col_split(ks, j * 16, k0), fq = frag_col_split(qs, j * 16, k0);
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          if (x >= j) {  // tokens j .. j + 31 before x
#pragma unroll
            for (int q = PF - 1; q >= 0; --q) dq[a][0][x] = mma(fk, frag_row_split(m.s.x[q], x * 16 + l, j * 16), dq[a][0][x]);
            dk[a][0][x] = mma(fk, frag_row_split(m.s.y, x * 16 + l, j * 16), dk[a][0][x]);
          }
          if (x < j + 2) {  // tokens j .. j + 31 behind x
            dk[a][0][x] = mma(fq, frag_col_split(m.s.x[0], j * 16, x * 16), dk[a][0][x]);
            dk[a][0][x] = mma(fk, frag_col_split(m.s.y, j * 16, x * 16), dk[a][0][x]);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < NI; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          fsum[x] = fmaf(load1(&qs.e[(x * 16 + l) * qs.stride + k0 + 4 * g + r]), dq[a][0][x][r], fsum[x]);
      const int64_t stride = (int64_t)p.groups * K, part = (head % rep) * p.map.tokens;
      auto put = [&](void* whole, float* parts, const f32x4 (&x)[1][NI]) {
        if (parts)
          put_rows<NI, 1>(parts + ((part + token) * p.groups + group) * K, stride, n, K, k0 + 4 * g, 0, l, x);
        else
          put_rows<NI, 1>(static_cast<E*>(whole) + (token * p.groups + group) * K, stride, n, K, k0 + 4 * g, 0, l, x);
      };
      put(b.dq, b.dq_part, dq[a]);
      put(b.dk, b.dk_part, dk[a]);
    }
#pragma unroll
  for (int x = 0; x < NI; ++x) {
    fsum[x] = across_rows(fsum[x]);
    if (g == 0) fs[wave][x * 16 + l] = fsum[x];
  }
  xsum = wave_sum(xsum);
  if (lane == 0) xs[wave] = xsum;
  __syncthreads();
  if (wave == 0) {  // the chunk's decay gradients
    float f = 0.f, x = 0.f, y = 0.f;
    if (lane < n) {
#pragma unroll
      for (int w = 0; w < NW; ++w) f += fs[w][lane];
      f -= vd[lane];
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) x += xs[w];
    for (int i = lane; i < b.columns; i += 64) y += b.inner[block * (int64_t)b.columns + i];
    x = fmaf(x, __builtin_amdgcn_exp2f(dec.whole[C - 1] + dec.frac[C - 1]), wave_sum(y));
    f = __shfl(wave_scan(__shfl(f, 63 - lane)), 63 - lane);  // from a token on
    if (lane < n) b.dg[(token + lane) * p.heads + head] = f + x;
  }
}

// out[e] = sum over the parts, for the values of tokens inside the sequences.
template <typename E>
__global__ __launch_bounds__(256) void sum_parts(const float* __restrict__ parts, E* __restrict__ out, int n,
                                                 int64_t per_token, SequenceMap map) {
  const int64_t e = block_id() * 256 + threadIdx.x, size = map.tokens * per_token;
  const int64_t token = e / per_token;
  if (e >= size || (map.cu && (token < cu_at(map, 0) || token >= cu_at(map, map.sequences)))) return;
  float s = parts[e];
  for (int i = 1; i < n; ++i) s += parts[i * size + e];
  store1(out + e, s);
}

// ------------------------------------------------------------------ launches
// Value columns of a workgroup that walks back, and the parts of `inner` they leave.
int back_tile(int64_t V, const DeltaPlan& pl) { return V <= 64 || pl.a.tiny ? 64 : 128; }
int columns_of(int64_t V, const DeltaPlan& pl) {
  const int vt = back_tile(V, pl);
  return (int)((V + vt - 1) / vt) * (vt / 16);
}

// Byte offsets of the workspace's regions.
struct Regions {
  size_t systems, seg_state, seg_map, seg_dstate, chunk_state, chunk_dstate, errors, df, inner, dq_part, dk_part, end;
};
Regions regions(const DeltaPlan& pl, int64_t tokens, int64_t groups, int64_t heads, int64_t K, int64_t V, int dtype) {
  Regions r{};
  size_t at = 0;
  auto take = [&](int64_t floats) {
    const size_t here = at;
    at += ((size_t)floats * 4 + 255) / 256 * 256;
    return here;
  };
  const AttentionPlan& a = pl.a;
  r.systems = take(a.chunks * heads * (system_bytes(pl, dtype) / 4));
  r.seg_state = take(a.split ? a.slots * heads * K * V : 0);
  r.seg_map = take(a.split ? a.slots * heads * a.kp * a.kp : 0);
  r.seg_dstate = take(a.split ? a.slots * heads * K * V : 0);
  r.chunk_state = take(a.chunks * heads * K * V);
  r.chunk_dstate = take(a.chunks * heads * K * V);
  r.errors = take(tokens * heads * V);
  r.df = take(tokens * heads * V);
  r.inner = take(a.chunks * heads * columns_of(V, pl));
  r.dq_part = take(heads > groups ? tokens * heads * K : 0);
  r.dk_part = take(heads > groups ? tokens * heads * K : 0);
  r.end = at;
  return r;
}

template <typename F>
void with_keys(const DeltaPlan& pl, F f) {
  using std::integral_constant;
  if (pl.a.tiny)
    f(integral_constant<int, 256>(), integral_constant<bool, true>());
  else if (pl.a.kp == 32)
    f(integral_constant<int, 32>(), integral_constant<bool, false>());
  else if (pl.a.kp == 64)
    f(integral_constant<int, 64>(), integral_constant<bool, false>());
  else if (pl.a.kp == 128)
    f(integral_constant<int, 128>(), integral_constant<bool, false>());
  else
    f(integral_constant<int, 256>(), integral_constant<bool, false>());
}

template <typename E, int C, bool SUM>
hipError_t launch_walk_back(BackParams b, const DeltaPlan& pl, hipStream_t st) {
  const int vt = back_tile(b.d.V, pl);
  b.d.vtiles = (b.d.V + vt - 1) / vt;
  b.blocks = (uint32_t)(pl.a.slots * b.d.heads);
  b.columns = columns_of(b.d.V, pl);
  with_keys(pl, [&](auto kp, auto tiny) {
    const dim3 grid = grid_of(spread_blocks(b.blocks, b.d.vtiles), vt * 4), block(vt * 4);
    if (vt == 64)
      delta_walk_back<E, C, kp(), 64, SUM, tiny()><<<grid, block, 0, st>>>(b);
    else if constexpr (!tiny())
      delta_walk_back<E, C, kp(), 128, SUM, false><<<grid, block, 0, st>>>(b);
  });
  return hipGetLastError();
}

template <typename E, int C>
hipError_t launch_gradients(BackParams b, const DeltaPlan& pl, hipStream_t st) {
  b.blocks = (uint32_t)(pl.a.chunks * b.d.heads);
  b.columns = columns_of(b.d.V, pl);
  with_keys(pl, [&](auto kp, auto tiny) {
    constexpr int NW = kp() >= 128 ? 8 : 4;
    delta_gradients<E, C, kp(), NW, tiny()><<<grid_of(b.blocks, NW * 64), dim3(NW * 64), 0, st>>>(b);
  });
  return hipGetLastError();
}

template <typename E>
hipError_t launch_sum(const float* parts, void* out, int n, int64_t per_token, const SequenceMap& map, hipStream_t st) {
  sum_parts<E><<<grid_of((map.tokens * per_token + 255) / 256, 256), dim3(256), 0, st>>>(
      parts, static_cast<E*>(out), n, per_token, map);
  return hipGetLastError();
}

}  // namespace

size_t delta_backward_workspace_bytes(const DeltaPlan& pl, int64_t tokens, int64_t groups, int64_t heads,
                                      int64_t key_dim, int64_t value_dim, int dtype) {
  return regions(pl, tokens, groups, heads, key_dim, value_dim, dtype).end;
}

hipError_t launch_delta_backward(const DeltaBackwardArgs& a, const DeltaPlan& pl) {
  const AttentionArgs& f = a.d.f;
  const Regions rg = regions(pl, f.tokens, f.groups, f.heads, f.key_dim, f.value_dim, f.dtype);
  char* ws = static_cast<char*>(f.workspace);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  const bool bf16 = f.dtype == 1;
  BackParams b{};
  DeltaParams& p = b.d;
  p = delta_params(a.d, pl);
  p.systems = ws + rg.systems;
  p.seg_state = at(rg.seg_state);
  p.seg_map = at(rg.seg_map);
  p.chunk_state = at(rg.chunk_state);
  p.errors = at(rg.errors);
  b.d_o = a.d_o;
  for (int i = 0; i < 3; ++i) b.do_stride[i] = a.do_stride[i];
  b.dstate_out = a.dstate_out;
  b.seg_dstate = at(rg.seg_dstate);
  b.chunk_dstate = at(rg.chunk_dstate);
  b.df = at(rg.df);
  b.inner = at(rg.inner);
  b.dq = a.dq;
  b.dk = a.dk;
  b.dv = a.dv;
  const int rep = (int)(f.heads / f.groups);
  b.dq_part = rep > 1 ? at(rg.dq_part) : nullptr;
  b.dk_part = rep > 1 ? at(rg.dk_part) : nullptr;
  b.dg = a.dlog_decay;
  b.dbeta = a.dbeta;
  b.dstate_in = a.dstate_in;

  hipError_t e = launch_delta_systems(p, pl, f.dtype, f.stream);
  if (e == hipSuccess && pl.a.split) {
    p.last_maps = true;
    e = launch_delta_segments(p, pl, f.dtype, f.stream);
    if (e == hipSuccess)
      e = bf16 ? launch_walk_back<uint16_t, 64, true>(b, pl, f.stream) : launch_walk_back<float, 32, true>(b, pl, f.stream);
    if (e == hipSuccess) {
      const CarryParams c{b.seg_dstate, p.seg_map, b.dstate_out, p.map, p.heads, p.K, p.V, 0, 0};
      e = launch_delta_carry(c, pl, true, f.stream);
    }
  }
  if (e == hipSuccess) e = launch_delta_states(p, pl, f.dtype, f.stream);
  if (e == hipSuccess)
    e = bf16 ? launch_walk_back<uint16_t, 64, false>(b, pl, f.stream) : launch_walk_back<float, 32, false>(b, pl, f.stream);
  if (e == hipSuccess)
    e = bf16 ? launch_gradients<uint16_t, 64>(b, pl, f.stream) : launch_gradients<float, 32>(b, pl, f.stream);
  if (e == hipSuccess && rep > 1) {
    const int64_t n = f.groups * f.key_dim;
    for (int i = 0; i < 2 && e == hipSuccess; ++i) {
      const float* from = i ? b.dk_part : b.dq_part;
      void* to = i ? a.dk : a.dq;
      e = bf16 ? launch_sum<uint16_t>(from, to, rep, n, p.map, f.stream) : launch_sum<float>(from, to, rep, n, p.map, f.stream);
    }
  }
  return e;
}

}  // namespace ss2d
