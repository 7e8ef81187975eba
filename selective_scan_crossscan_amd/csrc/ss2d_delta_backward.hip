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
//
// us of 2 x 4096 tokens, 16 heads of 128, bf16: systems 39, both ways' segments 151 and carries 35, states 80, the walk
// back 113, all else 217 (192 KiB of H, D, E and dF in fp32 per chunk and head at 1.9 TB/s; matrix instructions 20% of the
// SIMDs' cycles, the waves waiting 58% of their time).
#include "ss2d_delta_walk.h"

namespace ss2d {
namespace {

// What the segments add to the state and their maps, and what they add to its gradient, in one grid: each alone leaves
// CUs idle where sequences had to be cut.
template <typename E, int C, int KP, bool TINY>
__global__ __launch_bounds__(256, 2) void delta_segment_pair(DeltaParams p, BackParams b, uint32_t first) {
  __shared__ union Both {
    WalkTiles<E, C, KP, 64, kSegments> w;
    BackTiles<E, C, KP, 64> b;
    __device__ Both() {}
  } lds;
  const uint32_t block = (uint32_t)block_id();
  if (block < first)
    walk<E, C, KP, 64, kSegments, TINY>(p, block, lds.w);
  else
    walk_back<E, C, KP, 64, true, TINY>(b, block - first, lds.b);
}

template <typename E, int C, int KP, int VT, bool TINY>
__global__ __launch_bounds__(VT * 4, VT == 64 ? 1 : 2) void delta_walk_back(BackParams b) {
  __shared__ BackTiles<E, C, KP, VT> lds;
  walk_back<E, C, KP, VT, false, TINY>(b, (uint32_t)block_id(), lds);
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

// Eight waves also for few keys: four would spill registers.
constexpr int kGradientWaves = 8;
// One workgroup per chunk and head; a wave owns key columns wave, wave + NW, ... by 16 and their dq and dk, transposed
// (rows k, columns token); the values are gone through in tiles of 64 columns.
template <typename E, int C, int KP, bool TINY>
__global__ __launch_bounds__(kGradientWaves * 64) void delta_gradients(BackParams b) {
  const DeltaParams& p = b.d;
  constexpr int NW = kGradientWaves, THREADS = NW * 64, NI = C / 16, NK = KP / 16, VT = kArrayTile, NV = VT / 16, PF = kFullParts<E>;
  constexpr int OK = (NK + NW - 1) / NW;
  constexpr int JS = NW / NI < NI ? NW / NI : NI;  // waves that share 16 tokens' scores
  constexpr int NS = NI / JS;                      // score tiles of a wave
  constexpr int TT = THREADS / C, PC = VT / TT;    // threads per token, each with PC columns of values
  static_assert(NW >= NI && PC % 4 == 0, "score tiles and columns are dealt evenly");
  struct Values {
    Tile<E, C, VT> d, z[PF], u[PF];
  };
  struct Scores {
    Tile<E, C, C> x[PF], y[PF];
  };
  __shared__ Tile<E, C, KP, 32> qs, ks;
  __shared__ union {
    Values v;
    Scores s;
  } m;
  __shared__ union Last {  // the values are done with before the sums are written
    Tile<E, C, VT> vs;
    float fs[NW][C];
    __device__ Last() {}
  } last;
  auto& vs = last.vs;
  auto& fs = last.fs;
  __shared__ Decays<C> dec;
  __shared__ float bs[C], vd[C], xs[NW];

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
  const int64_t place = (int64_t)block * p.tiles;  // the first tile of the chunks' arrays
  const E* vb = static_cast<const E*>(p.v) + sq * p.v_stride[0] + at * p.v_stride[1] + head * p.v_stride[2];
  const E* ob = static_cast<const E*>(b.d_o) + sq * b.do_stride[0] + at * b.do_stride[1] + head * b.do_stride[2];
  const int ti = threadIdx.x / TT, tc = threadIdx.x % TT * PC;  // this thread's token and columns
  const int it = wave % NI, share = wave / NI, i0 = it * 16 + l;
  const uint32_t et = 4 * (ti * kArrayTile + tc);  // bytes into a tile of the chunks' arrays
  E* vto = static_cast<E*>(b.dv) + (token * p.heads + head) * p.V;
  const uint32_t vt = (uint32_t)ti * (uint32_t)(p.heads * p.V) + tc;  // 64 tokens' are under 2^32

  // a tile of 64 value columns on its way: two tiles' loads are in flight beside one's products
  struct Ahead {
    TileLoad<E, C, VT, 16, THREADS, TINY> d, v;
    f32x4 e[PC / 4], f[PC / 4];
  };
  auto fetch = [&](Ahead& x, int v0) {
    const int nv = min(p.V - v0, VT);
    if (kAhead<KP>) {
      x.d.load(ob + v0, b.do_stride[1], n, nv);
      x.v.load(vb + v0, p.v_stride[1], n, nv);
    }
    const int64_t at = (place + v0 / VT) * (C * kArrayTile);
    const f32x4 *e = reinterpret_cast<const f32x4*>(by_bytes(p.errors + at, et)),
                *f = reinterpret_cast<const f32x4*>(by_bytes(b.df + at, et));
#pragma unroll
    for (int c = 0; c < PC / 4; ++c) {
      x.e[c] = e[c];
      x.f[c] = f[c];
    }
  };
  Ahead x;
  {
    TileLoad<E, C, KP, 32, THREADS, TINY && KP == 32> q, k;
    q.load(static_cast<const E*>(p.q) + sq * p.q_stride[0] + at * p.q_stride[1] + group * p.q_stride[2], p.q_stride[1], n, K);
    if (!kAhead<KP>) {
      q.store(qs, n, K);
      __builtin_amdgcn_sched_barrier(0);
    }
    k.load(static_cast<const E*>(p.k) + sq * p.k_stride[0] + at * p.k_stride[1] + group * p.k_stride[2], p.k_stride[1], n, K);
    const int64_t t = at + min(lane, n - 1);
    const float decay = p.g[sq * p.g_stride[0] + t * p.g_stride[1] + head * p.g_stride[2]];
    const float beta = p.beta[sq * p.b_stride[0] + t * p.b_stride[1] + head * p.b_stride[2]];
    if (kAhead<KP>) fetch(x, 0);
    if (wave == 0) {
      if (lane < C) bs[lane] = lane < n ? beta : 0.f;
      scan_decays<C>(lane < n ? decay : 0.f, dec);
    }
    if (kAhead<KP>) q.store(qs, n, K);
    k.store(ks, n, K);
  }

  f32x4 dq[OK][1][NI], dk[OK][1][NI], dz[OK][NI], sx[NS], sy[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) sx[i] = sy[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int a = 0; a < OK; ++a) dq[a][0][i] = dk[a][0][i] = dz[a][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float xsum = 0.f, bsum = 0.f, vsum = 0.f;
  // the state and its gradient: rows k of the wave's key columns, four values at a time
  constexpr int HS = kAhead<KP> ? OK : 1;  // of all key columns, or one after the other
  f32x4 h[HS][NV], d[HS][NV];
  auto fetch_states = [&](int v0, int from) {
#pragma unroll
    for (int a = 0; a < HS; ++a) {
      const int64_t at = (place + v0 / VT) * (KP * kArrayTile);
      const uint32_t row = 4 * (((wave + (from + a) * NW) % NK * 16 + l) * kArrayTile + 4 * g);
      const f32x4 *hp = reinterpret_cast<const f32x4*>(by_bytes(p.chunk_state + at, row)),
                  *dp = reinterpret_cast<const f32x4*>(by_bytes(b.chunk_dstate + at, row));
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        h[a][c] = hp[4 * c];
        d[a][c] = dp[4 * c];
      }
    }
  };
  for (int v0 = 0; v0 < p.V; v0 += VT) {
    const int nv = min(p.V - v0, VT);
    if (kAhead<KP>)
      fetch_states(v0, 0);
    else
      fetch(x, v0);
    __syncthreads();  // the tiles before have been read, the decays are there
    f32x4 zs[PC / 4];
    {
      const float be = bs[ti];
#pragma unroll
      for (int c = 0; c < PC / 4; ++c) {
        const f32x4 z = x.f[c] * be;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          bsum = fmaf(x.e[c][r], x.f[c][r], bsum);
        }
        put4_parts(m.v.u, ti * m.v.u[0].stride + tc + 4 * c, x.e[c] * be);
        put4_parts(m.v.z, ti * m.v.z[0].stride + tc + 4 * c, z);
        zs[c] = z;
      }
      if (!kAhead<KP>) {  // tile by tile, with few registers
        __builtin_amdgcn_sched_barrier(0);
        x.d.load(ob + v0, b.do_stride[1], n, nv);
      }
      x.d.store(m.v.d, n, nv);
      if (!kAhead<KP>) {
        __builtin_amdgcn_sched_barrier(0);
        x.v.load(vb + v0, p.v_stride[1], n, nv);
      }
      x.v.store(vs, n, nv);
    }
    __syncthreads();
    if (kAhead<KP>) fetch(x, v0 + VT < p.V ? v0 + VT : v0);  // always: a load under a condition would be waited for
#pragma unroll
    for (int c = 0; c < PC / 4; ++c) {
      const f32x4 v = load4(&vs.e[ti * vs.stride + tc + 4 * c], 4);
#pragma unroll
      for (int r = 0; r < 4; ++r) vsum = fmaf(zs[c][r], v[r], vsum);
    }
#pragma unroll
    for (int a = 0; a < OK; ++a)
      if (wave + a * NW < NK) {
        const int at = kAhead<KP> ? a : 0;
        if (!kAhead<KP>) {
          __builtin_amdgcn_sched_barrier(0);
          fetch_states(v0, a);
        }
#pragma unroll
        for (int c = 0; c < NV; c += 2) {
          float u[8];
          Frag<E> f[PF];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            xsum = fmaf(h[at][c][r], d[at][c][r], xsum);
            xsum = fmaf(h[at][c + 1][r], d[at][c + 1][r], xsum);
          }
          // parts in the order in which each tile's are read once: the largest of one with all of the other's first
          stack(d[at][c], d[at][c + 1], u);
          split_parts(u, f);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
#pragma unroll
            for (int q = 0; q < PF; ++q) {
              const Frag<E> x = frag_row_split(m.v.u[q], i * 16 + l, c * 16);
#pragma unroll
              for (int n = PF - 1 - q; n >= 0; --n) dk[a][0][i] = mma(f[n], x, dk[a][0][i]);
            }
            if (!kAhead<KP>) __builtin_amdgcn_sched_barrier(0);  // or their registers add up and spill
          }
          stack(h[at][c], h[at][c + 1], u);
          split_parts(u, f);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const Frag<E> o = frag_row_split(m.v.d, i * 16 + l, c * 16);
#pragma unroll
            for (int q = 0; q < PF; ++q) {
              const Frag<E> x = frag_row_split(m.v.z[q], i * 16 + l, c * 16);
#pragma unroll
              for (int n = PF - 1 - q; n >= 0; --n) dz[a][i] = mma(f[n], x, dz[a][i]);
              dq[a][0][i] = mma(f[PF - 1 - q], o, dq[a][0][i]);
            }
            if (!kAhead<KP>) __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    __builtin_amdgcn_sched_barrier(0);
    // behind the uses of what was loaded before: a wait for that would be one for these stores and loads too
#pragma unroll
    for (int c = 0; c < PC / 4; ++c) {
      const int left = ti < n ? nv - tc - 4 * c : 0;
      if (left > 0) store4(vto + v0 + vt + 4 * c, left, zs[c]);
    }
    __builtin_amdgcn_sched_barrier(0);
    // (do . u) and (dz . u), transposed: rows j, columns i
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int jt = i * JS + share;
      if (share < JS && jt <= it)
#pragma unroll
        for (int c = 0; c < VT; c += 32) {
          const Frag<E> fd = frag_row(m.v.d, i0, c);
          Frag<E> fu[PF], fz[PF];
#pragma unroll
          for (int q = 0; q < PF; ++q) {
            fu[q] = frag_row(m.v.u[q], jt * 16 + l, c);
            fz[q] = frag_row(m.v.z[q], i0, c);
          }
#pragma unroll
          for (int q = PF - 1; q >= 0; --q) sx[i] = mma(fu[q], fd, sx[i]);
#pragma unroll
          for (int s = PF - 1; s >= 0; --s)
#pragma unroll
            for (int q = 0; q <= s; ++q) sy[i] = mma(fu[q], fz[s - q], sy[i]);
        }
    }
  }
  // The lane anew, from the hardware: kept over the values' loop its parts would be spilled there.
  const int at_lane = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));
  const int eg = at_lane >> 4, el = at_lane & 15, ei = it * 16 + el;
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
  for (int i = 0; i < NS; ++i) {
    const int jt = i * JS + share;
    if (share < JS && jt <= (it | 1)) {  // the last may be all masked: pairs are read
      const f32x4 e = dec.between4(ei, jt * 16 + 4 * eg);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = jt * 16 + 4 * eg + r;
        const float x = sx[i][r] * (p.scale * e[r]), y = -sy[i][r] * e[r];
        sx[i][r] = j <= ei ? x : 0.f;
        sy[i][r] = j < ei ? y : 0.f;
      }
      put4_parts(m.s.x, ei * m.s.x[0].stride + jt * 16 + 4 * eg, sx[i]);
      put4_parts(m.s.y, ei * m.s.y[0].stride + jt * 16 + 4 * eg, sy[i]);
    }
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
        const int i = x * 16 + el;
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
            for (int q = PF - 1; q >= 0; --q) {
              dq[a][0][x] = mma(fk, frag_row_split(m.s.x[q], x * 16 + el, j * 16), dq[a][0][x]);
              dk[a][0][x] = mma(fk, frag_row_split(m.s.y[q], x * 16 + el, j * 16), dk[a][0][x]);
            }
          }
          if (x < j + 2)  // tokens j .. j + 31 behind x
#pragma unroll
            for (int q = PF - 1; q >= 0; --q) {
              dk[a][0][x] = mma(fq, frag_col_split(m.s.x[q], j * 16, x * 16), dk[a][0][x]);
              dk[a][0][x] = mma(fk, frag_col_split(m.s.y[q], j * 16, x * 16), dk[a][0][x]);
            }
        }
      }
#pragma unroll
      for (int x = 0; x < NI; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          fsum[x] = fmaf(load1(&qs.e[(x * 16 + el) * qs.stride + k0 + 4 * eg + r]), dq[a][0][x][r], fsum[x]);
      const int64_t stride = (int64_t)p.groups * K, part = (head % rep) * p.map.tokens;
      auto put = [&](void* whole, float* parts, const f32x4 (&x)[1][NI]) {
        if (parts)
          put_rows<NI, 1>(parts + ((part + token) * p.groups + group) * K, stride, n, K, k0 + 4 * eg, 0, el, x);
        else
          put_rows<NI, 1>(static_cast<E*>(whole) + (token * p.groups + group) * K, stride, n, K, k0 + 4 * eg, 0, el, x);
      };
      put(b.dq, b.dq_part, dq[a]);
      put(b.dk, b.dk_part, dk[a]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
  for (int x = 0; x < NI; ++x) {
    fsum[x] = across_rows(fsum[x]);
    if (eg == 0) fs[wave][x * 16 + el] = fsum[x];
  }
  xsum = wave_sum(xsum);
  if (at_lane == 0) xs[wave] = xsum;
  __syncthreads();
  if (wave == 0) {  // the chunk's decay gradients
    float f = 0.f, x = 0.f, y = 0.f;
    if (at_lane < n) {
#pragma unroll
      for (int w = 0; w < NW; ++w) f += fs[w][at_lane];
      f -= vd[at_lane];
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) x += xs[w];
    for (int i = at_lane; i < b.columns; i += 64) y += b.inner[block * (int64_t)b.columns + i];
    x = fmaf(x, __builtin_amdgcn_exp2f(dec.whole[C - 1] + dec.frac[C - 1]), wave_sum(y));
    f = __shfl(wave_scan(__shfl(f, 63 - at_lane)), 63 - at_lane);  // from a token on
    if (at_lane < n) b.dg[(token + at_lane) * p.heads + head] = f + x;
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
// Value columns of a workgroup that walks back, and the parts of `inner` they leave.  Of 128 values half the workgroups
// read the keys and systems once (2 x 2048 tokens, 16 heads of 128, all gradients 368 us, 387 in tiles of 64; 64 keys 258
// and 257, 32 keys 210 and 209).
int back_tile(int64_t V, const DeltaPlan& pl) { return V <= 64 || pl.a.tiny ? 64 : 128; }
int columns_of(int64_t V, const DeltaPlan& pl) {
  const int vt = back_tile(V, pl);
  return (int)((V + vt - 1) / vt) * (vt / 16);
}

// Values padded for the chunks' arrays: whole tiles of all walks.
int64_t padded_values(int64_t V, const DeltaPlan& pl) {
  const int vt = back_tile(V, pl);
  return (V + vt - 1) / vt * vt;
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
  r.seg_state = take(a.split ? pl.parts * heads * K * V : 0);
  r.seg_map = take(a.split ? pl.parts * heads * a.kp * a.kp : 0);
  r.seg_dstate = take(a.split ? pl.parts * heads * K * V : 0);
  const int64_t per = a.chunks * heads * padded_values(V, pl);
  r.chunk_state = take(per * a.kp);
  r.chunk_dstate = take(per * a.kp);
  r.errors = take(per * a.chunk);
  r.df = take(per * a.chunk);
  r.inner = take(a.chunks * heads * columns_of(V, pl));
  r.dq_part = take(heads > groups ? tokens * heads * K : 0);
  r.dk_part = take(heads > groups ? tokens * heads * K : 0);
  r.end = at;
  return r;
}

template <typename E, int C>
hipError_t launch_walk_back(BackParams b, const DeltaPlan& pl, hipStream_t st) {
  const int vt = back_tile(b.d.V, pl);
  b.d.vtiles = (b.d.V + vt - 1) / vt;
  b.blocks = (uint32_t)(pl.a.slots * b.d.heads);
  b.columns = columns_of(b.d.V, pl);
  with_keys(pl, [&](auto kp, auto tiny) {
    const dim3 grid = grid_of(spread_blocks(b.blocks, b.d.vtiles), vt * 4), block(vt * 4);
    if (vt == 64)
      delta_walk_back<E, C, kp(), 64, tiny()><<<grid, block, 0, st>>>(b);
    else if constexpr (!tiny())
      delta_walk_back<E, C, kp(), 128, false><<<grid, block, 0, st>>>(b);
  });
  return hipGetLastError();
}

// Both ways' segments and their carries.
template <typename E, int C>
hipError_t launch_segments(DeltaParams p, BackParams b, const DeltaPlan& pl, hipStream_t st) {
  p.last_maps = true;
  p.vtiles = b.d.vtiles = (p.V + 63) / 64;
  p.ktiles = (pl.a.kp + 63) / 64;
  p.blocks = b.blocks = (uint32_t)(pl.parts * p.heads);
  const int64_t first = spread_blocks(p.blocks, p.vtiles + p.ktiles);
  with_keys(pl, [&](auto kp, auto tiny) {
    delta_segment_pair<E, C, kp(), tiny()>
        <<<grid_of(first + spread_blocks(b.blocks, b.d.vtiles), 256), dim3(256), 0, st>>>(p, b, (uint32_t)first);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const CarryParams c{p.seg_state, p.seg_map, p.state_in, p.map, p.cut, p.heads, p.K, p.V, 0, 0};
  const CarryParams r{b.seg_dstate, p.seg_map, b.dstate_out, p.map, p.cut, p.heads, p.K, p.V, 0, 0};
  return launch_delta_carry(c, &r, pl, st);
}

template <typename E, int C>
hipError_t launch_gradients(BackParams b, const DeltaPlan& pl, hipStream_t st) {
  b.blocks = (uint32_t)(pl.a.chunks * b.d.heads);
  b.columns = columns_of(b.d.V, pl);
  with_keys(pl, [&](auto kp, auto tiny) {
    constexpr int threads = kGradientWaves * 64;
    delta_gradients<E, C, kp(), tiny()><<<grid_of(b.blocks, threads), dim3(threads), 0, st>>>(b);
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
  p.tiles = (int)padded_values(p.V, pl) / kArrayTile;
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
  if (e == hipSuccess && pl.a.split)
    e = bf16 ? launch_segments<uint16_t, 64>(p, b, pl, f.stream) : launch_segments<float, 32>(p, b, pl, f.stream);
  if (e == hipSuccess) e = launch_delta_states(p, pl, f.dtype, f.stream);
  if (e == hipSuccess)
    e = bf16 ? launch_walk_back<uint16_t, 64>(b, pl, f.stream) : launch_walk_back<float, 32>(b, pl, f.stream);
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
