// Linear attention with a decay per head: the gradients.
//
// With h the state before a chunk of C tokens, d the gradient of the state behind
// it, M_ij = scale exp(G_i - G_j) for j <= i and 0 otherwise, S = q k', D = do v':
//   dq_i = sum_j (D M)_ij k_j + scale exp(G_i) h do_i
//   dk_j = sum_i (D M)_ij q_i + w_j d v_j,          w_j = exp(G_last - G_j)
//   dv_j = sum_i (S M)_ij do_i + w_j d' k_j
//   d   <- exp(G_last) d + sum_i scale exp(G_i) q_i do_i'   (the chunk before's d)
// and the gradient of g_t, what passes from before t to t or behind it:
//   dg_t = sum_{i >= t > j} W_ij + sum_{i >= t} F_i + sum_{j < t} E_j + X,
//   W = S D M, F_i = q_i . (scale exp(G_i) h do_i), E_j = k_j . (w_j d v_j),
//   X = exp(G_last) <h, d>.
// The usual q.dq - k.dk summed to the sequence's end is the same in exact
// arithmetic, but there every token's own term enters twice with opposite signs
// and its error adds up over the whole sequence; here only W's row and column
// sums inside one chunk are subtracted, of the same fp32 values.
//
// The states h of all chunks come from a pass before (ss2d_attention_state.hip)
// through memory; one workgroup walks a segment's chunks backwards with d in
// registers, twice: as result tiles with rows k and columns v, where a wave owns
// value columns and forms their dv, and transposed, where a wave owns key
// columns and forms their dq and dk.  Either product sums over the rows, so
// both read d as it lies; keeping it twice costs the update's products twice,
// which the matrix cores have room for, and spares publishing 64 KiB of d in
// parts through LDS at every chunk.  S, D and W are split over the waves, S M
// and D M go through LDS.
//
// 2 x 4096 tokens, 16 heads of 128 in bf16: 180 us of 284 in all (119 TFLOP/s).
// One workgroup of eight waves per CU (97 KiB of LDS, 256 registers), bound by the
// latency of a chunk's phases, of which the registers leave no more to overlap: in
// bf16 17 are spilled at 128 x 128 (72 bytes a lane), 4 at 64 x 128, 88 to 150 for
// keys over 128 channels.
//
// Where several heads share keys and queries or the values take several tiles,
// dq, dk (and dg) are written as fp32 parts and added in order by sum_parts.
#include "ss2d_attention.h"

namespace ss2d {
namespace {

using namespace tok;

struct BackwardParams {
  const void *q, *k, *v, *d_o;
  const float* g;
  const float* dstate_out;   // or null
  const float* seg_dstate;   // (slot, head, K, V): the gradient of the state behind a segment
  const float* chunk_state;
  void *dq, *dk, *dv;
  float* dg;
  float* dstate_in;          // or null
  float *dq_part, *dk_part;  // (part, token, group, K), or null: dq and dk themselves
  float* dg_part;            // (value tile, token, head), or null
  SequenceMap map;
  int64_t q_stride[3], k_stride[3], v_stride[3], do_stride[3], g_stride[3];
  int groups, heads, K, V, vtiles;
  uint32_t blocks;  // workgroups
  float scale;
};

template <typename E, int C, int KP, int VT, int NW, bool TINY>
__global__ __launch_bounds__(NW * 64) void attention_backward_kernel(BackwardParams p) {
  constexpr int THREADS = NW * 64;
  constexpr int NI = C / 16, NK = KP / 16, NV = VT / 16;
  constexpr int OK = (NK + NW - 1) / NW, OV = NV / NW;  // key and value tiles a wave owns: wave, wave + NW, ...
  constexpr int JS = NW / NI < NI ? NW / NI : NI;       // waves that share 16 tokens' scores
  constexpr int PF = kFullParts<E>;
  static_assert(NV % NW == 0 && NW >= NI, "value tiles and token tiles are dealt evenly");
  __shared__ Tile<E, C, KP, 32> qs;
  __shared__ Tile<E, C, KP> ks;
  __shared__ Tile<E, C, VT> vs, ds;
  __shared__ Tile<E, C, C, 32> sm;  // S M, rows i
  __shared__ Tile<E, C, C> dm;      // D M
  __shared__ Decays<C> dec;
  __shared__ float wrow[NW][C], wcol[NW][C], fs[NW][C], es[NW][C], xs[NW];

  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const uint32_t block = (uint32_t)block_id();
  if (block >= p.blocks) return;
  const int vt = block % p.vtiles, head = block / p.vtiles % p.heads;
  const int64_t slot = block / (p.vtiles * p.heads);
  Segment seg;
  if (!find_segment(p.map, slot, seg)) return;
  const int rep = p.heads / p.groups, group = head / rep;
  const int K = p.K, v0 = vt * VT, nv = min(p.V - v0, VT);
  const int64_t first = p.map.cu ? seg.start : 0, sq = p.map.cu ? 0 : seg.s;
  const E* qb = static_cast<const E*>(p.q) + sq * p.q_stride[0] + first * p.q_stride[1] + group * p.q_stride[2];
  const E* kb = static_cast<const E*>(p.k) + sq * p.k_stride[0] + first * p.k_stride[1] + group * p.k_stride[2];
  const E* vb = static_cast<const E*>(p.v) + sq * p.v_stride[0] + first * p.v_stride[1] + head * p.v_stride[2] + v0;
  const E* db = static_cast<const E*>(p.d_o) + sq * p.do_stride[0] + first * p.do_stride[1] + head * p.do_stride[2] + v0;
  const float* gb = p.g + sq * p.g_stride[0] + first * p.g_stride[1] + head * p.g_stride[2];

  // d: dv_[k tile][own value tile] rows k = 16 kt + 4g + r, column v; dk_[value tile][own key tile] rows v, column k
  f32x4 dkv[NK][OV], dvk[NV][OK];
  const int64_t kv = (int64_t)K * p.V, qh = ((int64_t)seg.s * p.heads + head) * kv;
  const float* from = !seg.last ? p.seg_dstate + (slot * p.heads + head) * kv : p.dstate_out ? p.dstate_out + qh : nullptr;
  auto entry = [&](int k, int v) {  // loaded at a place inside, dropped outside: no branch around the load
    const float x = from ? from[(int64_t)min(k, K - 1) * p.V + v0 + min(v, nv - 1)] : 0.f;
    return k < K && v < nv ? x : 0.f;
  };
#pragma unroll
  for (int a = 0; a < NK; ++a)
#pragma unroll
    for (int b = 0; b < OV; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) dkv[a][b][r] = entry(a * 16 + 4 * g + r, (wave + b * NW) * 16 + l);
#pragma unroll
  for (int a = 0; a < NV; ++a)
#pragma unroll
    for (int b = 0; b < OK; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) dvk[a][b][r] = entry((wave + b * NW) * 16 + l, a * 16 + 4 * g + r);

  struct Chunk {
    TileLoad<E, C, KP, 32, THREADS, TINY> q;
    TileLoad<E, C, KP, 16, THREADS, TINY> k;
    TileLoad<E, C, VT, 16, THREADS, TINY> v, d;
    float g;
  };
  auto fetch = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.q.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    x.v.load(vb + at * p.v_stride[1], p.v_stride[1], n, nv);
    x.d.load(db + at * p.do_stride[1], p.do_stride[1], n, nv);
    x.g = wave == 0 && lane < n ? gb[(at + lane) * p.g_stride[1]] : 0.f;
  };
  auto land = [&](const Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.q.store(qs, n, K);
    x.k.store(ks, n, K);
    x.v.store(vs, n, nv);
    x.d.store(ds, n, nv);
    if (wave == 0) scan_decays<C>(x.g, dec);
  };
  // wave 0, behind a barrier: the chunk's decay gradients from the waves' sums
  auto decay_gradient = [&](int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    float f = 0.f, e = 0.f, x = 0.f;
    if (lane < C) {
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        f += fs[w][lane] + (wrow[w][lane] - wcol[w][lane]);
        e += es[w][lane];
      }
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) x += xs[w];
    float before = __shfl_up(e, 1);  // the sum of e before a token, that of f from it on (scanned mirrored)
    before = wave_scan(lane == 0 ? 0.f : before);
    f = __shfl(wave_scan(__shfl(f, 63 - lane)), 63 - lane);
    if (lane < n) {
      const int64_t token = seg.start + at + lane;
      const float r = (f + before) + x;
      if (p.dg_part)
        p.dg_part[((int64_t)vt * p.map.tokens + token) * p.heads + head] = r;
      else
        p.dg[token * p.heads + head] = r;
    }
  };
  // a chunk's rows of a gradient of q or k: the gradient itself or this head's and tile's part
  const int part = (head % rep) * p.vtiles + vt;
  auto put_qk = [&](void* whole, float* parts, int64_t token, int n, int k, const f32x4 (&x)[1][NI]) {
    const int64_t stride = (int64_t)p.groups * K;
    if (parts)
      put_rows<NI, 1>(parts + ((part * p.map.tokens + token) * p.groups + group) * K, stride, n, K, k, 0, l, x);
    else
      put_rows<NI, 1>(static_cast<E*>(whole) + (token * p.groups + group) * K, stride, n, K, k, 0, l, x);
  };

  const int64_t chunks = (seg.end - seg.begin + C - 1) / C;
  if (chunks > 0) {
    Chunk x;
    fetch(x, seg.begin + (chunks - 1) * C);
    land(x, seg.begin + (chunks - 1) * C);
  }
  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int64_t at = seg.begin + c * C;
    const int n = (int)min((int64_t)C, seg.end - at);
    __syncthreads();  // the chunk has landed
    // the state before the chunk: rows v = 16 a + 4 g + r, own key columns
    f32x4 h[NV][OK];
    {
      const float* hb = p.chunk_state + ((chunk_number<C>(p.map, seg, at) * p.heads + head) * p.vtiles + vt) * (KP * VT);
#pragma unroll
      for (int b = 0; b < OK; ++b)
        if (wave + b * NW < NK)
#pragma unroll
          for (int a = 0; a < NV; ++a)
            h[a][b] = *reinterpret_cast<const f32x4*>(hb + ((a * NK + wave + b * NW) * 64 + lane) * 4);
    }
    __builtin_amdgcn_sched_barrier(0);  // here and below: phases in order, or their registers add up and spill

    // ---- S and D, transposed (rows j, columns i): 16 tokens i per JS waves, which take every JS-th tile of j
    {
      const int it = wave % NI, share = wave / NI, i = it * 16 + l;
      float rows = 0.f;
#pragma unroll
      for (int jt = 0; jt < NI; ++jt) {
        f32x4 cols = f32x4{0.f, 0.f, 0.f, 0.f};
        if (share < JS && jt % JS == share && jt <= (it | 1)) {  // the last may be all masked: pairs are read
          f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f}, d = s;
          if (jt <= it) {
#pragma unroll
            for (int x = 0; x < KP; x += 32) s = mma(frag_row(ks, jt * 16 + l, x), frag_row(qs, i, x), s);
#pragma unroll
            for (int x = 0; x < VT; x += 32) d = mma(frag_row(vs, jt * 16 + l, x), frag_row(ds, i, x), d);
          }
          const f32x4 e = dec.between4(i, jt * 16 + 4 * g) * p.scale;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = jt * 16 + 4 * g + r;
            const float smv = s[r] * e[r], dmv = d[r] * e[r], w = smv * d[r];
            cols[r] = j < i ? w : 0.f;
            rows += cols[r];
            s[r] = j <= i ? smv : 0.f;
            d[r] = j <= i ? dmv : 0.f;
          }
          put4(&sm.e[i * sm.stride + jt * 16 + 4 * g], s);
          put4(&dm.e[i * dm.stride + jt * 16 + 4 * g], d);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          cols[r] = row16_sum(cols[r]);
          if (l == 0) wcol[wave][jt * 16 + 4 * g + r] = cols[r];
        }
      }
      rows = across_rows(rows);
#pragma unroll
      for (int x = 0; x < NI; ++x)
        if (g == 0) wrow[wave][x * 16 + l] = x == it ? rows : 0.f;
    }
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);

    // ---- own keys: dq, dk, and the flows F, E, X
    const float all = __builtin_amdgcn_exp2f(dec.whole[C - 1] + dec.frac[C - 1]);
    float fsum[NI], esum[NI], xsum = 0.f;
#pragma unroll
    for (int x = 0; x < NI; ++x) fsum[x] = esum[x] = 0.f;
#pragma unroll
    for (int b = 0; b < OK; ++b)
      if (wave + b * NW < NK) {
        const int k0 = (wave + b * NW) * 16;
        f32x4 dq_[1][NI], dk_[1][NI];
        auto& dq = dq_[0];
        auto& dk = dk_[0];
#pragma unroll
        for (int x = 0; x < NI; ++x) dq[x] = dk[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int a = 0; a < NV; a += 2) {
          float u[8];
          Frag<E> hp[PF], dp[PF];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            u[r] = h[a][b][r];
            u[4 + r] = h[a + 1][b][r];
            xsum = fmaf(u[r], dvk[a][b][r], xsum);
            xsum = fmaf(u[4 + r], dvk[a + 1][b][r], xsum);
          }
          split_parts(u, hp);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            u[r] = dvk[a][b][r];
            u[4 + r] = dvk[a + 1][b][r];
          }
          split_parts(u, dp);
#pragma unroll
          for (int x = 0; x < NI; ++x) {
            const Frag<E> fd = frag_row_split(ds, x * 16 + l, a * 16), fv = frag_row_split(vs, x * 16 + l, a * 16);
#pragma unroll
            for (int q = 0; q < PF; ++q) {
              dq[x] = mma(hp[q], fd, dq[x]);
              dk[x] = mma(dp[q], fv, dk[x]);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const int i = x * 16 + l;
          dq[x] *= p.scale * __builtin_amdgcn_exp2f(dec.whole[i] + dec.frac[i]);
          dk[x] *= dec.between(C - 1, i);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            fsum[x] = fmaf(load1(&qs.e[i * qs.stride + k0 + 4 * g + r]), dq[x][r], fsum[x]);
            esum[x] = fmaf(load1(&ks.e[i * ks.stride + k0 + 4 * g + r]), dk[x][r], esum[x]);
          }
        }
#pragma unroll
        for (int j = 0; j < NI; j += 2) {
          const Frag<E> fk = frag_col_split(ks, j * 16, k0), fq = frag_col_split(qs, j * 16, k0);
#pragma unroll
          for (int x = 0; x < NI; ++x) {
            if (x >= j) dq[x] = mma(fk, frag_row_split(dm, x * 16 + l, j * 16), dq[x]);  // tokens j .. j + 31 before i
            if (x < j + 2) dk[x] = mma(fq, frag_col_split(dm, j * 16, x * 16), dk[x]);   // tokens i = j .. j + 31
          }
        }
        put_qk(p.dq, p.dq_part, seg.start + at, n, k0 + 4 * g, dq_);
        put_qk(p.dk, p.dk_part, seg.start + at, n, k0 + 4 * g, dk_);
      }
#pragma unroll
    for (int x = 0; x < NI; ++x) {
      fsum[x] = across_rows(fsum[x]);
      esum[x] = across_rows(esum[x]);
      if (g == 0) {
        fs[wave][x * 16 + l] = fsum[x];
        es[wave][x * 16 + l] = esum[x];
      }
    }
    xsum = wave_sum(xsum);
    if (lane == 0) xs[wave] = xsum * all;

    __builtin_amdgcn_sched_barrier(0);
    // the loads of the chunk before run beside the rest of this one's products (from its start on they would cost the
    // keys' phase its registers); always: a load under a condition would be waited for where the paths meet
    Chunk next;
    const int64_t ahead = c > 0 ? at - C : at;
    fetch(next, ahead);
    __builtin_amdgcn_sched_barrier(0);

    // ---- own values: dv
#pragma unroll
    for (int b = 0; b < OV; ++b) {
      const int w0 = (wave + b * NW) * 16;
      f32x4 dv_[1][NI];
      auto& dv = dv_[0];
#pragma unroll
      for (int x = 0; x < NI; ++x) dv[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int a = 0; a < NK; a += 2) {
        float u[8];
        Frag<E> dp[1];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          u[r] = dkv[a][b][r];
          u[4 + r] = dkv[a + 1][b][r];
        }
        split_parts(u, dp);
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const Frag<E> fk = frag_row_split(ks, x * 16 + l, a * 16);
          dv[x] = mma(dp[0], fk, dv[x]);
        }
      }
#pragma unroll
      for (int x = 0; x < NI; ++x) dv[x] *= dec.between(C - 1, x * 16 + l);
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const Frag<E> fd = frag_col_split(ds, j * 16, w0);
#pragma unroll
        for (int x = 0; x < NI; ++x)
          if (x < j + 2) dv[x] = mma(fd, frag_col_split(sm, j * 16, x * 16), dv[x]);
      }
      put_rows<NI, 1>(static_cast<E*>(p.dv) + ((seg.start + at) * p.heads + head) * p.V + v0, (int64_t)p.heads * p.V, n,
                      nv, w0 + 4 * g, 0, l, dv_);
    }

    __builtin_amdgcn_sched_barrier(0);

    // ---- d for the chunk before
#pragma unroll
    for (int a = 0; a < NK; ++a)
#pragma unroll
      for (int b = 0; b < OV; ++b) dkv[a][b] *= all;
#pragma unroll
    for (int a = 0; a < NV; ++a)
#pragma unroll
      for (int b = 0; b < OK; ++b) dvk[a][b] *= all;
#pragma unroll
    for (int j = 0; j < NI; j += 2) {
      const f32x4 f0 = dec.since4(j * 16 + 4 * g) * p.scale, f1 = dec.since4(j * 16 + 16 + 4 * g) * p.scale;
      Frag<E> fd[OV][PF];
#pragma unroll
      for (int b = 0; b < OV; ++b) {
        float u[8];
        frag_values(frag_col_split(ds, j * 16, (wave + b * NW) * 16), u);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          u[r] *= f0[r];
          u[4 + r] *= f1[r];
        }
        split_parts(u, fd[b]);
      }
#pragma unroll
      for (int a = 0; a < NK; ++a) {
        const Frag<E> fq = frag_col_split(qs, j * 16, a * 16);
#pragma unroll
        for (int b = 0; b < OV; ++b)
#pragma unroll
          for (int q = 0; q < PF; ++q) dkv[a][b] = mma(fq, fd[b][q], dkv[a][b]);
      }
#pragma unroll
      for (int b = 0; b < OK; ++b)
        if (wave + b * NW < NK) {
          float u[8];
          Frag<E> fq[PF];
          frag_values(frag_col_split(qs, j * 16, (wave + b * NW) * 16), u);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            u[r] *= f0[r];
            u[4 + r] *= f1[r];
          }
          split_parts(u, fq);
#pragma unroll
          for (int a = 0; a < NV; ++a) {
            const Frag<E> fv = frag_col_split(ds, j * 16, a * 16);
#pragma unroll
            for (int q = 0; q < PF; ++q) dvk[a][b] = mma(fv, fq[q], dvk[a][b]);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();  // the chunk has been read, the waves' sums are there
    if (wave == 0) decay_gradient(at);
    land(next, ahead);
  }

  if (seg.begin == 0 && p.dstate_in)
#pragma unroll
    for (int a = 0; a < NV; ++a)
#pragma unroll
      for (int b = 0; b < OK; ++b) {
        const int k = (wave + b * NW) * 16 + l, v = a * 16 + 4 * g;
        if (k < K) store4(p.dstate_in + qh + (int64_t)k * p.V + v0 + v, nv - v, dvk[a][b]);
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

// Byte offsets of the workspace's regions.
struct Regions {
  size_t chunk_state, seg_state, seg_dstate, seg_decay, seg_decay_back, dq_part, dk_part, dg_part, end;
  int parts;
};
Regions regions(const AttentionPlan& pl, int64_t tokens, int64_t groups, int64_t heads, int64_t K, int64_t V) {
  Regions r{};
  size_t at = 0;
  auto take = [&](int64_t floats) {
    const size_t here = at;
    at += ((size_t)floats * 4 + 255) / 256 * 256;
    return here;
  };
  r.parts = (int)(heads / groups) * pl.vtiles;
  r.chunk_state = take(pl.chunks * heads * pl.vtiles * pl.kp * pl.vt);
  r.seg_state = take(pl.split ? pl.slots * heads * K * V : 0);
  r.seg_dstate = take(pl.split ? pl.slots * heads * K * V : 0);
  r.seg_decay = take(pl.split ? pl.slots * heads : 0);
  r.seg_decay_back = take(pl.split ? pl.slots * heads : 0);
  r.dq_part = take(r.parts > 1 ? r.parts * tokens * groups * K : 0);
  r.dk_part = take(r.parts > 1 ? r.parts * tokens * groups * K : 0);
  r.dg_part = take(pl.vtiles > 1 ? pl.vtiles * tokens * heads : 0);
  r.end = at;
  return r;
}

template <typename E, int C, int VT, int NW>
hipError_t launch_k(const BackwardParams& p, const AttentionPlan& pl, hipStream_t st) {
  const dim3 grid = grid_of(p.blocks, NW * 64), block(NW * 64);
  if (pl.tiny) {
    attention_backward_kernel<E, C, 256, 64, 4, true><<<grid, dim3(256), 0, st>>>(p);
    return hipGetLastError();
  }
  switch (pl.kp) {
    case 32: attention_backward_kernel<E, C, 32, VT, NW, false><<<grid, block, 0, st>>>(p); break;
    case 64: attention_backward_kernel<E, C, 64, VT, NW, false><<<grid, block, 0, st>>>(p); break;
    case 128: attention_backward_kernel<E, C, 128, VT, NW, false><<<grid, block, 0, st>>>(p); break;
    default: attention_backward_kernel<E, C, 256, VT, NW, false><<<grid, block, 0, st>>>(p);
  }
  return hipGetLastError();
}

template <typename E>
hipError_t launch_sum(const float* parts, void* out, int n, int64_t per_token, const SequenceMap& map, hipStream_t st) {
  sum_parts<E><<<grid_of((map.tokens * per_token + 255) / 256, 256), dim3(256), 0, st>>>(
      parts, static_cast<E*>(out), n, per_token, map);
  return hipGetLastError();
}

}  // namespace

size_t attention_backward_workspace_bytes(const AttentionPlan& pl, int64_t tokens, int64_t groups, int64_t heads,
                                          int64_t key_dim, int64_t value_dim) {
  return regions(pl, tokens, groups, heads, key_dim, value_dim).end;
}

hipError_t launch_attention_backward(const AttentionBackwardArgs& a, const AttentionPlan& pl) {
  const AttentionArgs& f = a.f;
  const Regions rg = regions(pl, f.tokens, f.groups, f.heads, f.key_dim, f.value_dim);
  char* ws = static_cast<char*>(f.workspace);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };

  StateParams s{};
  s.g = f.log_decay;
  s.map = sequence_map(f, pl);
  s.seg_decay = at(rg.seg_decay);
  s.chunk_state = at(rg.chunk_state);
  s.groups = (int)f.groups;
  s.heads = (int)f.heads;
  s.K = (int)f.key_dim;
  s.V = (int)f.value_dim;
  s.tiles = pl.vtiles * (pl.vt / 64);
  count_blocks(s, pl);
  s.scale = f.scale;
  s.split = pl.split;
  for (int i = 0; i < 3; ++i) s.g_stride[i] = f.g_stride[i];
  s.k = f.k;
  s.v = f.v;
  s.state_in = f.state_in;
  s.seg_state = at(rg.seg_state);
  for (int i = 0; i < 3; ++i) {
    s.k_stride[i] = f.k_stride[i];
    s.v_stride[i] = f.v_stride[i];
  }
  hipError_t e = hipSuccess;
  if (pl.split) {  // the states before the segments and the gradients of those behind them
    StateParams r = s;
    r.k = f.q;
    r.v = a.d_o;
    r.state_in = a.dstate_out;
    r.seg_state = at(rg.seg_dstate);
    r.seg_decay = at(rg.seg_decay_back);
    for (int i = 0; i < 3; ++i) {
      r.k_stride[i] = f.q_stride[i];
      r.v_stride[i] = a.do_stride[i];
    }
    e = launch_segment_pair(s, r, pl, f.dtype, f.stream);
    if (e != hipSuccess) return e;
  }
  e = launch_chunk_states(s, pl, f.dtype, f.stream);
  if (e != hipSuccess) return e;

  BackwardParams p{};
  p.q = f.q;
  p.k = f.k;
  p.v = f.v;
  p.d_o = a.d_o;
  p.g = f.log_decay;
  p.dstate_out = a.dstate_out;
  p.seg_dstate = at(rg.seg_dstate);
  p.chunk_state = s.chunk_state;
  p.dq = a.dq;
  p.dk = a.dk;
  p.dv = a.dv;
  p.dg = a.dlog_decay;
  p.dstate_in = a.dstate_in;
  p.dq_part = rg.parts > 1 ? at(rg.dq_part) : nullptr;
  p.dk_part = rg.parts > 1 ? at(rg.dk_part) : nullptr;
  p.dg_part = pl.vtiles > 1 ? at(rg.dg_part) : nullptr;
  p.map = s.map;
  for (int i = 0; i < 3; ++i) {
    p.q_stride[i] = f.q_stride[i];
    p.k_stride[i] = f.k_stride[i];
    p.v_stride[i] = f.v_stride[i];
    p.do_stride[i] = a.do_stride[i];
    p.g_stride[i] = f.g_stride[i];
  }
  p.groups = s.groups;
  p.heads = s.heads;
  p.K = s.K;
  p.V = s.V;
  p.vtiles = pl.vtiles;
  p.blocks = (uint32_t)(pl.slots * f.heads * pl.vtiles);
  p.scale = f.scale;
  if (f.dtype == 1)
    e = pl.vt == 64 ? launch_k<uint16_t, 64, 64, 4>(p, pl, f.stream) : launch_k<uint16_t, 64, 128, 8>(p, pl, f.stream);
  else
    e = pl.vt == 64 ? launch_k<float, 32, 64, 4>(p, pl, f.stream) : launch_k<float, 32, 128, 8>(p, pl, f.stream);
  if (e == hipSuccess && rg.parts > 1) {
    const int64_t n = f.groups * f.key_dim;
    for (int i = 0; i < 2 && e == hipSuccess; ++i) {
      const float* from = i ? p.dk_part : p.dq_part;
      void* to = i ? a.dk : a.dq;
      e = f.dtype == 1 ? launch_sum<uint16_t>(from, to, rg.parts, n, p.map, f.stream)
                       : launch_sum<float>(from, to, rg.parts, n, p.map, f.stream);
    }
  }
  if (e == hipSuccess && pl.vtiles > 1) e = launch_sum<float>(p.dg_part, p.dg, pl.vtiles, f.heads, p.map, f.stream);
  return e;
}

}  // namespace ss2d
