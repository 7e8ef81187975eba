// The gated delta rule: the walks over the chunks, forwards and backwards, as what kernels of either kind, or of both,
// are made of (ss2d_delta.hip, ss2d_delta_backward.hip).
//
// One workgroup walks a segment of one sequence and head for VT value columns; a wave owns 16 of them, and the state,
// errors and outputs of its columns never leave its registers.  Keys, queries, values and the chunk's systems come
// through LDS, read by all waves.  Three passes share the forward walk: outputs; a segment's own part of the state and
// its map of the state before it; the states before all chunks and the errors, for the gradients.
//
// Bound by latency and issue, not by memory: of 16 x 2048 tokens, 16 heads of 128 in bf16, the outputs' walk takes
// 329 us, vector instructions 42% and matrix instructions 36% of the SIMDs' cycles, the waves waiting 38% of their time
// (chunk after chunk barriers, reads from LDS, and products that need the ones before).
#pragma once

#include <type_traits>

#include "ss2d_delta.h"

namespace ss2d {
namespace {

using namespace tok;

constexpr int kArrayTile = 64;  // columns of a tile of the chunks' arrays
// Whether the next chunk's loads wait in registers while one is worked on.  256 keys leave no registers for that, and
// are loaded when the chunk before has been read.  (128 keys, forward of 2 x 16384 tokens of 16 heads 701 us, loaded late
// 729; 2 x 2048 tokens 134 and 129.)
template <int KP>
constexpr bool kAhead = KP <= 128;

enum DeltaPass { kOutputs, kSegments, kStates };

template <typename E, int C, int KP, int VT, DeltaPass PASS>
struct WalkTiles {
  using S = Systems<E, C>;
  Tile<E, PASS == kOutputs ? C : 1, KP> qs;
  Tile<E, C, KP, 16> ks;
  Tile<E, C, VT, PASS == kOutputs ? 16 : 32> vs;  // 16: two workgroups' outputs fit a CU at 128 keys
  __attribute__((aligned(16))) char sys[(PASS == kOutputs ? 2 : 1) * S::kFrags * S::kParts * S::kFragBytes];
  Rates<C> rates;
};
template <typename E, int C, int KP, int VT, DeltaPass PASS, bool TINY>
__device__ __forceinline__ void walk(const DeltaParams& p, uint32_t block, WalkTiles<E, C, KP, VT, PASS>& lds) {
  constexpr int NW = VT / 16, THREADS = NW * 64, NI = C / 16, NK = KP / 16, PF = kFullParts<E>;
  using S = Systems<E, C>;
  constexpr int PN = S::kParts;
  constexpr int kSystem = PASS == kOutputs ? S::kForward : S::kOne;  // bytes read per chunk
  auto& qs = lds.qs;
  auto& ks = lds.ks;
  auto& vs = lds.vs;
  auto& sys = lds.sys;
  auto& rates = lds.rates;

  static_assert(PASS != kStates || VT == kArrayTile, "the chunks' arrays are in this walk's tiles");
  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  uint32_t unit, at_tile;
  if (!spread(block, p.blocks, PASS == kSegments ? p.vtiles + p.ktiles : p.vtiles, unit, at_tile)) return;
  const int tile = at_tile, head = unit % p.heads;
  const int64_t slot = unit / p.heads;  // of kSegments a part
  Segment seg;
  if (!find_segment(p.map, slot, seg, PASS == kSegments && p.cut)) return;
  const bool map = PASS == kSegments && tile >= p.vtiles;  // columns of the identity instead of values
  if (PASS == kSegments && seg.last && !(map && p.last_maps && seg.begin > 0)) return;  // of no use
  const int group = head / (p.heads / p.groups);
  const int K = p.K, v0 = (map ? tile - p.vtiles : tile) * VT, nv = min((map ? KP : p.V) - v0, VT);
  const int vw = wave * 16, v = vw + l;
  const uint32_t lane_at = 4 * (4 * g * kArrayTile + vw + l);  // bytes into a tile of the chunks' arrays
  const bool active = PASS == kStates || vw < nv;  // the chunks' arrays are written whole
  const int64_t token0 = p.map.cu ? seg.start : 0, sq = p.map.cu ? 0 : seg.s;
  const E* qb = static_cast<const E*>(p.q) + sq * p.q_stride[0] + token0 * p.q_stride[1] + group * p.q_stride[2];
  const E* kb = static_cast<const E*>(p.k) + sq * p.k_stride[0] + token0 * p.k_stride[1] + group * p.k_stride[2];
  const E* vb = static_cast<const E*>(p.v) + sq * p.v_stride[0] + token0 * p.v_stride[1] + head * p.v_stride[2] + (map ? 0 : v0);
  const float* gb = p.g + sq * p.g_stride[0] + token0 * p.g_stride[1] + head * p.g_stride[2];
  const float* bb = p.beta + sq * p.b_stride[0] + token0 * p.b_stride[1] + head * p.b_stride[2];
  const int64_t chunk0 = chunk_number<C>(p.map, seg, seg.begin);
  const char* sb = p.systems + (chunk0 * p.heads + head) * p.system_stride;
  const int64_t sstep = p.heads * p.system_stride;

  struct Chunk {
    TileLoad<E, PASS == kOutputs ? C : 1, KP, 16, THREADS, TINY && KP == 32> q;
    TileLoad<E, C, KP, 16, THREADS, TINY && KP == 32> k;
    TileLoad<E, C, VT, PASS == kOutputs ? 16 : 32, THREADS, TINY> v;
    SystemLoad<E, kSystem, THREADS> s;
    float g, b;
  };
  auto fetch_rest = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    const char* from = sb + (at - seg.begin) / C * sstep;
    x.s.load(from);
    const int64_t t = at + min(lane, n - 1);
    x.g = gb[t * p.g_stride[1]];
    x.b = bb[t * p.b_stride[1]];
  };
  auto land_rest = [&](const Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.s.store(sys);
    if (wave == 0) scan_rates<C>(lane < n ? x.g : 0.f, lane < n ? x.b : 0.f, rates);
  };
  auto fetch = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    if (PASS == kOutputs) x.q.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    if (!map) x.v.load(vb + at * p.v_stride[1], p.v_stride[1], n, nv);
  };
  auto land = [&](const Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    if (PASS == kOutputs) x.q.store(qs, n, K);
    x.k.store(ks, n, K);
    if (!map) x.v.store(vs, n, nv);
    land_rest(x, at);
  };
  auto bring = [&](int64_t at) {  // tile by tile, with few registers
    const int n = (int)min((int64_t)C, seg.end - at);
    Chunk x;
    if (PASS == kOutputs) {
      x.q.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
      x.q.store(qs, n, K);
      __builtin_amdgcn_sched_barrier(0);
    }
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    x.k.store(ks, n, K);
    __builtin_amdgcn_sched_barrier(0);
    if (!map) {
      x.v.load(vb + at * p.v_stride[1], p.v_stride[1], n, nv);
      x.v.store(vs, n, nv);
    }
    __builtin_amdgcn_sched_barrier(0);
    fetch_rest(x, at);
    land_rest(x, at);
  };
  Chunk first;  // on its way while the state is read
  if (kAhead<KP> && seg.begin < seg.end) {
    fetch(first, seg.begin);
    fetch_rest(first, seg.begin);
  }

  // the state: rows 16 kt + 4 g + r, column v
  f32x4 h[NK];
  const int64_t kv = (int64_t)K * p.V, qh = ((int64_t)seg.s * p.heads + head) * kv;
  const float* from = PASS == kSegments ? nullptr : p.split && seg.several() ? p.seg_state + (part_number(p.map, p.cut, seg) * p.heads + head) * kv : p.state_in ? p.state_in + qh : nullptr;
  if (from) {
    const float* c = from + v0 + min(v, nv - 1);
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) h[kt][r] = c[(int64_t)min(kt * 16 + 4 * g + r, K - 1) * p.V];
  }
#pragma unroll
  for (int kt = 0; kt < NK; ++kt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int k = kt * 16 + 4 * g + r;
      h[kt][r] = from ? (k < K && v < nv ? h[kt][r] : 0.f) : map && k == v0 + v && k < K ? 1.f : 0.f;
    }
  if (map)
    for (int i = threadIdx.x; i < C * vs.stride; i += THREADS) vs.e[i] = (E)0;
  if (seg.begin < seg.end) {
    if (kAhead<KP>)
      land(first, seg.begin);
    else
      bring(seg.begin);
  }
  for (int64_t at = seg.begin; at < seg.end; at += C) {
    const int n = (int)min((int64_t)C, seg.end - at);
    __syncthreads();  // the chunk has landed
    // the next chunk's loads run beside this one's products; always, the last one's again: a load under a condition
    // would be waited for where the paths meet
    Chunk next;
    const int64_t ahead = at + C < seg.end ? at + C : at;
    if (kAhead<KP>) fetch(next, ahead);
    if (kAhead<KP> && PASS != kOutputs) fetch_rest(next, ahead);

    if (active) {
      if (PASS == kStates) {
        float* to = by_bytes(p.chunk_state + ((chunk_number<C>(p.map, seg, at) * p.heads + head) * p.tiles + tile) * (KP * kArrayTile), lane_at);
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
          for (int r = 0; r < 4; ++r) to[(kt * 16 + r) * kArrayTile] = h[kt][r];
      }
      f32x4 z[NI], o[1][NI];
#pragma unroll
      for (int x = 0; x < NI; ++x) z[x] = o[0][x] = f32x4{0.f, 0.f, 0.f, 0.f};
      // K h and h' Q'
#pragma unroll
      for (int c = 0; c < NK; c += 2) {
        Frag<E> b[PF];
        float u[8];
        stack(h[c], h[c + 1], u);
        split_parts(u, b);
        Frag<E> k[NI];
#pragma unroll
        for (int x = 0; x < NI; ++x) k[x] = frag_row_split(ks, x * 16 + l, c * 16);
#pragma unroll
        for (int q = PF - 1; q >= 0; --q)  // independent products next to each other
#pragma unroll
          for (int x = 0; x < NI; ++x) z[x] = mma(k[x], b[q], z[x]);
        if (PASS == kOutputs)
#pragma unroll
          for (int x = 0; x < NI; ++x) {
            const Frag<E> f = frag_row_split(qs, x * 16 + l, c * 16);
#pragma unroll
            for (int q = PF - 1; q >= 0; --q) o[0][x] = mma(b[q], f, o[0][x]);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (PASS == kOutputs)
#pragma unroll
        for (int x = 0; x < NI; ++x) o[0][x] *= p.scale * rates.since[x * 16 + l];
      // the errors E = Z + N Z, Z = V - exp(G) K h
      f32x4 e[NI];
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const f32x4 f0 = rates.four(&rates.since[j * 16 + 4 * g]), f1 = rates.four(&rates.since[j * 16 + 16 + 4 * g]);
        float u[8];
        frag_values(frag_col_split(vs, j * 16, vw), u);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          z[j][r] = fmaf(-f0[r], z[j][r], u[r]);
          z[j + 1][r] = fmaf(-f1[r], z[j + 1][r], u[4 + r]);
        }
        e[j] = z[j];
        e[j + 1] = z[j + 1];
      }
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> a[NI][PN];
#pragma unroll
        for (int x = j; x < NI; ++x)
#pragma unroll
          for (int q = 0; q < PN; ++q) a[x][q] = system_frag<E>(sys, S::lower(x, j / 2), q);
        float u[8];
        Frag<E> b[PN];
        stack(z[j], z[j + 1], u);
        split_parts(u, b);
        j == 0 ? mma_parts<0, NI>(a, b, e) : mma_parts<2, NI>(a, b, e);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (PASS == kStates) {
        float* to = by_bytes(p.errors + ((chunk_number<C>(p.map, seg, at) * p.heads + head) * p.tiles + tile) * (C * kArrayTile), lane_at);
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) to[(x * 16 + r) * kArrayTile] = e[x][r];
      }
      // U = b E; P U to the outputs, K' (w U) to the state
#pragma unroll
      for (int x = 0; x < NI; ++x) e[x] *= rates.four(&rates.beta[x * 16 + 4 * g]);
      if (PASS == kOutputs) {
#pragma unroll
        for (int j = 0; j < NI; j += 2) {
          Frag<E> a[PF];
          float u[8];
          stack(e[j], e[j + 1], u);
          split_parts(u, a);
#pragma unroll
          for (int x = j; x < NI; ++x) {
            Frag<E> s[PF];
#pragma unroll
            for (int q = 0; q < PF; ++q) s[q] = system_frag<E>(sys, S::kFrags + S::lower(x, j / 2), q);
#pragma unroll
            for (int n = PF - 1; n >= 0; --n)
#pragma unroll
              for (int q = 0; q <= n; ++q) o[0][x] = mma(a[q], s[n - q], o[0][x]);
          }
        }
        E* ob = static_cast<E*>(p.o) + ((seg.start + at) * p.heads + head) * p.V + v0;
        put_rows<NI, 1>(ob, (int64_t)p.heads * p.V, n, nv, vw + 4 * g, 0, l, o);
        __builtin_amdgcn_sched_barrier(0);  // the outputs' registers are free for what follows
      }
      // The next systems, late, in registers that the outputs had; loads under the condition, alike for a wave's threads.
      if (kAhead<KP> && PASS == kOutputs) fetch_rest(next, ahead);
      const float all = rates.since[C - 1];
#pragma unroll
      for (int kt = 0; kt < NK; ++kt) h[kt] *= all;
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> b[PF];
        const f32x4 w0 = rates.four(&rates.left[j * 16 + 4 * g]), w1 = rates.four(&rates.left[j * 16 + 16 + 4 * g]);
        float u[8];
        stack(e[j] * w0, e[j + 1] * w1, u);
        split_parts(u, b);
#pragma unroll
        for (int kt = 0; kt < NK; kt += 2) {
          const Frag<E> k0 = frag_col_split(ks, j * 16, kt * 16), k1 = frag_col_split(ks, j * 16, kt * 16 + 16);
#pragma unroll
          for (int q = PF - 1; q >= 0; --q) {
            h[kt] = mma(k0, b[q], h[kt]);
            h[kt + 1] = mma(k1, b[q], h[kt + 1]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (kAhead<KP> && PASS == kOutputs && !active) fetch_rest(next, ahead);
    __syncthreads();  // the chunk has been read
    if (kAhead<KP>)
      land(next, ahead);
    else if (at + C < seg.end)  // all waves alike
      bring(ahead);
  }

  float* to = PASS == kSegments ? (map ? p.seg_map + (slot * p.heads + head) * (KP * KP) : p.seg_state + (slot * p.heads + head) * kv)
              : PASS == kOutputs && seg.last && p.state_out ? p.state_out + qh : nullptr;
  if (to) {
    const int rows = map ? KP : K, step = map ? KP : p.V;
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = kt * 16 + 4 * g + r;
        if (k < rows && v < nv) to[(int64_t)k * step + v0 + v] = h[kt][r];
      }
  }
}

struct BackParams {
  DeltaParams d;
  const void* d_o;
  int64_t do_stride[3];
  const float* dstate_out;  // or null
  float* seg_dstate;        // (part, head, K, V): what a segment adds, after the carry the gradient behind it
  float* chunk_dstate;      // (chunk, head, tile, KP, 64): D behind every chunk
  float* df;                // (chunk, head, tile, C, 64)
  float* inner;             // (chunk, head, 16-column tile): parts of sum_j u_j . (w K D)_j
  void *dq, *dk, *dv;
  float *dq_part, *dk_part;  // (part, token, group, K), or null: dq and dk themselves
  float *dg, *dbeta;
  float* dstate_in;         // or null
  int columns;              // 16-column tiles of `inner`
  uint32_t blocks;
};

template <typename E, int C, int KP, int VT>
struct BackTiles {
  using S = Systems<E, C>;
  Tile<E, C, KP, 16> qs, ks;  // 16 all: at 128 keys two workgroups of a pair of segment passes fit a CU
  Tile<E, C, VT, 16> ds;
  __attribute__((aligned(16))) char sys[2 * S::kFrags * S::kParts * S::kFragBytes];  // the transposed inverse and P'
  Rates<C> rates;
};
template <typename E, int C, int KP, int VT, bool SUM, bool TINY>
__device__ __forceinline__ void walk_back(const BackParams& b, uint32_t block, BackTiles<E, C, KP, VT>& lds) {
  const DeltaParams& p = b.d;
  constexpr int NW = VT / 16, THREADS = NW * 64, NI = C / 16, NK = KP / 16, PF = kFullParts<E>;
  using S = Systems<E, C>;
  constexpr int PN = S::kParts;
  constexpr int kSystem = S::kBackward - S::kOne;  // the transposed inverse and P'
  auto& qs = lds.qs;
  auto& ks = lds.ks;
  auto& ds = lds.ds;
  auto& sys = lds.sys;
  auto& rates = lds.rates;

  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  uint32_t unit, tile;
  if (!spread(block, b.blocks, p.vtiles, unit, tile)) return;
  const int vt = tile, head = unit % p.heads;
  const int64_t slot = unit / p.heads;  // of SUM a part
  Segment seg;
  if (!find_segment(p.map, slot, seg, SUM && p.cut)) return;
  if (SUM && seg.begin == 0) return;  // of no use
  const int group = head / (p.heads / p.groups);
  const int K = p.K, v0 = vt * VT, nv = min(p.V - v0, VT), v = wave * 16 + l;
  // in the chunks' arrays: this wave's tile, this lane's bytes into it
  const int array_tile = v0 / kArrayTile + wave * 16 / kArrayTile;
  const uint32_t lane_at = 4 * (4 * g * kArrayTile + wave * 16 % kArrayTile + l);
  const bool active = !SUM || wave * 16 < nv;  // the chunks' arrays are written whole
  const int64_t token0 = p.map.cu ? seg.start : 0, sq = p.map.cu ? 0 : seg.s;
  const E* qb = static_cast<const E*>(p.q) + sq * p.q_stride[0] + token0 * p.q_stride[1] + group * p.q_stride[2];
  const E* kb = static_cast<const E*>(p.k) + sq * p.k_stride[0] + token0 * p.k_stride[1] + group * p.k_stride[2];
  const E* db = static_cast<const E*>(b.d_o) + sq * b.do_stride[0] + token0 * b.do_stride[1] + head * b.do_stride[2] + v0;
  const float* gb = p.g + sq * p.g_stride[0] + token0 * p.g_stride[1] + head * p.g_stride[2];
  const float* bb = p.beta + sq * p.b_stride[0] + token0 * p.b_stride[1] + head * p.b_stride[2];
  const int64_t chunk0 = chunk_number<C>(p.map, seg, seg.begin);
  const char* sb = p.systems + (chunk0 * p.heads + head) * p.system_stride + S::kOne;
  const int64_t sstep = p.heads * p.system_stride;

  struct Chunk {
    TileLoad<E, C, KP, 16, THREADS, TINY && KP == 32> q, k;
    TileLoad<E, C, VT, 16, THREADS, TINY> d;
    SystemLoad<E, kSystem, THREADS> s;
    float g, b;
  };
  auto fetch_rest = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    const char* from = sb + (at - seg.begin) / C * sstep;
    x.s.load(from);
    const int64_t t = at + min(lane, n - 1);
    x.g = gb[t * p.g_stride[1]];
    x.b = bb[t * p.b_stride[1]];
  };
  auto land_rest = [&](const Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.s.store(sys);
    if (wave == 0) scan_rates<C>(lane < n ? x.g : 0.f, lane < n ? x.b : 0.f, rates);
  };
  auto fetch = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.q.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    x.d.load(db + at * b.do_stride[1], b.do_stride[1], n, nv);
    fetch_rest(x, at);
  };
  auto land = [&](const Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.q.store(qs, n, K);
    x.k.store(ks, n, K);
    x.d.store(ds, n, nv);
    land_rest(x, at);
  };
  auto bring = [&](int64_t at) {  // tile by tile, with few registers
    const int n = (int)min((int64_t)C, seg.end - at);
    Chunk x;
    x.q.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
    x.q.store(qs, n, K);
    __builtin_amdgcn_sched_barrier(0);
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    x.k.store(ks, n, K);
    __builtin_amdgcn_sched_barrier(0);
    x.d.load(db + at * b.do_stride[1], b.do_stride[1], n, nv);
    x.d.store(ds, n, nv);
    __builtin_amdgcn_sched_barrier(0);
    fetch_rest(x, at);
    land_rest(x, at);
  };
  const int64_t chunks = (seg.end - seg.begin + C - 1) / C;
  Chunk first;  // on its way while the gradient is read
  if (kAhead<KP> && chunks > 0) fetch(first, seg.begin + (chunks - 1) * C);

  // D: rows 16 kt + 4 g + r, column v
  f32x4 d[NK];
  const int64_t kv = (int64_t)K * p.V, qh = ((int64_t)seg.s * p.heads + head) * kv;
  const float* from = SUM ? nullptr : !seg.last ? b.seg_dstate + (part_number(p.map, p.cut, seg) * p.heads + head) * kv : b.dstate_out ? b.dstate_out + qh : nullptr;
#pragma unroll
  for (int kt = 0; kt < NK; ++kt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int k = kt * 16 + 4 * g + r;
      const float x = from ? from[(int64_t)min(k, K - 1) * p.V + v0 + min(v, nv - 1)] : 0.f;
      d[kt][r] = k < K && v < nv ? x : 0.f;
    }
  if (chunks > 0) {
    if (kAhead<KP>)
      land(first, seg.begin + (chunks - 1) * C);
    else
      bring(seg.begin + (chunks - 1) * C);
  }
  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int64_t at = seg.begin + c * C;
    __syncthreads();  // the chunk has landed
    const int64_t chunk = (chunk0 + c) * p.heads + head, place = chunk * p.tiles + array_tile;
    // The errors before the next chunk's loads and D's stores, all of which would be waited for with them otherwise
    // (memory operations are counted in order).
    f32x4 e[NI];
    const float* errors = by_bytes(p.errors + place * (C * kArrayTile), lane_at);
    if (!SUM)
#pragma unroll
      for (int x = 0; x < NI; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) e[x][r] = errors[(x * 16 + r) * kArrayTile];
    __builtin_amdgcn_sched_barrier(0);
    Chunk next;  // as in the forward
    const int64_t ahead = c > 0 ? at - C : at;
    if (kAhead<KP>) fetch(next, ahead);
    __builtin_amdgcn_sched_barrier(0);
    if (active) {
      if (!SUM) {
        float* to = by_bytes(b.chunk_dstate + place * (KP * kArrayTile), lane_at);
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
          for (int r = 0; r < 4; ++r) to[(kt * 16 + r) * kArrayTile] = d[kt][r];
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
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const f32x4 be = rates.four(&rates.beta[x * 16 + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) s = v < nv ? fmaf(be[r] * e[x][r], u[x][r], s) : s;
        }
        s = __shfl(wave_sum(s), 0);
        b.inner[chunk * b.columns + vt * NW + wave] = s;  // by all lanes, which have the same sum
      }
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const Frag<E> f = frag_col_split(ds, j * 16, wave * 16);
#pragma unroll
        for (int q = PF - 1; q >= 0; --q)
#pragma unroll
          for (int x = 0; x < j + 2; ++x)
            u[x] = mma(system_frag<E>(sys, S::kFrags + S::upper(x, j / 2), q), f, u[x]);
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
          for (int q = 0; q < PN; ++q) a[x][q] = system_frag<E>(sys, S::upper(x, j / 2), q);
        stack(u[j], u[j + 1], y);
        split_parts(y, f);
        j == 0 ? mma_parts<0, 2>(a, f, z) : mma_parts<0, NI>(a, f, z);
      }
      if (!SUM) {
        float* to = by_bytes(b.df + place * (C * kArrayTile), lane_at);
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) to[(x * 16 + r) * kArrayTile] = z[x][r];
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
    }
    __syncthreads();  // the chunk has been read
    if (kAhead<KP>)
      land(next, ahead);
    else if (c > 0)
      bring(ahead);
  }
  float* to = SUM ? b.seg_dstate + (slot * p.heads + head) * kv : seg.begin == 0 && b.dstate_in ? b.dstate_in + qh : nullptr;
  if (to)
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = kt * 16 + 4 * g + r;
        if (k < K && v < nv) to[(int64_t)k * p.V + v0 + v] = d[kt][r];
      }
}

// Calls f with the padded key size and whether rows are tiny as constants (the keys' only at 32 keys).
template <typename F>
void with_keys(const DeltaPlan& pl, F f) {
  using std::integral_constant;
  if (pl.a.tiny && pl.a.kp == 32)
    f(integral_constant<int, 32>(), integral_constant<bool, true>());
  else if (pl.a.tiny)
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

}  // namespace
}  // namespace ss2d
