// The gated delta rule over prompts: the walk over the chunks (ss2d_delta.h has the mathematics).
//
// One workgroup walks a segment of one sequence and head for VT value columns; a wave owns 16 NV of them, and the state,
// errors and outputs of its columns never leave its registers.  Keys, queries, values and the chunk's systems come
// through LDS, read by all waves.  Three passes share the walk: outputs; a segment's own part of the state and its map
// of the state before it; the states before all chunks and the errors, for the gradients.
//
// Few sequences and heads leave CUs idle, so sequences are then cut into segments.  What a segment does to the state is
// affine, h -> M h + u: u is the walk from 0, M (keys x keys) the walk from the identity with values 0, both by the same
// kernel, and a carry along the segments gives the states before them.
#include <type_traits>

#include "ss2d_delta.h"

namespace ss2d {
namespace {

using namespace tok;

constexpr int kCarryColumns = 32;

enum DeltaPass { kOutputs, kSegments, kStates };

template <typename E, int C, int KP, int VT, int NV, DeltaPass PASS, bool TINY>
__global__ __launch_bounds__(VT * 4 / NV, 2) void delta_walk(DeltaParams p) {
  constexpr int NW = VT / 16 / NV, THREADS = NW * 64, NI = C / 16, NK = KP / 16, PF = kFullParts<E>;
  using S = Systems<E, C>;
  constexpr int PN = S::kParts;
  constexpr int kSystem = PASS == kOutputs ? S::kForward : S::kInverse;  // bytes read per chunk
  constexpr int kPieces = (kSystem / 16 + THREADS - 1) / THREADS;
  __shared__ Tile<E, PASS == kOutputs ? C : 1, KP> qs;
  __shared__ Tile<E, C, KP, 16> ks;
  __shared__ Tile<E, C, VT, 32> vs;
  __shared__ __attribute__((aligned(16))) char sys[kSystem];
  __shared__ Rates<C> rates;

  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  uint32_t unit, at_tile;
  if (!spread((uint32_t)block_id(), p.blocks, PASS == kSegments ? p.vtiles + p.ktiles : p.vtiles, unit, at_tile)) return;
  const int tile = at_tile, head = unit % p.heads;
  const int64_t slot = unit / p.heads;
  Segment seg;
  if (!find_segment(p.map, slot, seg)) return;
  const bool map = PASS == kSegments && tile >= p.vtiles;  // columns of the identity instead of values
  if (PASS == kSegments && seg.last && !(map && p.last_maps && seg.begin > 0)) return;  // of no use
  const int group = head / (p.heads / p.groups);
  const int K = p.K, v0 = (map ? tile - p.vtiles : tile) * VT, nv = min((map ? KP : p.V) - v0, VT);
  const int vw = wave * 16 * NV;
  const bool active = vw < nv;
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
    TileLoad<E, PASS == kOutputs ? C : 1, KP, 16, THREADS, TINY> q;
    TileLoad<E, C, KP, 16, THREADS, TINY> k;
    TileLoad<E, C, VT, 32, THREADS, TINY> v;
    uint4 s[kPieces];
    float g, b;
  };
  auto fetch = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    if (PASS == kOutputs) x.q.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    if (!map) x.v.load(vb + at * p.v_stride[1], p.v_stride[1], n, nv);
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
    if (PASS == kOutputs) x.q.store(qs, n, K);
    x.k.store(ks, n, K);
    if (!map) x.v.store(vs, n, nv);
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (kSystem / 16 % THREADS == 0 || threadIdx.x + i * THREADS < kSystem / 16)
        *reinterpret_cast<uint4*>(sys + (threadIdx.x + i * THREADS) * 16) = x.s[i];
    if (wave == 0) scan_rates<C>(lane < n ? x.g : 0.f, lane < n ? x.b : 0.f, rates);
  };
  Chunk first;  // on its way while the state is read
  if (seg.begin < seg.end) fetch(first, seg.begin);

  // the state: rows 16 kt + 4 g + r, column vw + 16 t + l
  f32x4 h[NK][NV];
  const int64_t kv = (int64_t)K * p.V, sh = ((int64_t)slot * p.heads + head) * kv, qh = ((int64_t)seg.s * p.heads + head) * kv;
  const float* from = PASS == kSegments ? nullptr : p.split && seg.several() ? p.seg_state + sh : p.state_in ? p.state_in + qh : nullptr;
#pragma unroll
  for (int t = 0; t < NV; ++t) {
    const int v = vw + t * 16 + l;
    if (from) {
      const float* c = from + v0 + min(v, nv - 1);
#pragma unroll
      for (int kt = 0; kt < NK; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) h[kt][t][r] = c[(int64_t)min(kt * 16 + 4 * g + r, K - 1) * p.V];
    }
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = kt * 16 + 4 * g + r;
        h[kt][t][r] = from ? (k < K && v < nv ? h[kt][t][r] : 0.f) : map && k == v0 + v && k < K ? 1.f : 0.f;
      }
  }
  if (map)
    for (int i = threadIdx.x; i < C * vs.stride; i += THREADS) vs.e[i] = (E)0;
  if (seg.begin < seg.end) land(first, seg.begin);
  for (int64_t at = seg.begin; at < seg.end; at += C) {
    const int n = (int)min((int64_t)C, seg.end - at);
    __syncthreads();  // the chunk has landed
    // the next chunk's loads run beside this one's products; always, the last one's again: a load under a condition
    // would be waited for where the paths meet
    Chunk next;
    const int64_t ahead = at + C < seg.end ? at + C : at;
    fetch(next, ahead);

    if (active) {
      if (PASS == kStates) {
        float* to = p.chunk_state + ((chunk_number<C>(p.map, seg, at) * p.heads + head) * kv + v0);
#pragma unroll
        for (int t = 0; t < NV; ++t)
#pragma unroll
          for (int kt = 0; kt < NK; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int k = kt * 16 + 4 * g + r, v = vw + t * 16 + l;
              if (k < K && v < nv) to[k * p.V + v] = h[kt][t][r];
            }
      }
      f32x4 z[NI][NV], o[NV][NI];
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int x = 0; x < NI; ++x) z[x][t] = o[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
      // K h and h' Q'
#pragma unroll
      for (int c = 0; c < NK; c += 2) {
        Frag<E> b[NV][PF];
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          float u[8];
          stack(h[c][t], h[c + 1][t], u);
          split_parts(u, b[t]);
        }
        Frag<E> k[NI];
#pragma unroll
        for (int x = 0; x < NI; ++x) k[x] = frag_row_split(ks, x * 16 + l, c * 16);
#pragma unroll
        for (int q = PF - 1; q >= 0; --q)  // independent products next to each other
#pragma unroll
          for (int x = 0; x < NI; ++x)
#pragma unroll
            for (int t = 0; t < NV; ++t) z[x][t] = mma(k[x], b[t][q], z[x][t]);
        if (PASS == kOutputs)
#pragma unroll
          for (int x = 0; x < NI; ++x) {
            const Frag<E> f = frag_row_split(qs, x * 16 + l, c * 16);
#pragma unroll
            for (int t = 0; t < NV; ++t) o[t][x] = mma(b[t][0], f, o[t][x]);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (PASS == kOutputs)
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const float f = p.scale * rates.since[x * 16 + l];
#pragma unroll
          for (int t = 0; t < NV; ++t) o[t][x] *= f;
        }
      // the errors E = Z + N Z, Z = V - exp(G) K h
      f32x4 e[NV][NI];
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const f32x4 f0 = rates.four(&rates.since[j * 16 + 4 * g]), f1 = rates.four(&rates.since[j * 16 + 16 + 4 * g]);
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          float u[8];
          frag_values(frag_col_split(vs, j * 16, vw + t * 16), u);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            z[j][t][r] = fmaf(-f0[r], z[j][t][r], u[r]);
            z[j + 1][t][r] = fmaf(-f1[r], z[j + 1][t][r], u[4 + r]);
          }
          e[t][j] = z[j][t];
          e[t][j + 1] = z[j + 1][t];
        }
      }
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> a[NI][PN];
#pragma unroll
        for (int x = j; x < NI; ++x)
#pragma unroll
          for (int q = 0; q < PN; ++q) a[x][q] = system_frag<E>(sys + (S::lower(x, j / 2) * PN + q) * S::kFragBytes);
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          float u[8];
          Frag<E> b[PN];
          stack(z[j][t], z[j + 1][t], u);
          split_parts(u, b);
          j == 0 ? mma_parts<0, NI>(a, b, e[t]) : mma_parts<2, NI>(a, b, e[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (PASS == kStates) {
        float* to = p.errors + ((seg.start + at) * p.heads + head) * p.V + v0;
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
          for (int t = 0; t < NV; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int i = x * 16 + 4 * g + r, v = vw + t * 16 + l;
              if (i < n && v < nv) to[(uint32_t)i * (uint32_t)(p.heads * p.V) + v] = e[t][x][r];
            }
      }
      // U = b E; P U to the outputs, K' (w U) to the state
#pragma unroll
      for (int x = 0; x < NI; ++x) {
        const f32x4 b = rates.four(&rates.beta[x * 16 + 4 * g]);
#pragma unroll
        for (int t = 0; t < NV; ++t) e[t][x] *= b;
      }
      if (PASS == kOutputs) {
#pragma unroll
        for (int j = 0; j < NI; j += 2) {
          // two parts: the scores and the state are rounded once, and so is all that an output is made of
          constexpr int PU = PF > 1 ? 2 : 1;
          Frag<E> a[NV][PU];
#pragma unroll
          for (int t = 0; t < NV; ++t) {
            float u[8];
            stack(e[t][j], e[t][j + 1], u);
            split_parts(u, a[t]);
          }
#pragma unroll
          for (int x = j; x < NI; ++x) {
            const Frag<E> s = system_frag<E>(sys + S::kInverse + S::lower(x, j / 2) * S::kFragBytes);
#pragma unroll
            for (int q = PU - 1; q >= 0; --q)
#pragma unroll
              for (int t = 0; t < NV; ++t) o[t][x] = mma(a[t][q], s, o[t][x]);
          }
        }
        E* ob = static_cast<E*>(p.o) + ((seg.start + at) * p.heads + head) * p.V + v0;
        put_rows<NI, NV>(ob, (int64_t)p.heads * p.V, n, nv, vw + 4 * g, 16, l, o);
        __builtin_amdgcn_sched_barrier(0);  // the outputs' registers are free for what follows
      }
      const float all = rates.since[C - 1];
#pragma unroll
      for (int kt = 0; kt < NK; ++kt)
#pragma unroll
        for (int t = 0; t < NV; ++t) h[kt][t] *= all;
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> b[NV][PF];
        const f32x4 w0 = rates.four(&rates.left[j * 16 + 4 * g]), w1 = rates.four(&rates.left[j * 16 + 16 + 4 * g]);
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          float u[8];
          stack(e[t][j] * w0, e[t][j + 1] * w1, u);
          split_parts(u, b[t]);
        }
#pragma unroll
        for (int kt = 0; kt < NK; kt += 2) {
          const Frag<E> k0 = frag_col_split(ks, j * 16, kt * 16), k1 = frag_col_split(ks, j * 16, kt * 16 + 16);
#pragma unroll
          for (int q = PF - 1; q >= 0; --q)
#pragma unroll
            for (int t = 0; t < NV; ++t) {
              h[kt][t] = mma(k0, b[t][q], h[kt][t]);
              h[kt + 1][t] = mma(k1, b[t][q], h[kt + 1][t]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();  // the chunk has been read
    land(next, ahead);
  }

  float* to = PASS == kSegments ? (map ? p.seg_map + ((int64_t)slot * p.heads + head) * (KP * KP) : p.seg_state + sh)
              : PASS == kOutputs && seg.last && p.state_out ? p.state_out + qh : nullptr;
  if (to) {
    const int rows = map ? KP : K, step = map ? KP : p.V;
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = kt * 16 + 4 * g + r, v = vw + t * 16 + l;
          if (k < rows && v < nv) to[(int64_t)k * step + v0 + v] = h[kt][t][r];
        }
  }
}

// One workgroup carries 32 value columns of a head along its sequence's segments: h <- M h + u forwards, h <- M' h + u
// backwards, h before (behind) each segment in the place of its u.  The first one's too: the last segment's workgroup may
// write the final state over the initial one before the first has begun.  A wave owns 16 (at 256 keys 32) rows of the
// result and reads those of M alone, the next segment's while this one's are multiplied; h goes round through LDS as
// fragments in parts.  (With 16 columns per wave and all of M read by each, a step took 10 us where it takes 2.)
template <int KP, bool REVERSE>
__global__ __launch_bounds__(KP == 256 ? 512 : KP * 4) void delta_carry(CarryParams p) {
  constexpr int NK = KP / 16, NW = NK < 8 ? NK : 8, OWN = NK / NW, NC = KP / 32, NV = kCarryColumns / 16, PF = 3;
  __shared__ __attribute__((aligned(16))) uint32_t parts[2][NC][NV][PF][64][4];
  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const uint32_t block = (uint32_t)block_id();
  if (block >= p.blocks) return;
  const int tile = block % p.vtiles, head = block / p.vtiles % p.heads, s = block / p.vtiles / p.heads;
  int64_t slot, len;
  if (p.map.cu) {
    const int64_t start = cu_at(p.map, s), end = cu_at(p.map, s + 1);
    slot = start / p.map.seg_len + s;
    len = end - start;
  } else {
    slot = (int64_t)s * p.map.nseg;
    len = p.map.len;
  }
  const int64_t n = (len + p.map.seg_len - 1) / p.map.seg_len;  // segments
  if (n < 2) return;
  const int64_t kv = (int64_t)p.K * p.V;
  auto row = [&](int a, int r) { return (wave + a * NW) * 16 + 4 * g + r; };
  auto col = [&](int t) { return tile * kCarryColumns + t * 16 + l; };
  auto place = [&](int a, int t, int r) { return (int64_t)min(row(a, r), p.K - 1) * p.V + min(col(t), p.V - 1); };
  auto inside = [&](int a, int t, int r) { return row(a, r) < p.K && col(t) < p.V; };
  auto at = [&](int64_t i) { return (slot + (REVERSE ? n - 1 - i : i)) * p.heads + head; };
  f32x4 h[OWN][NV], add[OWN][NV];
  float m[OWN][NC][8];
  auto load = [&](int64_t i) {  // segment i's u and M
    const float *u = p.seg + at(i) * kv, *map = p.seg_map + at(i) * (KP * KP);
#pragma unroll
    for (int a = 0; a < OWN; ++a) {
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) add[a][t][r] = u[place(a, t, r)];
      const int k = (wave + a * NW) * 16 + l;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (REVERSE) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            m[a][c][r] = map[(c * 32 + 4 * g + r) * KP + k];
            m[a][c][4 + r] = map[(c * 32 + 16 + 4 * g + r) * KP + k];
          }
        } else {
          const float* x = map + k * KP + c * 32 + 4 * g;
          stack(*reinterpret_cast<const f32x4*>(x), *reinterpret_cast<const f32x4*>(x + 16), m[a][c]);
        }
      }
    }
  };
  load(0);
  const float* from = p.from ? p.from + ((int64_t)s * p.heads + head) * kv : nullptr;
#pragma unroll
  for (int a = 0; a < OWN; ++a)
#pragma unroll
    for (int t = 0; t < NV; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = from ? from[place(a, t, r)] : 0.f;
        h[a][t][r] = inside(a, t, r) ? x : 0.f;
      }
  for (int64_t i = 0; i < n; ++i) {
    float* u = p.seg + at(i) * kv;
#pragma unroll
    for (int a = 0; a < OWN; ++a)
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (inside(a, t, r)) u[place(a, t, r)] = h[a][t][r];
    if (i + 1 == n) break;
    auto& buffer = parts[i & 1];
#pragma unroll
    for (int a = 0; a < OWN; ++a)
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int k = wave + a * NW;
        f32x4 x = h[a][t];
#pragma unroll
        for (int q = 0; q < PF; ++q) {
          const uint32_t w[2] = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
          __builtin_memcpy(__builtin_assume_aligned(&buffer[k / 2][t][q][lane][2 * (k & 1)], 8), w, 8);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            x[2 * r] -= __uint_as_float(w[r] << 16);
            x[2 * r + 1] -= __uint_as_float(w[r] & 0xffff0000u);
          }
        }
      }
    Frag<uint16_t> f[OWN][NC][PF];
#pragma unroll
    for (int a = 0; a < OWN; ++a) {
#pragma unroll
      for (int c = 0; c < NC; ++c) split_parts(m[a][c], f[a][c]);
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) h[a][t][r] = inside(a, t, r) ? add[a][t][r] : 0.f;
    }
    __syncthreads();  // h is whole; the buffer is next written behind the next barrier
    load(i + 2 < n ? i + 1 : i);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        Frag<uint16_t> b[PF];
#pragma unroll
        for (int q = 0; q < PF; ++q) __builtin_memcpy(&b[q], __builtin_assume_aligned(buffer[c][t][q][lane], 16), 16);
#pragma unroll
        for (int x = PF - 1; x >= 0; --x)
#pragma unroll
          for (int q = 0; q <= x; ++q)
#pragma unroll
            for (int a = 0; a < OWN; ++a) h[a][t] = mma(f[a][c][q], b[x - q], h[a][t]);
      }
  }
}

// Calls f with the padded key size and whether rows are tiny as constants.
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

template <typename E, int C, DeltaPass PASS>
hipError_t launch_walk(DeltaParams p, const DeltaPlan& pl, hipStream_t st) {
  p.vtiles = (p.V + 63) / 64;
  p.ktiles = (pl.a.kp + 63) / 64;
  p.blocks = (uint32_t)(pl.a.slots * p.heads);
  const int64_t blocks = spread_blocks(p.blocks, PASS == kSegments ? p.vtiles + p.ktiles : p.vtiles);
  with_keys(pl, [&](auto kp, auto tiny) {
    delta_walk<E, C, kp(), 64, 1, PASS, tiny()><<<grid_of(blocks, 256), dim3(256), 0, st>>>(p);
  });
  return hipGetLastError();
}

// Chunks of 64 tokens (32 in fp32).  Sequences are cut so that there are about two workgroups per CU, packed ones, of which
// only some may be long, four; into three segments at least, as two would be walked twice for less than twice the speed.
// 16 heads of 128, us for 2, 3 and 4 workgroups per CU: 8192 tokens in one sequence 220, 258, 283, 38144 in six packed
// ones 897, 771, 750; gradients of 2 x 4096 tokens 718 (one 846, four 799).
DeltaPlan make_plan(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim, bool packed,
                    int dtype, int64_t want, int least) {
  DeltaPlan pl;
  AttentionPlan& a = pl.a;
  const int64_t few = dtype == 1 ? 8 : 4;  // values in 16 bytes
  a.tiny = key_dim < few || value_dim < few;
  a.kp = a.tiny ? 256 : key_dim <= 32 ? 32 : key_dim <= 64 ? 64 : key_dim <= 128 ? 128 : 256;
  a.vt = 64;
  a.vtiles = (int)((value_dim + 63) / 64);
  const int64_t chunk = a.chunk = dtype == 1 ? 64 : 32;
  const int64_t longest = packed ? tokens : tokens / sequences;
  if (packed && sequences > 1) want *= 2;
  const int64_t each = want / (heads * a.vtiles);  // segments of all sequences together
  int64_t parts = packed ? (each - sequences > each / 2 ? each - sequences : each / 2) : each / sequences;
  if (parts < 1) parts = 1;
  int64_t seg = (longest + parts - 1) / parts;
  if (seg < 4 * chunk) seg = 4 * chunk;
  seg = (seg + chunk - 1) / chunk * chunk;
  a.split = longest > (least - 1) * seg;
  if (!a.split) seg = (longest + chunk - 1) / chunk * chunk;
  a.seg_len = seg;
  a.nseg = (int)((longest + seg - 1) / seg);
  a.slots = packed ? tokens / seg + sequences : sequences * a.nseg;
  a.chunks = packed ? tokens / chunk + sequences : sequences * ((longest + chunk - 1) / chunk);
  return pl;
}

struct Regions {
  size_t systems, seg_state, seg_map, end;
};
Regions regions(const DeltaPlan& pl, int64_t heads, int64_t K, int64_t V, int dtype) {
  Regions r{};
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += ((size_t)bytes + 255) / 256 * 256;
    return here;
  };
  r.systems = take(pl.a.chunks * heads * system_bytes(pl, dtype));
  r.seg_state = take(pl.a.split ? pl.a.slots * heads * K * V * 4 : 0);
  r.seg_map = take(pl.a.split ? pl.a.slots * heads * pl.a.kp * pl.a.kp * 4 : 0);
  r.end = at;
  return r;
}

}  // namespace

DeltaPlan plan_delta(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim, bool packed,
                     int dtype) {
  DeltaPlan pl = make_plan(sequences, tokens, heads, key_dim, value_dim, packed, dtype, 512, 3);
  pl.backward = false;
  return pl;
}

DeltaPlan plan_delta_backward(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim,
                              bool packed, int dtype) {
  DeltaPlan pl = make_plan(sequences, tokens, heads, key_dim, value_dim, packed, dtype, 512, 3);
  pl.backward = true;
  return pl;
}

int64_t delta_blocks(const DeltaPlan& pl, int64_t sequences, int64_t heads, int64_t value_dim) {
  const int64_t v = (value_dim + 63) / 64, k = (pl.a.kp + 63) / 64;
  const int64_t walk = tok::spread_blocks(pl.a.slots * heads, (int)(v + k)), systems = pl.a.chunks * heads, carry = sequences * heads * ((value_dim + kCarryColumns - 1) / kCarryColumns);
  return walk > systems ? (walk > carry ? walk : carry) : systems > carry ? systems : carry;
}

size_t delta_workspace_bytes(const DeltaPlan& pl, int64_t heads, int64_t key_dim, int64_t value_dim, int dtype) {
  return regions(pl, heads, key_dim, value_dim, dtype).end;
}

DeltaParams delta_params(const DeltaArgs& a, const DeltaPlan& pl) {
  DeltaParams p{};
  const AttentionArgs& f = a.f;
  p.q = f.q;
  p.k = f.k;
  p.v = f.v;
  p.g = f.log_decay;
  p.beta = a.beta;
  p.state_in = f.state_in;
  p.o = f.o;
  p.state_out = f.state_out;
  p.map = sequence_map(f, pl.a);
  p.chunk_map = p.map;
  p.chunk_map.seg_len = pl.a.chunk;
  p.chunk_map.nseg = (int)((f.tokens / f.sequences + pl.a.chunk - 1) / pl.a.chunk);
  for (int i = 0; i < 3; ++i) {
    p.q_stride[i] = f.q_stride[i];
    p.k_stride[i] = f.k_stride[i];
    p.v_stride[i] = f.v_stride[i];
    p.g_stride[i] = f.g_stride[i];
    p.b_stride[i] = a.beta_stride[i];
  }
  p.groups = (int)f.groups;
  p.heads = (int)f.heads;
  p.K = (int)f.key_dim;
  p.V = (int)f.value_dim;
  p.scale = f.scale;
  p.split = pl.a.split;
  p.system_stride = system_bytes(pl, f.dtype);
  return p;
}

hipError_t launch_delta_segments(DeltaParams p, const DeltaPlan& pl, int dtype, hipStream_t st) {
  const hipError_t e = dtype == 1 ? launch_walk<uint16_t, 64, kSegments>(p, pl, st) : launch_walk<float, 32, kSegments>(p, pl, st);
  if (e != hipSuccess) return e;
  CarryParams c{p.seg_state, p.seg_map, p.state_in, p.map, p.heads, p.K, p.V, 0, 0};
  return launch_delta_carry(c, pl, false, st);
}

hipError_t launch_delta_carry(CarryParams c, const DeltaPlan& pl, bool reverse, hipStream_t st) {
  c.vtiles = (c.V + kCarryColumns - 1) / kCarryColumns;
  c.blocks = (uint32_t)((int64_t)c.map.sequences * c.heads * c.vtiles);
  with_keys(pl, [&](auto kp, auto) {
    constexpr int threads = kp() == 256 ? 512 : kp() * 4;
    const dim3 grid = grid_of(c.blocks, threads), block(threads);
    if (reverse)
      delta_carry<kp(), true><<<grid, block, 0, st>>>(c);
    else
      delta_carry<kp(), false><<<grid, block, 0, st>>>(c);
  });
  return hipGetLastError();
}

hipError_t launch_delta_states(DeltaParams p, const DeltaPlan& pl, int dtype, hipStream_t st) {
  return dtype == 1 ? launch_walk<uint16_t, 64, kStates>(p, pl, st) : launch_walk<float, 32, kStates>(p, pl, st);
}

hipError_t launch_delta(const DeltaArgs& a, const DeltaPlan& pl) {
  const AttentionArgs& f = a.f;
  const Regions rg = regions(pl, f.heads, f.key_dim, f.value_dim, f.dtype);
  char* ws = static_cast<char*>(f.workspace);
  DeltaParams p = delta_params(a, pl);
  p.systems = ws + rg.systems;
  p.seg_state = reinterpret_cast<float*>(ws + rg.seg_state);
  p.seg_map = reinterpret_cast<float*>(ws + rg.seg_map);
  hipError_t e = launch_delta_systems(p, pl, f.dtype, f.stream);
  if (e == hipSuccess && pl.a.split) e = launch_delta_segments(p, pl, f.dtype, f.stream);
  if (e != hipSuccess) return e;
  return f.dtype == 1 ? launch_walk<uint16_t, 64, kOutputs>(p, pl, f.stream) : launch_walk<float, 32, kOutputs>(p, pl, f.stream);
}

}  // namespace ss2d
