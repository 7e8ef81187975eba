// Linear attention with a decay per head: the passes that only form states.
//
// Walking a segment's chunks of C tokens, h <- exp(G_last) h + sum_j w_j k_j v_j'
// with w_j = exp(G_last - G_j); backwards, for the state's gradient,
// d <- exp(G_last) d + sum_i scale exp(G_i) q_i do_i': the same sum with q, do
// and other weights, chunks in reverse.
//
// One workgroup of four waves owns 64 value columns of a head and one segment; a
// wave owns 16 of them.  (128 columns would read the keys half as often, but took
// as long: more and smaller workgroups per CU hide more of the latency.)  The state
// is kept transposed (result tiles with rows v and columns k): a lane then holds four
// consecutive values of one key row for 16-byte accesses, and a pair of tiles is, as
// it lies in registers, an operand whose inner index is v.  The decayed v (do) goes
// into the product in parts that keep all of its bits.
//
// 38144 packed tokens, 16 heads of 128 in bf16: segment states 116 us, bound as the
// walk that follows, their carry 20 us for 30 segments' 31 MB read and written in
// order.  2 x 4096 tokens: states before all chunks 54 us (268 MB written, 5.0 TB/s),
// both ways' segments 45 us, their carries 20 us.
#include <type_traits>

#include "ss2d_attention.h"

namespace ss2d {
namespace {

using namespace tok;

template <typename E, int C, int KP>
struct StateTiles {
  Tile<E, C, KP, 32> ks;
  Tile<E, C, 64, 32> vs;
  Decays<C> dec;
};

// One segment's tile of 64 value columns; block: its number among the pass's.
template <typename E, int C, int KP, StatePass PASS, bool TINY>
__device__ __forceinline__ void state_walk(const StateParams& p, uint32_t block, StateTiles<E, C, KP>& lds) {
  constexpr bool REVERSE = PASS == kSegmentGradients;
  constexpr int VT = 64, NI = C / 16, NK = KP / 16, PF = kFullParts<E>;
  auto& ks = lds.ks;
  auto& vs = lds.vs;
  auto& dec = lds.dec;
  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const int vt = block % p.tiles;
  const int head = (block / p.tiles) % p.heads;
  const int64_t slot = block / (p.tiles * p.heads);
  Segment seg;
  if (!find_segment(p.map, slot, seg)) return;
  if (PASS == kSegmentStates ? seg.last : PASS == kSegmentGradients ? seg.begin == 0 : false) return;  // of no use
  const int group = head / (p.heads / p.groups);
  const int K = p.K, v0 = vt * VT, nv = min(p.V - v0, VT), vw = wave * 16;
  const bool active = vw < nv;
  const int64_t token0 = p.map.cu ? seg.start : 0, sq = p.map.cu ? 0 : seg.s;
  const E* kb = static_cast<const E*>(p.k) + sq * p.k_stride[0] + token0 * p.k_stride[1] + group * p.k_stride[2];
  const E* vb = static_cast<const E*>(p.v) + sq * p.v_stride[0] + token0 * p.v_stride[1] + head * p.v_stride[2] + v0;
  const float* gb = p.g + sq * p.g_stride[0] + token0 * p.g_stride[1] + head * p.g_stride[2];

  struct Chunk {
    TileLoad<E, C, KP, 32, 256, TINY> k;
    TileLoad<E, C, VT, 32, 256, TINY> v;
    float g;
  };
  auto fetch = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    x.v.load(vb + at * p.v_stride[1], p.v_stride[1], n, nv);
    x.g = wave == 0 && lane < n ? gb[(at + lane) * p.g_stride[1]] : 0.f;
  };
  auto land = [&](const Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.k.store(ks, n, K);
    x.v.store(vs, n, nv);
    if (wave == 0) scan_decays<C>(x.g, dec);
  };
  const int64_t chunks = (seg.end - seg.begin + C - 1) / C;
  auto start_of = [&](int64_t c) { return seg.begin + (REVERSE ? chunks - 1 - c : c) * C; };
  float whole = 0.f, frac = 0.f;  // the segment's log2 decay so far
  Chunk first;  // on its way while the state is read
  if (chunks > 0) fetch(first, start_of(0));

  // rows v = vw + 4 g + r, column k = 16 kt + l
  f32x4 h[NK];
  const int64_t sh = (slot * p.heads + head) * K * p.V;
  const float* from = PASS != kChunkStates              ? nullptr
                      : p.split && seg.several()        ? p.seg_state + sh
                      : p.state_in                      ? p.state_in + ((int64_t)seg.s * p.heads + head) * K * p.V
                                                        : nullptr;
  if (from)
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        h[kt][r] = from[(int64_t)min(kt * 16 + l, K - 1) * p.V + v0 + min(vw + 4 * g + r, nv - 1)];
#pragma unroll
  for (int kt = 0; kt < NK; ++kt)
#pragma unroll
    for (int r = 0; r < 4; ++r) h[kt][r] = from && kt * 16 + l < K && vw + 4 * g + r < nv ? h[kt][r] : 0.f;
  if (chunks > 0) land(first, start_of(0));
  for (int64_t c = 0; c < chunks; ++c) {
    if (PASS == kChunkStates) {  // before the chunk, as it lies in registers: 1 KiB per tile and wave
      const int64_t chunk = chunk_number<C>(p.map, seg, start_of(c));
      float* to = p.chunk_state + ((chunk * p.heads + head) * p.tiles + vt) * (KP * VT);
#pragma unroll
      for (int kt = 0; kt < NK; ++kt) *reinterpret_cast<f32x4*>(to + ((wave * NK + kt) * 64 + lane) * 4) = h[kt];
      if (c + 1 == chunks) break;  // the state behind the last chunk is not needed
    }
    __syncthreads();  // the chunk has landed
    // the next chunk's loads run beside this one's products; always, the last one's again: a load under a condition
    // would be waited for where the paths meet
    Chunk next;
    const int64_t ahead = start_of(c + 1 < chunks ? c + 1 : c);
    fetch(next, ahead);
    const float a = __builtin_amdgcn_exp2f(dec.whole[C - 1] + dec.frac[C - 1]);
    whole += dec.whole[C - 1];
    frac += dec.frac[C - 1];
    if (active) {
#pragma unroll
      for (int kt = 0; kt < NK; ++kt) h[kt] *= a;
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        const int i0 = j * 16 + 4 * g;
        const f32x4 w0 = REVERSE ? dec.since4(i0) * p.scale : dec.between4(C - 1, i0);
        const f32x4 w1 = REVERSE ? dec.since4(i0 + 16) * p.scale : dec.between4(C - 1, i0 + 16);
        Frag<E> b[PF];
        float x[8];
        frag_values(frag_col_split(vs, j * 16, vw), x);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] *= w0[r];
          x[4 + r] *= w1[r];
        }
        split_parts(x, b);
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
          const Frag<E> k = frag_col_split(ks, j * 16, kt * 16);
#pragma unroll
          for (int q = 0; q < PF; ++q) h[kt] = mma(b[q], k, h[kt]);
        }
      }
    }
    __syncthreads();  // the chunk has been read
    land(next, ahead);
  }
  if (PASS != kChunkStates) {
    const int v = vw + 4 * g;
#pragma unroll
    for (int kt = 0; kt < NK; ++kt) {
      const int k = kt * 16 + l;
      if (k < K) store4(p.seg_state + sh + (int64_t)k * p.V + v0 + v, nv - v, h[kt]);
    }
    if (vt == 0 && threadIdx.x == 0) p.seg_decay[slot * p.heads + head] = __builtin_amdgcn_exp2f(whole + frac);
  }
}

template <typename E, int C, int KP, StatePass PASS, bool TINY>
__global__ __launch_bounds__(256, KP <= 64 ? 4 : 2) void state_kernel(StateParams p) {
  __shared__ StateTiles<E, C, KP> lds;
  const uint32_t block = (uint32_t)block_id();
  if (block < p.blocks) state_walk<E, C, KP, PASS, TINY>(p, block, lds);
}

// What the segments add to the state and to its gradient, one after the other in
// one grid: each alone leaves CUs idle where sequences had to be cut.
template <typename E, int C, int KP, bool TINY>
__global__ __launch_bounds__(256, KP <= 64 ? 4 : 2) void state_pair_kernel(StateParams p, StateParams r) {
  __shared__ StateTiles<E, C, KP> lds;
  const uint32_t block = (uint32_t)block_id(), n = p.blocks;
  if (block < n)
    state_walk<E, C, KP, kSegmentStates, TINY>(p, block, lds);
  else if (block - n < n)
    state_walk<E, C, KP, kSegmentGradients, TINY>(r, block - n, lds);
}

// seg_state: from what each segment adds to the state before it, or, in reverse, to
// the gradient of the state behind it, for every segment of a sequence of several
// (the first one's is a copy of the initial state: the last segment's workgroup may
// write the final state over that one before the first has begun).  One thread per
// state entry walks its sequence's segments, eight sums read at a time.
__device__ __forceinline__ void carry_walk(const StateParams& p, const float* from, bool reverse, uint32_t block) {
  const int kv = p.K * p.V, blocks = (kv + 255) / 256;
  const int e = block % blocks * 256 + threadIdx.x, head = block / blocks % p.heads, s = block / blocks / p.heads;
  if (e >= kv) return;
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
  // along the walk: a segment's sum moves the state on, and what lies before (behind) the next one replaces its sum
  if (reverse) slot += n - 1;
  const int dir = reverse ? -1 : 1;
  const int64_t step = (int64_t)dir * p.heads * kv;
  float* u = p.seg_state + (slot * p.heads + head) * kv + e;
  const float* a = p.seg_decay + slot * p.heads + head;
  float h = from ? from[((int64_t)s * p.heads + head) * kv + e] : 0.f;
  constexpr int N = 8;
  float first = *u;  // the sum of segment i, kept: its place is overwritten
  *u = h;
  for (int64_t i = 0; i + 1 < n; i += N) {
    float add[N], decay[N];
    add[0] = first;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t at = i + j < n - 1 ? i + j : n - 1;  // a place inside, no branch around the load
      if (j > 0) add[j] = u[at * step];
      decay[j] = a[at * dir * p.heads];
    }
    first = u[(i + N < n - 1 ? i + N : n - 1) * step];
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (i + j + 1 < n) {
        h = fmaf(decay[j], h, add[j]);
        u[(i + j + 1) * step] = h;
      }
  }
}

__global__ __launch_bounds__(256) void state_carry(StateParams p, const float* from) {
  const uint32_t block = (uint32_t)block_id();
  if (block < p.carry_blocks) carry_walk(p, from, false, block);
}

__global__ __launch_bounds__(256) void state_carry_pair(StateParams p, const float* from, StateParams r,
                                                        const float* behind) {
  const uint32_t block = (uint32_t)block_id(), n = p.carry_blocks;
  if (block < n)
    carry_walk(p, from, false, block);
  else if (block - n < n)
    carry_walk(r, behind, true, block - n);
}

// Calls f with the padded key size and whether rows are tiny as constants.
template <typename F>
void with_keys(const AttentionPlan& pl, F f) {
  using std::integral_constant;
  if (pl.tiny)
    f(integral_constant<int, 256>(), integral_constant<bool, true>());
  else if (pl.kp == 32)
    f(integral_constant<int, 32>(), integral_constant<bool, false>());
  else if (pl.kp == 64)
    f(integral_constant<int, 64>(), integral_constant<bool, false>());
  else if (pl.kp == 128)
    f(integral_constant<int, 128>(), integral_constant<bool, false>());
  else
    f(integral_constant<int, 256>(), integral_constant<bool, false>());
}


template <typename E, int C>
void launch_single(StatePass pass, const StateParams& p, const AttentionPlan& pl, hipStream_t st) {
  with_keys(pl, [&](auto kp, auto tiny) {
    if (pass == kSegmentStates)
      state_kernel<E, C, kp(), kSegmentStates, tiny()><<<grid_of(p.blocks, 256), dim3(256), 0, st>>>(p);
    else
      state_kernel<E, C, kp(), kChunkStates, tiny()><<<grid_of(p.blocks, 256), dim3(256), 0, st>>>(p);
  });
}

template <typename E, int C>
void launch_pair(const StateParams& p, const StateParams& r, const AttentionPlan& pl, hipStream_t st) {
  with_keys(pl, [&](auto kp, auto tiny) {
    state_pair_kernel<E, C, kp(), tiny()><<<grid_of(2 * (int64_t)p.blocks, 256), dim3(256), 0, st>>>(p, r);
  });
}

}  // namespace

void count_blocks(StateParams& p, const AttentionPlan& pl) {
  p.blocks = (uint32_t)(pl.slots * p.heads * p.tiles);
  p.carry_blocks = (uint32_t)(((int64_t)p.K * p.V + 255) / 256 * p.heads * p.map.sequences);
}

hipError_t launch_segment_states(const StateParams& p, const AttentionPlan& pl, int dtype, hipStream_t st) {
  dtype == 1 ? launch_single<uint16_t, 64>(kSegmentStates, p, pl, st) : launch_single<float, 32>(kSegmentStates, p, pl, st);
  state_carry<<<grid_of(p.carry_blocks, 256), dim3(256), 0, st>>>(p, p.state_in);
  return hipGetLastError();
}

hipError_t launch_segment_pair(const StateParams& p, const StateParams& r, const AttentionPlan& pl, int dtype,
                               hipStream_t st) {
  dtype == 1 ? launch_pair<uint16_t, 64>(p, r, pl, st) : launch_pair<float, 32>(p, r, pl, st);
  state_carry_pair<<<grid_of(2 * (int64_t)p.carry_blocks, 256), dim3(256), 0, st>>>(p, p.state_in, r, r.state_in);
  return hipGetLastError();
}

hipError_t launch_chunk_states(const StateParams& p, const AttentionPlan& pl, int dtype, hipStream_t st) {
  dtype == 1 ? launch_single<uint16_t, 64>(kChunkStates, p, pl, st) : launch_single<float, 32>(kChunkStates, p, pl, st);
  return hipGetLastError();
}

}  // namespace ss2d
