// Linear attention with a decay per head: the passes that only form states.
//
// Walking a segment's chunks of C tokens, h <- exp(G_last) h + sum_j w_j k_j v_j'
// with w_j = exp(G_last - G_j); backwards, for the state's gradient,
// d <- exp(G_last) d + sum_i scale exp(G_i) q_i do_i': the same sum with q, do
// and other weights, chunks in reverse.
//
// One workgroup of four waves owns a head's VT value columns of one segment; a
// wave owns VT / 4 of them.  The state is kept transposed (result tiles with
// rows v and columns k): a lane then holds four consecutive values of one key
// row for 16-byte accesses, and a pair of tiles is, as it lies in registers, an
// operand whose inner index is v.  The decayed v (do) goes into the product in
// parts that keep all of its bits.
#include "ss2d_attention.h"

namespace ss2d {
namespace {

using namespace tok;

template <typename E, int C, int KP, int VT, StatePass PASS, bool TINY>
__global__ __launch_bounds__(256, 2) void state_kernel(StateParams p) {
  constexpr bool REVERSE = PASS == kSegmentGradients;
  constexpr int NI = C / 16, NK = KP / 16, NV = VT / 64, PF = kFullParts<E>;
  __shared__ Tile<E, C, KP, 32> ks;
  __shared__ Tile<E, C, VT, 32> vs;
  __shared__ Decays<C> dec;
  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const int vt = blockIdx.x % p.vtiles;
  const int head = (blockIdx.x / p.vtiles) % p.heads;
  const int64_t slot = blockIdx.x / (p.vtiles * p.heads);
  Segment seg;
  if (!find_segment(p.map, slot, seg)) return;
  if (PASS == kSegmentStates ? seg.last : PASS == kSegmentGradients ? seg.begin == 0 : false) return;  // of no use
  const int group = head / (p.heads / p.groups);
  const int K = p.K, v0 = vt * VT, nv = min(p.V - v0, VT), vw = wave * (VT / 4);
  const bool active = vw < nv;
  const int64_t first = p.map.cu ? seg.start : 0, sq = p.map.cu ? 0 : seg.s;
  const E* kb = static_cast<const E*>(p.k) + sq * p.k_stride[0] + first * p.k_stride[1] + group * p.k_stride[2];
  const E* vb = static_cast<const E*>(p.v) + sq * p.v_stride[0] + first * p.v_stride[1] + head * p.v_stride[2] + v0;
  const float* gb = p.g + sq * p.g_stride[0] + first * p.g_stride[1] + head * p.g_stride[2];

  // rows v = vw + 16 t + 4 g + r, column k = 16 kt + l
  f32x4 h[NV][NK];
  const int64_t sh = (slot * p.heads + head) * K * p.V;
  const float* from = PASS != kChunkStates              ? nullptr
                      : p.split && seg.begin > 0        ? p.seg_state + sh
                      : p.state_in                      ? p.state_in + ((int64_t)seg.s * p.heads + head) * K * p.V
                                                        : nullptr;
  if (from)
#pragma unroll
    for (int t = 0; t < NV; ++t)
#pragma unroll
      for (int kt = 0; kt < NK; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          h[t][kt][r] = from[(int64_t)min(kt * 16 + l, K - 1) * p.V + v0 + min(vw + t * 16 + 4 * g + r, nv - 1)];
#pragma unroll
  for (int t = 0; t < NV; ++t)
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        h[t][kt][r] = from && kt * 16 + l < K && vw + t * 16 + 4 * g + r < nv ? h[t][kt][r] : 0.f;

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
  if (chunks > 0) {
    Chunk x;
    fetch(x, start_of(0));
    land(x, start_of(0));
  }
  for (int64_t c = 0; c < chunks; ++c) {
    if (PASS == kChunkStates) {  // before the chunk, as it lies in registers: 1 KiB per tile and wave
      float* to = p.chunk_state + ((chunk_number<C>(p.map, seg, start_of(c)) * p.heads + head) * p.vtiles + vt) * (KP * VT);
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
          *reinterpret_cast<f32x4*>(to + (((wave * NV + t) * NK + kt) * 64 + lane) * 4) = h[t][kt];
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
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) h[t][kt] *= a;
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> b[NV][PF];
        const int i0 = j * 16 + 4 * g;
        const f32x4 w0 = REVERSE ? dec.since4(i0) * p.scale : dec.between4(C - 1, i0);
        const f32x4 w1 = REVERSE ? dec.since4(i0 + 16) * p.scale : dec.between4(C - 1, i0 + 16);
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          float x[8];
          frag_values(frag_col_split(vs, j * 16, vw + t * 16), x);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r] *= w0[r];
            x[4 + r] *= w1[r];
          }
          split_parts(x, b[t]);
        }
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
          const Frag<E> k = frag_col_split(ks, j * 16, kt * 16);
#pragma unroll
          for (int q = 0; q < PF; ++q)
#pragma unroll
            for (int t = 0; t < NV; ++t) h[t][kt] = mma(b[t][q], k, h[t][kt]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();  // the chunk has been read
    land(next, ahead);
  }
  if (PASS != kChunkStates) {
#pragma unroll
    for (int t = 0; t < NV; ++t)
#pragma unroll
      for (int kt = 0; kt < NK; ++kt) {
        const int k = kt * 16 + l, v = vw + t * 16 + 4 * g;
        if (k < K) store4(p.seg_state + sh + (int64_t)k * p.V + v0 + v, nv - v, h[t][kt]);
      }
    if (vt == 0 && threadIdx.x == 0) p.seg_decay[slot * p.heads + head] = __builtin_amdgcn_exp2f(whole + frac);
  }
}

// One thread per state entry walks its sequence's segments.
__global__ __launch_bounds__(256) void state_carry(StateParams p, const float* from, bool reverse) {
  const int64_t kv = (int64_t)p.K * p.V;
  const int64_t blocks = (kv + 255) / 256;
  const int64_t e = blockIdx.x % blocks * 256 + threadIdx.x;
  const int head = (int)(blockIdx.x / blocks % p.heads), s = (int)(blockIdx.x / blocks / p.heads);
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
  // along the walk: the first segment's sum moves the state on, and what lies before (behind) the next one replaces its sum
  if (reverse) slot += n - 1;
  const int dir = reverse ? -1 : 1;
  const int64_t step = dir * p.heads * kv;
  float* u = p.seg_state + (slot * p.heads + head) * kv + e;
  float h = from ? from[((int64_t)s * p.heads + head) * kv + e] : 0.f;
  float add = *u;
  for (int64_t i = 0; i + 1 < n; ++i, slot += dir) {
    h = fmaf(p.seg_decay[slot * p.heads + head], h, add);
    u += step;
    if (i + 2 < n) add = *u;
    *u = h;
  }
}

template <typename E, int C, int VT, StatePass PASS>
hipError_t launch_k(const StateParams& p, const AttentionPlan& pl, hipStream_t st) {
  const dim3 grid((unsigned)(pl.slots * p.heads * pl.vtiles)), block(256);
  if (pl.tiny) {
    state_kernel<E, C, 256, 64, PASS, true><<<grid, block, 0, st>>>(p);
    return hipGetLastError();
  }
  switch (pl.kp) {
    case 32: state_kernel<E, C, 32, VT, PASS, false><<<grid, block, 0, st>>>(p); break;
    case 64: state_kernel<E, C, 64, VT, PASS, false><<<grid, block, 0, st>>>(p); break;
    case 128: state_kernel<E, C, 128, VT, PASS, false><<<grid, block, 0, st>>>(p); break;
    default: state_kernel<E, C, 256, VT, PASS, false><<<grid, block, 0, st>>>(p);
  }
  return hipGetLastError();
}

template <typename E, int C, int VT>
hipError_t launch_p(StatePass pass, const StateParams& p, const AttentionPlan& pl, hipStream_t st) {
  if (pass == kSegmentStates) return launch_k<E, C, VT, kSegmentStates>(p, pl, st);
  if (pass == kChunkStates) return launch_k<E, C, VT, kChunkStates>(p, pl, st);
  return launch_k<E, C, VT, kSegmentGradients>(p, pl, st);
}

}  // namespace

hipError_t launch_state_pass(StatePass pass, const StateParams& p, const AttentionPlan& pl, int dtype, hipStream_t st) {
  if (dtype == 1)
    return pl.vt == 64 ? launch_p<uint16_t, 64, 64>(pass, p, pl, st) : launch_p<uint16_t, 64, 128>(pass, p, pl, st);
  return pl.vt == 64 ? launch_p<float, 32, 64>(pass, p, pl, st) : launch_p<float, 32, 128>(pass, p, pl, st);
}

hipError_t launch_state_carry(bool reverse, const StateParams& p, const float* from, hipStream_t st) {
  const int64_t blocks = ((int64_t)p.K * p.V + 255) / 256;
  state_carry<<<dim3((unsigned)(blocks * p.heads * p.map.sequences)), dim3(256), 0, st>>>(p, from, reverse);
  return hipGetLastError();
}

}  // namespace ss2d
