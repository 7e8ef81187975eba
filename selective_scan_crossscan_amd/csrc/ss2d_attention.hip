// Linear attention with a decay per head, over prompts (gfx950).
//
//   h_t = exp(g_t) h_{t-1} + k_t v_t',   o_t = scale h_t' q_t.
//
// In chunks of C tokens, with G the sum of g inside the chunk up to a token and
// h the state before the chunk:
//   o_i = scale (sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j + exp(G_i) h' q_i),
//   h  <- exp(G_last) h + sum_j exp(G_last - G_j) k_j v_j'.
//
// One workgroup of four waves walks a segment of one sequence and head for VT
// value columns, chunk after chunk; the state never leaves its registers.  Each
// wave owns VT / 4 value columns: their part of the state (all key rows, fp32,
// as result tiles whose rows are the key index), of v and of the output.  The
// scores are the one thing waves share: each computes 16 tokens' (transposed,
// so that a lane has four consecutive keys' scores of one token), applies decay
// and mask, and puts them into LDS.  The output is formed transposed too, four
// consecutive columns of one token per lane.
//
// Few sequences and heads leave CUs idle, so sequences are then cut into
// segments: a first pass computes what each segment adds to a state from 0 and
// its whole decay, attention_carry turns these into the states before the
// segments, and the second pass starts from them.
#include "ss2d_attention.h"

namespace ss2d {

using namespace tok;

struct AttentionParams {
  const void *q, *k, *v;
  const float* g;
  const float* state_in;
  void* o;
  float* state_out;
  float* seg_state;  // (slot, head, K, V): what a segment adds, then the state before it
  float* seg_decay;  // (slot, head): the segment's whole decay
  SequenceMap map;
  int64_t q_stride[3], k_stride[3], v_stride[3], g_stride[3];
  int groups, heads, K, V, vtiles;
  float scale;
  bool split;  // second pass of segments: they start from seg_state
};

template <typename E, int C, int KP, int VT, bool STATE_ONLY>
__global__ __launch_bounds__(kAttThreads) void attention_kernel(AttentionParams p) {
  constexpr int NI = C / 16;        // token tiles
  constexpr int NK = KP / 16;       // key tiles
  constexpr int NV = VT / 64;       // value tiles of a wave
  constexpr int PF = kFullParts<E>, PH = kHalfParts<E>;
  __shared__ Tile<E, STATE_ONLY ? 1 : C, STATE_ONLY ? 1 : KP> qs;
  __shared__ Tile<E, C, KP> ks;
  __shared__ Tile<E, C, VT> vs;
  __shared__ Tile<E, STATE_ONLY ? 1 : C, STATE_ONLY ? 1 : C> ps;
  __shared__ Decays<C> dec;

  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const int vt = blockIdx.x % p.vtiles;
  const int head = (blockIdx.x / p.vtiles) % p.heads;
  const int64_t slot = blockIdx.x / (p.vtiles * p.heads);
  Segment seg;
  if (!find_segment(p.map, slot, seg)) return;
  if (STATE_ONLY && seg.last) return;  // nothing follows it
  const int group = head / (p.heads / p.groups);
  const int K = p.K, v0 = vt * VT, nv = min(p.V - v0, VT);
  const int vw = wave * (VT / 4);  // this wave's first column in the tile
  const bool active = vw < nv;     // it has columns at all
  const int64_t first = p.map.cu ? seg.start : 0, sq = p.map.cu ? 0 : seg.s;
  const E* qb = static_cast<const E*>(p.q) + sq * p.q_stride[0] + first * p.q_stride[1] + group * p.q_stride[2];
  const E* kb = static_cast<const E*>(p.k) + sq * p.k_stride[0] + first * p.k_stride[1] + group * p.k_stride[2];
  const E* vb = static_cast<const E*>(p.v) + sq * p.v_stride[0] + first * p.v_stride[1] + head * p.v_stride[2] + v0;
  const float* gb = p.g + sq * p.g_stride[0] + first * p.g_stride[1] + head * p.g_stride[2];

  // the state: rows 16 kt + 4 g + r, column vw + 16 t + l
  f32x4 h[NK][NV];
  const int64_t sh = ((int64_t)slot * p.heads + head) * K * p.V, qh = ((int64_t)seg.s * p.heads + head) * K * p.V;
  {
    const float* from = STATE_ONLY ? nullptr : p.split && seg.begin > 0 ? p.seg_state + sh
                                           : p.state_in ? p.state_in + qh : nullptr;
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = kt * 16 + 4 * g + r, v = vw + t * 16 + l;
          h[kt][t][r] = from && k < K && v < nv ? from[(int64_t)k * p.V + v0 + v] : 0.f;
        }
  }

  TileLoad<E, C, KP> ql, kl;
  TileLoad<E, C, VT> vl;
  float gl = 0.f;
  auto fetch = [&](int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    if (!STATE_ONLY) ql.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
    kl.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    vl.load(vb + at * p.v_stride[1], p.v_stride[1], n, nv);
    if (wave == 0) gl = lane < n ? gb[(at + lane) * p.g_stride[1]] : 0.f;
  };
  float whole = 0.f, frac = 0.f;  // the segment's log2 decay so far
  if (seg.begin < seg.end) fetch(seg.begin);
  for (int64_t at = seg.begin; at < seg.end; at += C) {
    const int n = (int)min((int64_t)C, seg.end - at);
    __syncthreads();  // the previous chunk has been read
    if constexpr (!STATE_ONLY) ql.store(qs);
    kl.store(ks);
    vl.store(vs);
    if (wave == 0) scan_decays<C>(gl, dec);
    __syncthreads();
    if (at + C < seg.end) fetch(at + C);

    if constexpr (!STATE_ONLY) {
      // scores, transposed: rows j (keys), columns i (tokens); 16 tokens per wave (two waves per 16 where C = 32)
      const int it = NI == 4 ? wave : wave >> 1;
      f32x4 s[NI];
#pragma unroll
      for (int jt = 0; jt < NI; ++jt) s[jt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KP; c += 32) {
        const Frag<E> b = frag_row(qs, it * 16 + l, c);
#pragma unroll
        for (int jt = 0; jt < NI; ++jt)
          if (jt <= it && (NI == 4 || jt == (wave & 1))) s[jt] = mma(frag_row(ks, jt * 16 + l, c), b, s[jt]);
      }
      const int i = it * 16 + l;
#pragma unroll
      for (int jt = 0; jt < NI; ++jt)
        if (jt <= (it | 1) && (NI == 4 || jt == (wave & 1))) {  // the last may be all masked: the output reads pairs
          f32x4 w;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = jt * 16 + 4 * g + r;
            w[r] = j <= i ? s[jt][r] * (p.scale * dec.between(i, j)) : 0.f;
          }
          put4(&ps.e[i * ps.stride + jt * 16 + 4 * g], w);
        }
      __syncthreads();

      if (active) {
        f32x4 o[NV][NI];
#pragma unroll
        for (int t = 0; t < NV; ++t)
#pragma unroll
          for (int x = 0; x < NI; ++x) o[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
        // h' q'
#pragma unroll
        for (int c = 0; c < NK; c += 2) {
          Frag<E> a[NV][PH];
#pragma unroll
          for (int t = 0; t < NV; ++t) {
            float x[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              x[r] = h[c][t][r];
              x[4 + r] = h[c + 1][t][r];
            }
            split_parts(x, a[t]);
          }
#pragma unroll
          for (int x = 0; x < NI; ++x) {
            const Frag<E> b = frag_row_split(qs, x * 16 + l, c * 16);
#pragma unroll
            for (int t = 0; t < NV; ++t)
#pragma unroll
              for (int q = 0; q < PH; ++q) o[t][x] = mma(a[t][q], b, o[t][x]);
          }
        }
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const float f = p.scale * __builtin_amdgcn_exp2f(dec.whole[x * 16 + l] + dec.frac[x * 16 + l]);
#pragma unroll
          for (int t = 0; t < NV; ++t) o[t][x] *= f;
        }
        // v' scores'
#pragma unroll
        for (int j = 0; j < NI; j += 2)
#pragma unroll
          for (int t = 0; t < NV; ++t) {
            const Frag<E> a = frag_col_split(vs, j * 16, vw + t * 16);
#pragma unroll
            for (int x = j; x < NI; ++x) o[t][x] = mma(a, frag_row_split(ps, x * 16 + l, j * 16), o[t][x]);
          }
        E* ob = static_cast<E*>(p.o) + ((seg.start + at) * p.heads + head) * p.V + v0;
#pragma unroll
        for (int x = 0; x < NI; ++x)
          if (x * 16 + l < n)
#pragma unroll
            for (int t = 0; t < NV; ++t) {
              const int v = vw + t * 16 + 4 * g;
              store4(ob + (int64_t)(x * 16 + l) * p.heads * p.V + v, nv - v, o[t][x]);
            }
      }
    }

    if (active) {
      const float a = __builtin_amdgcn_exp2f(dec.whole[C - 1] + dec.frac[C - 1]);
#pragma unroll
      for (int kt = 0; kt < NK; ++kt)
#pragma unroll
        for (int t = 0; t < NV; ++t) h[kt][t] *= a;
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> b[NV][PF];
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          float x[8];
          frag_values(frag_col_split(vs, j * 16, vw + t * 16), x);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r] *= dec.between(C - 1, j * 16 + 4 * g + r);
            x[4 + r] *= dec.between(C - 1, j * 16 + 16 + 4 * g + r);
          }
          split_parts(x, b[t]);
        }
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
          const Frag<E> k = frag_col_split(ks, j * 16, kt * 16);
#pragma unroll
          for (int t = 0; t < NV; ++t)
#pragma unroll
            for (int q = 0; q < PF; ++q) h[kt][t] = mma(k, b[t][q], h[kt][t]);
        }
      }
    }
    if (STATE_ONLY) {
      whole += dec.whole[C - 1];
      frac += dec.frac[C - 1];
    }
  }

  float* to = STATE_ONLY ? p.seg_state + sh : seg.last && p.state_out ? p.state_out + qh : nullptr;
  if (to)
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = kt * 16 + 4 * g + r, v = vw + t * 16 + l;
          if (k < K && v < nv) to[(int64_t)k * p.V + v0 + v] = h[kt][t][r];
        }
  if (STATE_ONLY && vt == 0 && threadIdx.x == 0)
    p.seg_decay[slot * p.heads + head] = __builtin_amdgcn_exp2f(whole + frac);
}

// seg_state: from what each segment adds to the state before it.  One thread per
// state entry walks its sequence's segments.
__global__ __launch_bounds__(kAttThreads) void attention_carry(AttentionParams p) {
  const int64_t kv = (int64_t)p.K * p.V;
  const int64_t blocks = (kv + kAttThreads - 1) / kAttThreads;
  const int64_t e = blockIdx.x % blocks * kAttThreads + threadIdx.x;
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
  float h = p.state_in ? p.state_in[((int64_t)s * p.heads + head) * kv + e] : 0.f;
  const int64_t step = p.heads * kv;
  float* u = p.seg_state + slot * step + head * kv + e;
  float add = len > p.map.seg_len ? *u : 0.f;  // what the segment adds
  for (int64_t at = 0; at + p.map.seg_len < len; at += p.map.seg_len, ++slot) {
    h = fmaf(p.seg_decay[slot * p.heads + head], h, add);
    u += step;
    if (at + 2 * p.map.seg_len < len) add = *u;
    *u = h;  // the state before the next segment
  }
}

namespace {

template <typename E, int C, int KP, int VT>
hipError_t launch_kv(const AttentionParams& p, const AttentionPlan& pl, hipStream_t st) {
  const dim3 grid((unsigned)(pl.slots * p.heads * pl.vtiles)), block(kAttThreads);
  if (pl.split) {
    attention_kernel<E, C, KP, VT, true><<<grid, block, 0, st>>>(p);
    const int64_t blocks = ((int64_t)p.K * p.V + kAttThreads - 1) / kAttThreads;
    attention_carry<<<dim3((unsigned)(blocks * p.heads * p.map.sequences)), block, 0, st>>>(p);
  }
  attention_kernel<E, C, KP, VT, false><<<grid, block, 0, st>>>(p);
  return hipGetLastError();
}

template <typename E, int C, int VT>
hipError_t launch_k(const AttentionParams& p, const AttentionPlan& pl, hipStream_t st) {
  switch (pl.kp) {
    case 32: return launch_kv<E, C, 32, VT>(p, pl, st);
    case 64: return launch_kv<E, C, 64, VT>(p, pl, st);
    case 128: return launch_kv<E, C, 128, VT>(p, pl, st);
    default: return launch_kv<E, C, 256, VT>(p, pl, st);
  }
}

}  // namespace

AttentionPlan plan_attention(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim,
                             bool packed, int dtype) {
  AttentionPlan pl;
  pl.kp = key_dim <= 32 ? 32 : key_dim <= 64 ? 64 : key_dim <= 128 ? 128 : 256;
  pl.vt = 64;
  pl.vtiles = (int)((value_dim + pl.vt - 1) / pl.vt);
  const int64_t chunk = dtype == 1 ? 64 : 32;
  // about two workgroups per CU, at least four chunks each
  const int64_t want = 512;
  int64_t seg = (tokens * heads * pl.vtiles + want - 1) / want;
  if (seg < 4 * chunk) seg = 4 * chunk;
  seg = (seg + chunk - 1) / chunk * chunk;
  const int64_t longest = packed ? tokens : tokens / sequences;
  pl.split = longest > seg;
  if (!pl.split) seg = (longest + chunk - 1) / chunk * chunk;
  pl.seg_len = seg;
  pl.nseg = (int)((longest + seg - 1) / seg);
  pl.slots = packed ? tokens / seg + sequences : sequences * pl.nseg;
  return pl;
}

size_t attention_workspace_bytes(const AttentionPlan& pl, int64_t heads, int64_t key_dim, int64_t value_dim) {
  return pl.split ? (size_t)(pl.slots * heads) * (size_t)(key_dim * value_dim + 1) * 4 : 0;
}

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& pl) {
  AttentionParams p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.g = a.log_decay;
  p.state_in = a.state_in;
  p.o = a.o;
  p.state_out = a.state_out;
  p.map = SequenceMap{a.cu, a.tokens, pl.seg_len, (int)a.sequences, pl.nseg, a.cu ? 0 : a.tokens / a.sequences};
  for (int i = 0; i < 3; ++i) {
    p.q_stride[i] = a.q_stride[i];
    p.k_stride[i] = a.k_stride[i];
    p.v_stride[i] = a.v_stride[i];
    p.g_stride[i] = a.g_stride[i];
  }
  p.groups = (int)a.groups;
  p.heads = (int)a.heads;
  p.K = (int)a.key_dim;
  p.V = (int)a.value_dim;
  p.vtiles = pl.vtiles;
  p.scale = a.scale;
  p.split = pl.split;
  if (pl.split) {
    p.seg_state = static_cast<float*>(a.workspace);
    p.seg_decay = p.seg_state + pl.slots * a.heads * a.key_dim * a.value_dim;
  }
  if (a.dtype == 1) return launch_k<uint16_t, 64, 64>(p, pl, a.stream);
  return launch_k<float, 32, 64>(p, pl, a.stream);
}

}  // namespace ss2d
