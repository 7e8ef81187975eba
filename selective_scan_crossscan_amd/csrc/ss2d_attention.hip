// Linear attention with a decay per head, over prompts (gfx950).
//
//   h_t = exp(g_t) h_{t-1} + k_t v_t',   o_t = scale h_t' q_t.
//
// In chunks of C tokens, with G the sum of g inside the chunk up to a token and
// h the state before the chunk:
//   o_i = scale (sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j + exp(G_i) h' q_i),
//   h  <- exp(G_last) h + sum_j exp(G_last - G_j) k_j v_j'.
//
// One workgroup walks a segment of one sequence and head for VT value columns,
// chunk after chunk; the state never leaves its registers.  Each wave owns 16 value
// columns, 32 in tiles of 128 of up to 128 keys: their part of the state (all key rows, fp32, as result tiles
// whose rows are the key index), of v and of the output.  The
// scores are the one thing waves share: each computes 16 tokens' (transposed,
// so that a lane has four consecutive keys' scores of one token), applies decay
// and mask, and puts them into LDS.  The output is formed transposed too, four
// consecutive columns of one token per lane.
//
// Few sequences and heads leave CUs idle, so sequences are then cut into
// segments: a pass over keys and values computes what each segment adds to a
// state from 0 and its whole decay, a carry turns these into the states before
// the segments (ss2d_attention_state.hip), and the walk starts from them.
//
// 38144 packed tokens, 16 heads of 128 in bf16: the walk 227 to 243 us (240 in the
// middle: 2.7 TB/s, 167 TFLOP/s), the call with segments 319.  Bound by instruction issue and the latency between
// a chunk's barriers: vector instructions run in 35% of the busy cycles, LDS in 27%,
// matrix products in 22%, and it takes as long without its loads.  Two workgroups
// per CU: one with twice the LDS for two chunks took 271 us where two took 232.  In
// the 256 registers of two the 128 x 128 bf16 instance spills 24 (52 bytes a lane).
#include "ss2d_attention.h"

namespace ss2d {

using namespace tok;

struct AttentionParams {
  const void *q, *k, *v;
  const float* g;
  const float* state_in;
  void* o;
  float* state_out;
  const float* seg_state;  // (slot, head, K, V): the state before a segment
  SequenceMap map;
  uint32_t blocks;  // workgroups
  int64_t q_stride[3], k_stride[3], v_stride[3], g_stride[3];
  int groups, heads, K, V, vtiles;
  float scale;
  bool split;  // segments of a sequence of several start from seg_state
};

template <typename E, int C, int KP, int VT, int NV, bool TINY>
__global__ __launch_bounds__(VT * 4 / NV, 2) void attention_kernel(AttentionParams p) {
  constexpr int NW = VT / 16 / NV, THREADS = NW * 64;   // a wave owns NV tiles of 16 value columns
  constexpr int NI = C / 16;                            // token tiles
  constexpr int NK = KP / 16;                           // key tiles
  constexpr int JS = NW / NI < NI ? NW / NI : NI;       // waves that share 16 tokens' scores
  constexpr int PF = kFullParts<E>;
  __shared__ Tile<E, C, KP> qs;
  __shared__ Tile<E, C, KP, 32> ks;
  __shared__ Tile<E, C, VT, 32> vs;
  __shared__ Tile<E, C, C> ps;
  __shared__ Decays<C> dec;

  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const uint32_t block = (uint32_t)block_id();
  if (block >= p.blocks) return;  // asked first: behind the divisions 64 packed prompts of 64 tokens took 129 us, not 114
  const int vt = block % p.vtiles, head = block / p.vtiles % p.heads;
  const int64_t slot = block / (p.vtiles * p.heads);
  Segment seg;
  if (!find_segment(p.map, slot, seg)) return;
  const int group = head / (p.heads / p.groups);
  const int K = p.K, v0 = vt * VT, nv = min(p.V - v0, VT);
  const int vw = wave * 16 * NV;   // this wave's first column in the tile
  const bool active = vw < nv;     // it has columns at all
  const int64_t token0 = p.map.cu ? seg.start : 0, sq = p.map.cu ? 0 : seg.s;
  const E* qb = static_cast<const E*>(p.q) + sq * p.q_stride[0] + token0 * p.q_stride[1] + group * p.q_stride[2];
  const E* kb = static_cast<const E*>(p.k) + sq * p.k_stride[0] + token0 * p.k_stride[1] + group * p.k_stride[2];
  const E* vb = static_cast<const E*>(p.v) + sq * p.v_stride[0] + token0 * p.v_stride[1] + head * p.v_stride[2] + v0;
  const float* gb = p.g + sq * p.g_stride[0] + token0 * p.g_stride[1] + head * p.g_stride[2];

  struct Chunk {
    TileLoad<E, C, KP, 16, THREADS, TINY> q;
    TileLoad<E, C, KP, 32, THREADS, TINY> k;
    TileLoad<E, C, VT, 32, THREADS, TINY> v;
    float g;
  };
  auto fetch = [&](Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.q.load(qb + at * p.q_stride[1], p.q_stride[1], n, K);
    x.k.load(kb + at * p.k_stride[1], p.k_stride[1], n, K);
    x.v.load(vb + at * p.v_stride[1], p.v_stride[1], n, nv);
    x.g = wave == 0 && lane < n ? gb[(at + lane) * p.g_stride[1]] : 0.f;
  };
  auto land = [&](const Chunk& x, int64_t at) {
    const int n = (int)min((int64_t)C, seg.end - at);
    x.q.store(qs, n, K);
    x.k.store(ks, n, K);
    x.v.store(vs, n, nv);
    if (wave == 0) scan_decays<C>(x.g, dec);
  };
  Chunk first;  // on its way while the state is read
  if (seg.begin < seg.end) fetch(first, seg.begin);

  // the state: rows 16 kt + 4 g + r, column vw + 16 t + l
  f32x4 h[NK][NV];
  const int64_t sh = ((int64_t)slot * p.heads + head) * K * p.V, qh = ((int64_t)seg.s * p.heads + head) * K * p.V;
  const float* from = p.split && seg.several() ? p.seg_state + sh : p.state_in ? p.state_in + qh : nullptr;
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
      for (int r = 0; r < 4; ++r) h[kt][t][r] = from && kt * 16 + 4 * g + r < K && v < nv ? h[kt][t][r] : 0.f;
  }
  if (seg.begin < seg.end) land(first, seg.begin);
  for (int64_t at = seg.begin; at < seg.end; at += C) {
    const int n = (int)min((int64_t)C, seg.end - at);
    __syncthreads();  // the chunk has landed
    // the next chunk's loads run beside this one's products; always, the last one's again: a load under a condition
    // would be waited for where the paths meet
    Chunk next;
    const int64_t ahead = at + C < seg.end ? at + C : at;
    fetch(next, ahead);

    // scores, transposed (rows j, columns i): 16 tokens i per JS waves, which take every JS-th tile of keys j
    {
      const int it = wave % NI, share = wave / NI, i = it * 16 + l;
#pragma unroll
      for (int jt = 0; jt < NI; ++jt)
        if (share < JS && jt % JS == share && jt <= (it | 1)) {  // the last may be all masked: pairs are read
          f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
          if (jt <= it)
#pragma unroll
            for (int c = 0; c < KP; c += 32) s = mma(frag_row(ks, jt * 16 + l, c), frag_row(qs, i, c), s);
          const f32x4 e = dec.between4(i, jt * 16 + 4 * g);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float w = s[r] * (p.scale * e[r]);
            s[r] = jt * 16 + 4 * g + r <= i ? w : 0.f;
          }
          put4(&ps.e[i * ps.stride + jt * 16 + 4 * g], s);
        }
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
        Frag<E> a[NV][1];
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          float u[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            u[r] = h[c][t][r];
            u[4 + r] = h[c + 1][t][r];
          }
          split_parts(u, a[t]);
        }
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const Frag<E> b = frag_row_split(qs, x * 16 + l, c * 16);
#pragma unroll
          for (int t = 0; t < NV; ++t) o[t][x] = mma(a[t][0], b, o[t][x]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int x = 0; x < NI; ++x) {
        const float f = p.scale * __builtin_amdgcn_exp2f(dec.whole[x * 16 + l] + dec.frac[x * 16 + l]);
#pragma unroll
        for (int t = 0; t < NV; ++t) o[t][x] *= f;
      }
      // v' scores'
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> a[NV];
#pragma unroll
        for (int t = 0; t < NV; ++t) a[t] = frag_col_split(vs, j * 16, vw + t * 16);
#pragma unroll
        for (int x = j; x < NI; ++x) {
          const Frag<E> s = frag_row_split(ps, x * 16 + l, j * 16);
#pragma unroll
          for (int t = 0; t < NV; ++t) o[t][x] = mma(a[t], s, o[t][x]);
        }
      }
      E* ob = static_cast<E*>(p.o) + ((seg.start + at) * p.heads + head) * p.V + v0;
      put_rows<NI, NV>(ob, (int64_t)p.heads * p.V, n, nv, vw + 4 * g, 16, l, o);
      __builtin_amdgcn_sched_barrier(0);  // the outputs' registers are free for what follows

      // k' (decayed v)
      const float all = __builtin_amdgcn_exp2f(dec.whole[C - 1] + dec.frac[C - 1]);
#pragma unroll
      for (int kt = 0; kt < NK; ++kt)
#pragma unroll
        for (int t = 0; t < NV; ++t) h[kt][t] *= all;
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        Frag<E> b[NV][PF];
        const f32x4 w0 = dec.between4(C - 1, j * 16 + 4 * g), w1 = dec.between4(C - 1, j * 16 + 16 + 4 * g);
#pragma unroll
        for (int t = 0; t < NV; ++t) {
          float u[8];
          frag_values(frag_col_split(vs, j * 16, vw + t * 16), u);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            u[r] *= w0[r];
            u[4 + r] *= w1[r];
          }
          split_parts(u, b[t]);
        }
#pragma unroll
        for (int kt = 0; kt < NK; ++kt) {
          const Frag<E> k = frag_col_split(ks, j * 16, kt * 16);
#pragma unroll
          for (int q = 0; q < PF; ++q)
#pragma unroll
            for (int t = 0; t < NV; ++t) h[kt][t] = mma(k, b[t][q], h[kt][t]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();  // the chunk has been read
    land(next, ahead);
  }

  if (seg.last && p.state_out)
#pragma unroll
    for (int kt = 0; kt < NK; ++kt)
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = kt * 16 + 4 * g + r, v = vw + t * 16 + l;
          if (k < K && v < nv) p.state_out[qh + (int64_t)k * p.V + v0 + v] = h[kt][t][r];
        }
}

namespace {

template <typename E, int C, int VT>
hipError_t launch_k(const AttentionParams& p, const AttentionPlan& pl, hipStream_t st) {
  constexpr int NV = VT / 64;
  const dim3 grid = grid_of(p.blocks, pl.kp == 256 && !pl.tiny ? VT * 4 : 256);
  if (pl.tiny) {
    attention_kernel<E, C, 256, 64, 1, true><<<grid, dim3(256), 0, st>>>(p);
    return hipGetLastError();
  }
  switch (pl.kp) {
    case 32: attention_kernel<E, C, 32, VT, NV, false><<<grid, dim3(256), 0, st>>>(p); break;
    case 64: attention_kernel<E, C, 64, VT, NV, false><<<grid, dim3(256), 0, st>>>(p); break;
    case 128: attention_kernel<E, C, 128, VT, NV, false><<<grid, dim3(256), 0, st>>>(p); break;
    default: attention_kernel<E, C, 256, VT, 1, false><<<grid, dim3(VT * 4), 0, st>>>(p);
  }
  return hipGetLastError();
}

int64_t chunk_of(int dtype) { return dtype == 1 ? 64 : 32; }
bool tiny_rows(int64_t key_dim, int64_t value_dim, int dtype) {
  const int64_t least = dtype == 1 ? 8 : 4;  // values in 16 bytes
  return key_dim < least || value_dim < least;
}

// The plan for tiles of vt value columns.  Sequences are cut so that there are
// about `want` workgroups and no more: a few over a whole number per CU would
// cost as long as a full round.  Equal lengths are cut evenly; packed ones every
// tokens / (want per head and tile, less one ragged end per sequence) tokens,
// and where those ends would take a quarter of them, for twice as many (gradients
// of 38144 tokens in 6 sequences, 16 heads of 128: 1203 us against 1428; 8192 in
// one, whose ends take less, 333 against 282).  Segments have four chunks at least,
// and there are `least` of them or the sequences stay whole.
AttentionPlan make_plan(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim,
                        bool packed, int dtype, int vt, int64_t want, int least) {
  AttentionPlan pl;
  pl.tiny = tiny_rows(key_dim, value_dim, dtype);
  if (pl.tiny) vt = 64;
  pl.kp = pl.tiny ? 256 : key_dim <= 32 ? 32 : key_dim <= 64 ? 64 : key_dim <= 128 ? 128 : 256;
  pl.vt = vt;
  pl.vtiles = (int)((value_dim + vt - 1) / vt);
  const int64_t chunk = pl.chunk = chunk_of(dtype);
  const int64_t longest = packed ? tokens : tokens / sequences;
  int64_t each = want / (heads * pl.vtiles);  // segments of all sequences together
  for (; packed && 4 * sequences >= each && want < 1024; want *= 2) each = 2 * want / (heads * pl.vtiles);
  int64_t parts = packed ? (each - sequences > each / 2 ? each - sequences : each / 2) : each / sequences;
  if (parts < 1) parts = 1;
  int64_t seg = (longest + parts - 1) / parts;
  if (seg < 4 * chunk) seg = 4 * chunk;
  seg = (seg + chunk - 1) / chunk * chunk;
  pl.split = longest > (least - 1) * seg;
  if (!pl.split) seg = (longest + chunk - 1) / chunk * chunk;
  pl.seg_len = seg;
  pl.nseg = (int)((longest + seg - 1) / seg);
  pl.slots = packed ? tokens / seg + sequences : sequences * pl.nseg;
  pl.chunks = packed ? tokens / chunk + sequences : sequences * ((longest + chunk - 1) / chunk);
  return pl;
}

}  // namespace

AttentionPlan plan_attention(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim,
                             bool packed, int dtype) {
  // Tiles of 64 value columns for the wide heads of few tokens, which leave CUs idle; they read the keys twice.  16
  // heads of 128, us of tiles of 64 against 128: 256 tokens 21 (28), 2048 tokens 45 (54), 2 x 4096 92 (94), 38144
  // tokens 460 (314).  Two workgroups per CU: 38144 tokens for 256, 512 and 1024 workgroups 502, 327 and 336 us.
  // Three segments at least: 16 x 4096 tokens in two each 464 us, whole 371; 9 x 4096 in three 290, whole 364.
  const bool narrow = tokens / (4 * chunk_of(dtype)) * heads * ((value_dim + 63) / 64) <= 512;
  return make_plan(sequences, tokens, heads, key_dim, value_dim, packed, dtype, value_dim <= 64 || narrow ? 64 : 128,
                   512, 3);
}

AttentionPlan plan_attention_backward(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim,
                                      int64_t value_dim, bool packed, int dtype) {
  // One tile of value columns where they fit: a second one would make dq and dk sums of two parts in memory.  A
  // workgroup fills a CU's LDS unless the keys are narrow: 2 x 4096 tokens, 16 heads of 128, for 256 and 512
  // workgroups 270 and 309 us, 8192 tokens of 16 x 64 x 64 131 and 152, of 16 x 32 x 64 100 and 85.  Two segments pay
  // here, where the states are formed in any case: 8 x 8192 tokens 1669 us, whole 2316.
  return make_plan(sequences, tokens, heads, key_dim, value_dim, packed, dtype, value_dim <= 64 ? 64 : 128,
                   key_dim <= 32 ? 512 : 256, 2);
}

SequenceMap sequence_map(const AttentionArgs& a, const AttentionPlan& pl) {
  return SequenceMap{a.cu, a.tokens, pl.seg_len, (int)a.sequences, pl.nseg, a.cu ? 0 : a.tokens / a.sequences};
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
  p.map = sequence_map(a, pl);
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
  p.blocks = (uint32_t)(pl.slots * a.heads * pl.vtiles);
  p.scale = a.scale;
  p.split = pl.split;
  if (pl.split) {
    StateParams s{};
    s.k = a.k;
    s.v = a.v;
    s.g = a.log_decay;
    s.seg_state = static_cast<float*>(a.workspace);
    s.seg_decay = s.seg_state + pl.slots * a.heads * a.key_dim * a.value_dim;
    s.map = p.map;
    for (int i = 0; i < 3; ++i) {
      s.k_stride[i] = a.k_stride[i];
      s.v_stride[i] = a.v_stride[i];
      s.g_stride[i] = a.g_stride[i];
    }
    s.groups = p.groups;
    s.heads = p.heads;
    s.K = p.K;
    s.V = p.V;
    s.tiles = (int)((a.value_dim + 63) / 64);
    count_blocks(s, pl);
    s.state_in = a.state_in;
    p.seg_state = s.seg_state;
    const hipError_t e = launch_segment_states(s, pl, a.dtype, a.stream);
    if (e != hipSuccess) return e;
  }
  if (a.dtype == 1)
    return pl.vt == 64 ? launch_k<uint16_t, 64, 64>(p, pl, a.stream) : launch_k<uint16_t, 64, 128>(p, pl, a.stream);
  return pl.vt == 64 ? launch_k<float, 32, 64>(p, pl, a.stream) : launch_k<float, 32, 128>(p, pl, a.stream);
}

}  // namespace ss2d
