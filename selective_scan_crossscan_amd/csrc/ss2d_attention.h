// Linear attention with a decay per head over prompts: what the forward
// (ss2d_attention.hip) and the backward (ss2d_attention_backward.hip) share.
//
// Matrix fragments.  Every product runs on 16x16 tiles of the matrix cores with
// 32 steps of the inner index at a time.  A fragment is a lane's eight inner
// indices of one row (first operand) or column (second operand): row or column
// lane % 16, and with g = lane / 16 either the "plain" order 8g .. 8g+7 or the
// "split" order 4g .. 4g+3, 16+4g .. 16+4g+3; both operands of a product use the
// same one.  The split order is the one in which two result tiles, stacked along
// their rows, already lie in registers (a lane holds rows 4g .. 4g+3 of column
// lane % 16), so a result whose rows are summed over next needs no trip through
// LDS: the state is kept that way.  bf16 runs on v_mfma_f32_16x16x32_bf16; fp32
// on eight v_mfma_f32_16x16x4_f32, one per inner index of the fragment.
//
// Parts.  An fp32 value that enters a bf16 product as a state or a decayed
// operand is split into bf16 parts that add up to it, each the rounding of what
// the parts before left: three give all 24 bits.  What becomes an fp32 result
// (states, gradients of the decay) takes three.  What only ends in a bf16 output
// takes one, as the masked scores do: its rounding, 2^-8 of its share of the output
// at most, is that of the output itself.  The fp32 product takes the value itself.
#pragma once

#include "ss2d_token_ops.h"

namespace ss2d {

// Sequences and their segments.  A segment is seg_len tokens of one sequence
// (the last may be shorter); slot numbers are dense for equal lengths, and for
// packed sequences slot(s) = cu[s] / seg_len + s is the first of sequence s:
// ceil(len / seg_len) slots always fit before slot(s + 1), so no prefix sum over
// the lengths is needed.
struct SequenceMap {
  const int32_t* cu;  // or null: equal lengths
  int64_t tokens, seg_len;
  int sequences, nseg;  // nseg: segments per sequence of equal lengths
  int64_t len;          // equal length
};

struct AttentionArgs {
  const void *q, *k, *v;
  const float* log_decay;
  const float* state_in;  // or null
  const int32_t* cu;      // or null
  void* o;
  float* state_out;       // or null
  int64_t sequences, tokens, groups, heads, key_dim, value_dim;
  int64_t q_stride[3], k_stride[3], v_stride[3], g_stride[3];
  float scale;
  int dtype;
  void* workspace;
  hipStream_t stream;
};

struct AttentionPlan {
  int kp;           // key_dim rounded up to 32, 64, 128 or 256
  int vt;           // value columns per workgroup
  int vtiles;
  int chunk;        // tokens per chunk
  int64_t seg_len;  // tokens per segment, whole chunks
  int64_t slots;    // segments, an upper bound for packed sequences
  int64_t chunks;   // chunks, an upper bound for packed sequences
  int nseg;         // per sequence of equal lengths
  bool split;       // some sequence may have more than one segment
  bool tiny;        // rows of keys or values under 16 bytes: kp 256, vt 64, loaded value by value
};
AttentionPlan plan_attention(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim,
                             bool packed, int dtype);
size_t attention_workspace_bytes(const AttentionPlan& pl, int64_t heads, int64_t key_dim, int64_t value_dim);
hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& pl);
SequenceMap sequence_map(const AttentionArgs& a, const AttentionPlan& pl);

struct AttentionBackwardArgs {
  AttentionArgs f;  // the forward's inputs; workspace, stream
  const void* d_o;
  int64_t do_stride[3];
  const float* dstate_out;  // or null
  void *dq, *dk, *dv;
  float* dlog_decay;
  float* dstate_in;  // or null
};
AttentionPlan plan_attention_backward(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim,
                                      int64_t value_dim, bool packed, int dtype);
size_t attention_backward_workspace_bytes(const AttentionPlan& pl, int64_t tokens, int64_t groups, int64_t heads,
                                          int64_t key_dim, int64_t value_dim);
hipError_t launch_attention_backward(const AttentionBackwardArgs& a, const AttentionPlan& pl);

// The state's passes over keys and values alone (ss2d_attention_state.hip), in tiles
// of 64 value columns whatever the plan's.
enum StatePass {
  kSegmentStates,    // what each segment (but a sequence's last) adds to the state, from 0, and its whole decay
  kChunkStates,      // the state before every chunk
  kSegmentGradients  // what each segment (but the first) adds to the state's gradient, from 0, walking backwards
};
struct StateParams {
  const void *k, *v;      // gradients: q and d_o
  const float* g;
  const float* state_in;  // the sequences' initial states (gradients: of their final states), or null
  float* seg_state;       // (slot, head, K, V)
  float* seg_decay;       // (slot, head)
  float* chunk_state;     // chunk states: (chunk, head, tile, KP x 64 as the kernel lays it out)
  SequenceMap map;
  int64_t k_stride[3], v_stride[3], g_stride[3];
  int groups, heads, K, V, tiles;  // tiles of 64 value columns
  uint32_t blocks, carry_blocks;   // workgroups of a pass over the segments, of a carry
  float scale;
  bool split;             // segments start from seg_state
};
// Sets blocks and carry_blocks from the other sizes.
void count_blocks(StateParams& p, const AttentionPlan& pl);
// seg_state: the state before every segment of a sequence of several.
hipError_t launch_segment_states(const StateParams& p, const AttentionPlan& pl, int dtype, hipStream_t st);
// The same, and r's seg_state: the gradient of the state behind every segment of a sequence of several.
hipError_t launch_segment_pair(const StateParams& p, const StateParams& r, const AttentionPlan& pl, int dtype,
                               hipStream_t st);
hipError_t launch_chunk_states(const StateParams& p, const AttentionPlan& pl, int dtype, hipStream_t st);

namespace tok {

// This wave's number, in a scalar register.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

// Where a segment lies: sequence s, its first token and length, and the
// segment's range [begin, end) inside the sequence.
struct Segment {
  int s;
  int64_t start, len, begin, end;
  bool last;  // the sequence's last segment
  __device__ __forceinline__ bool several() const { return begin > 0 || !last; }  // the sequence has other segments
};

__device__ __forceinline__ int64_t cu_at(const SequenceMap& m, int s) {
  const int64_t c = m.cu[s];
  return c < 0 ? 0 : c > m.tokens ? m.tokens : c;
}

// Number of the chunk of C tokens that holds token `at` of segment g's sequence,
// counted like the segments' slots.
template <int C>
__device__ __forceinline__ int64_t chunk_number(const SequenceMap& m, const Segment& g, int64_t at) {
  return (m.cu ? g.start / C + g.s : g.s * ((m.len + C - 1) / C)) + at / C;
}

// False where no segment has this slot.
__device__ __forceinline__ bool find_segment(const SequenceMap& m, int64_t slot, Segment& g) {
  int64_t seg;
  if (!m.cu) {
    g.s = (int)(slot / m.nseg);
    seg = slot % m.nseg;
    g.start = (int64_t)g.s * m.len;
    g.len = m.len;
  } else {
    // the last sequence whose first slot is at most `slot`, by counting (first slots ascend): the lanes look at 64
    // sequences, spread over those left, until they are next to each other; one load's latency for up to 64 sequences,
    // two for 4096, where a search by halves would take one per halving and a walk over all of them one per 64
    const uint32_t seg_len = (uint32_t)m.seg_len;
    int lo = 0;
    for (int left = m.sequences, step; left > 1; left = min(left, step)) {
      step = (left + 63) / 64;
      const int ahead = min((int)(threadIdx.x & 63) * step, left);
      const bool before = ahead < left && (int64_t)((uint32_t)cu_at(m, lo + min(ahead, left - 1)) / seg_len) + lo + ahead <= slot;
      const int count = (int)__popcll(__ballot(before));
      const int skip = count > 1 ? (count - 1) * step : 0;  // offsets that do not ascend may leave none
      lo += skip;
      left -= skip;
    }
    g.s = lo;
    g.start = cu_at(m, lo);
    const int64_t end = cu_at(m, lo + 1);
    g.len = end > g.start ? end - g.start : 0;
    seg = slot - (g.start / m.seg_len + lo);
    if (seg < 0) return false;
  }
  g.begin = seg * m.seg_len;
  if (g.begin > 0 && g.begin >= g.len) return false;
  g.end = g.begin + m.seg_len < g.len ? g.begin + m.seg_len : g.len;
  g.last = g.end == g.len;
  return true;
}

// ---------------------------------------------------------------- fragments
template <typename E>
struct Frag;
template <>
struct Frag<uint16_t> {
  bf16x8 v;
};
template <>
struct Frag<float> {
  float v[8];
};

// Parts an fp32 value is split into for fp32 results (see above).
template <typename E>
constexpr int kFullParts = sizeof(E) == 2 ? 3 : 1;

__device__ __forceinline__ f32x4 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

template <int N>
__device__ __forceinline__ void split_parts(const float (&x)[8], Frag<uint16_t> (&f)[N]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = x[i];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(rest[2 * i], rest[2 * i + 1]);
      rest[2 * i] -= __uint_as_float(w[i] << 16);
      rest[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
    }
    __builtin_memcpy(&f[n].v, w, 16);
  }
}
__device__ __forceinline__ void split_parts(const float (&x)[8], Frag<float> (&f)[1]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[0].v[i] = x[i];
}
__device__ __forceinline__ void frag_values(const Frag<uint16_t>& f, float (&x)[8]) {
  uint32_t w[4];
  __builtin_memcpy(w, &f.v, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void frag_values(const Frag<float>& f, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = f.v[i];
}

// ---------------------------------------------------------------- LDS tiles
// A ROWS x COLS tile, row major, with PAD bytes behind each row: 16 spread
// sixteen rows' reads of 8 or 16 bytes over the banks (frag_row, frag_row_split),
// 32 the transposing reads of four rows by four 8-byte pieces (frag_col_split).
template <typename E, int ROWS, int COLS, int PAD = 16>
struct Tile {
  static constexpr int stride = COLS + PAD / (int)sizeof(E);
  E e[ROWS * stride];
};

// Fragment of row `row` (inner index along the row from c0), plain order.
template <typename E, int R, int C, int PAD>
__device__ __forceinline__ Frag<E> frag_row(const Tile<E, R, C, PAD>& m, int row, int c0) {
  const int g = (threadIdx.x & 63) >> 4;
  Frag<E> f;
  __builtin_memcpy(&f, __builtin_assume_aligned(&m.e[row * m.stride + c0 + 8 * g], 16), sizeof(f));
  return f;
}
// The same in split order.
template <typename E, int R, int C, int PAD>
__device__ __forceinline__ Frag<E> frag_row_split(const Tile<E, R, C, PAD>& m, int row, int c0) {
  const int g = (threadIdx.x & 63) >> 4;
  Frag<E> f;
  const E* p = &m.e[row * m.stride + c0 + 4 * g];
  __builtin_memcpy(&f, __builtin_assume_aligned(p, 4 * sizeof(E)), 4 * sizeof(E));
  __builtin_memcpy(reinterpret_cast<char*>(&f) + 4 * sizeof(E), __builtin_assume_aligned(p + 16, 4 * sizeof(E)),
                   4 * sizeof(E));
  return f;
}
// Fragment of column c0 + lane % 16 (inner index down the rows from r0), split
// order.  bf16: the transposing LDS read, in which the sixteen lanes of a group
// each read four columns of one of four rows and get four rows of one column.
template <int R, int C, int PAD>
__device__ __forceinline__ Frag<uint16_t> frag_col_split(const Tile<uint16_t, R, C, PAD>& m, int r0, int c0) {
  typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
  const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const uint16_t* p = &m.e[(r0 + 4 * g + (l >> 2)) * m.stride + c0 + 4 * (l & 3)];
  const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)p);
  const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p + 16 * m.stride));
  Frag<uint16_t> f;
  f.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return f;
}
template <int R, int C, int PAD>
__device__ __forceinline__ Frag<float> frag_col_split(const Tile<float, R, C, PAD>& m, int r0, int c0) {
  const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  Frag<float> f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[i] = m.e[(r0 + 4 * g + i) * m.stride + c0 + l];
    f.v[4 + i] = m.e[(r0 + 16 + 4 * g + i) * m.stride + c0 + l];
  }
  return f;
}

// A tile on its way from global memory to LDS, in registers, by THREADS threads
// with 16 bytes a piece.  Every piece is loaded, with no branch around it, so all
// are in flight together: rows behind the last read the last one, pieces behind
// the row's end and the piece across it read the 16 bytes that end there, and
// store() puts zeros or the piece's own part in their place.  `first` columns of
// the row lie before the tile's (the 16 bytes may begin there); a row of fewer
// than 16 bytes in all takes TINY, which loads value by value.
template <typename E, int ROWS, int COLS, int PAD, int THREADS, bool TINY>
struct TileLoad {
  static constexpr int kPer = 16 / (int)sizeof(E);  // elements per piece
  static constexpr int kRowPieces = COLS / kPer;
  static constexpr int kPieces = (ROWS * kRowPieces + THREADS - 1) / THREADS;
  Bytes16 r[kPieces];

  // nrows >= 1 rows of `base`, stride elements apart, of ncols >= 1 columns.
  __device__ __forceinline__ void load(const E* base, int64_t stride, int nrows, int ncols) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int idx = threadIdx.x + i * THREADS;
      const int row = min(idx / kRowPieces, nrows - 1), c = (idx % kRowPieces) * kPer;
      // 24-bit factors: the strides are checked, a chunk's rows span less than 2^31 elements.  Signed sums: the 16
      // bytes of a narrow tile may begin before its first column
      const int at = (int)__umul24((uint32_t)row, (uint32_t)stride);
      if (TINY) {
        E e[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) e[j] = base[at + min(c + j, ncols - 1)];
        __builtin_memcpy(&r[i], e, 16);
      } else {
        r[i] = *reinterpret_cast<const Bytes16*>(base + (at + min(c, ncols - kPer)));
      }
    }
  }
  // The same nrows and ncols.
  __device__ __forceinline__ void store(Tile<E, ROWS, COLS, PAD>& m, int nrows, int ncols) const {
    if (!TINY && nrows == ROWS && ncols == COLS) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int idx = threadIdx.x + i * THREADS;
        if (ROWS * kRowPieces % THREADS == 0 || idx < ROWS * kRowPieces)
          __builtin_memcpy(__builtin_assume_aligned(&m.e[idx / kRowPieces * m.stride + (idx % kRowPieces) * kPer], 16),
                           &r[i], 16);
      }
      return;
    }
    const bool ragged = TINY || ncols % kPer != 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int idx = threadIdx.x + i * THREADS;
      const int row = idx / kRowPieces, c = (idx % kRowPieces) * kPer;
      if (ROWS * kRowPieces % THREADS != 0 && row >= ROWS) continue;
      E* to = &m.e[row * m.stride + c];
      const int n = row < nrows ? ncols - c : 0;  // elements of the piece that are there
      Bytes16 x = r[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) x.w[j] = n > 0 ? x.w[j] : 0;
      __builtin_memcpy(__builtin_assume_aligned(to, 16), &x, 16);
      if (ragged && n > 0 && n < kPer) {  // across the end: the loaded bytes end where the row does
        E e[kPer];
        __builtin_memcpy(e, &r[i], 16);
        const int shift = TINY ? 0 : kPer - n;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j >= shift && j - shift < n) to[j - shift] = e[j];
#pragma unroll
        for (int j = 1; j < kPer; ++j)
          if (j >= n) to[j] = (E)0;
      }
    }
  }
};

// ---------------------------------------------------------------- decays
// Cumulative log2 decays of a chunk, each an integer and a fraction: differences
// of the integers are exact and those of the fractions lose nothing to the
// sums' size, so a decay between two near tokens is good to fp32 however much
// the chunk decays as a whole.
template <int C>
struct Decays {
  __attribute__((aligned(16))) float whole[C], frac[C];
  __device__ __forceinline__ float between(int i, int j) const {  // exp(G_i - G_j)
    return __builtin_amdgcn_exp2f((whole[i] - whole[j]) + (frac[i] - frac[j]));
  }
  // exp(G_i - G_j) for j .. j + 3
  __device__ __forceinline__ f32x4 between4(int i, int j) const {
    const f32x4 w = *reinterpret_cast<const f32x4*>(&whole[j]), f = *reinterpret_cast<const f32x4*>(&frac[j]);
    const float wi = whole[i], fi = frac[i];
    f32x4 e;
#pragma unroll
    for (int r = 0; r < 4; ++r) e[r] = __builtin_amdgcn_exp2f((wi - w[r]) + (fi - f[r]));
    return e;
  }
  // exp(G_j) for j .. j + 3
  __device__ __forceinline__ f32x4 since4(int j) const {
    const f32x4 w = *reinterpret_cast<const f32x4*>(&whole[j]), f = *reinterpret_cast<const f32x4*>(&frac[j]);
    f32x4 e;
#pragma unroll
    for (int r = 0; r < 4; ++r) e[r] = __builtin_amdgcn_exp2f(w[r] + f[r]);
    return e;
  }
};

// One wave: lane t holds token t's log decay (0 behind the end).
template <int C>
__device__ __forceinline__ void scan_decays(float g, Decays<C>& d) {
  const int lane = threadIdx.x & 63;
  const double s = wave_scan((double)clamp_log_decay(g) * 1.4426950408889634074);
  if (lane < C) {
    const double w = rint(s);
    d.whole[lane] = (float)w;
    d.frac[lane] = (float)(s - w);
  }
}

// Four consecutive elements p[0..3], of which the first n are there.
__device__ __forceinline__ void store4(float* p, int n, f32x4 v) {
  if (n >= 4) {
    Bytes16 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.w[i] = __float_as_uint(v[i]);
    *reinterpret_cast<Bytes16*>(p) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, int n, f32x4 v) {
  Bytes8 b;
  b.w[0] = pack_bf16(v[0], v[1]);
  b.w[1] = pack_bf16(v[2], v[3]);
  if (n >= 4) {
    *reinterpret_cast<Bytes8*>(p) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (uint16_t)(i & 1 ? b.w[i / 2] >> 16 : b.w[i / 2]);
  }
}
// Transposed result tiles to memory: tile [t][x] holds, for token 16 x + l, the
// four columns from c0 + t * step on; `tokens` rows, stride elements apart (64 of
// them under 2^32), and `cols` columns exist.
template <int NI, int NV, typename O>
__device__ __forceinline__ void put_rows(O* base, int64_t stride, int tokens, int cols, int c0, int step, int l,
                                         const f32x4 (&x)[NV][NI]) {
  const uint32_t at = (uint32_t)l * (uint32_t)stride + (uint32_t)c0;
  if (tokens == NI * 16 && cols % 4 == 0) {  // whole tokens, whole pieces or none
#pragma unroll
    for (int t = 0; t < NV; ++t)
      if (c0 + t * step < cols)
#pragma unroll
        for (int i = 0; i < NI; ++i) store4(base + i * 16 * stride + (at + (uint32_t)(t * step)), 4, x[t][i]);
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (i * 16 + l < tokens)
#pragma unroll
        for (int t = 0; t < NV; ++t)
          store4(base + i * 16 * stride + (at + (uint32_t)(t * step)), cols - c0 - t * step, x[t][i]);
  }
}
// Four elements into an LDS row (aligned to four elements).
__device__ __forceinline__ void put4(uint16_t* p, f32x4 v) {
  const uint32_t w[2] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  __builtin_memcpy(__builtin_assume_aligned(p, 8), w, 8);
}
__device__ __forceinline__ void put4(float* p, f32x4 v) {
  __builtin_memcpy(__builtin_assume_aligned(p, 16), &v, 16);
}

}  // namespace tok
}  // namespace ss2d
