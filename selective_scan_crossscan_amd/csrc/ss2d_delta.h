// The gated delta rule over prompts: what its forward (ss2d_delta.hip) and its
// gradients (ss2d_delta_backward.hip) share.
//
//   h_t = a_t h_{t-1} + b_t k_t (v_t - a_t h_{t-1}' k_t)',   o_t = scale h_t' q_t,
// a = exp(g), b = beta.  In chunks of C tokens, with G the sum of g inside the chunk up
// to a token, H the state before the chunk, L_ij = exp(G_i - G_j) k_i . k_j for j < i
// and P_ij = scale exp(G_i - G_j) q_i . k_j for j <= i (both 0 otherwise):
//   E = (1 + L diag(b))^-1 (V - exp(G) K H)     the tokens' errors v - a h' k
//   U = b E,   o = scale exp(G) Q H + P U,   H <- exp(G_last) H + K' (w U),
// w_j = exp(G_last - G_j): with U known, linear attention whose values are U.  What does
// not depend on the state, the inverse and P, is formed for all chunks at once before
// (delta_systems); the walk over the chunks is left with products only.
//
// Fragments, parts and tiles are ss2d_attention.h's.  The state is kept as result tiles
// with rows k and columns v, E and U with rows token and columns v: each then lies in
// registers as the next product's operand (K H sums over k, the inverse and K' U over
// tokens), so a wave that owns value columns needs nothing from other waves.
#pragma once

#include "ss2d_attention.h"

namespace ss2d {

// Sizes of a chunk's systems: fragments in the order of their tiles, those of a triangle's
// 16-row tiles x by pairs of 16-column tiles; in memory in fp32, in the walks' LDS in parts.
template <typename E, int C>
struct Systems {
  static constexpr int NI = C / 16;
  static constexpr int kFrags = NI / 2 * (NI / 2 + 1);
  static constexpr int kParts = sizeof(E) == 2 ? 3 : 1;  // into which the walks split them
  static constexpr int kFragBytes = 64 * 8 * (int)sizeof(E);  // of one part
  static constexpr int kOne = kFrags * 64 * 8 * 4;  // an inverse without its diagonal of ones, or scores
  static constexpr int kForward = 2 * kOne;
  static constexpr int kBackward = 3 * kOne;
  // Rows i, columns j <= i: tile row x has the pairs 0 .. x / 2.
  static __host__ __device__ constexpr int lower(int x, int pair) { return (x / 2) * (x / 2 + 1) + (x & 1) * (x / 2 + 1) + pair; }
  // Rows j, columns i >= j: tile row x has the pairs x / 2 .. NI / 2 - 1; the mirror image.
  static __host__ __device__ constexpr int upper(int x, int pair) { return lower(NI - 1 - x, NI / 2 - 1 - pair); }
};

struct DeltaArgs {
  AttentionArgs f;  // as linear attention's
  const float* beta;
  int64_t beta_stride[3];
};

struct DeltaPlan {
  AttentionPlan a;      // kp, chunk, segments, slots, chunks; vt the walk's
  bool backward;
  bool cut;             // segments' states are kept for sequences of several segments alone
  int64_t parts;        // segments whose states are kept, an upper bound
};
DeltaPlan plan_delta(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim, bool packed,
                     int dtype, bool backward);
size_t delta_workspace_bytes(const DeltaPlan& pl, int64_t heads, int64_t key_dim, int64_t value_dim, int dtype);
hipError_t launch_delta(const DeltaArgs& a, const DeltaPlan& pl);

struct DeltaBackwardArgs {
  DeltaArgs d;  // the forward's inputs; workspace, stream
  const void* d_o;
  int64_t do_stride[3];
  const float* dstate_out;  // or null
  void *dq, *dk, *dv;
  float *dlog_decay, *dbeta;
  float* dstate_in;  // or null
};
size_t delta_backward_workspace_bytes(const DeltaPlan& pl, int64_t tokens, int64_t groups, int64_t heads,
                                      int64_t key_dim, int64_t value_dim, int dtype);
hipError_t launch_delta_backward(const DeltaBackwardArgs& a, const DeltaPlan& pl);

// Workgroups of the largest grid a plan launches.
int64_t delta_blocks(const DeltaPlan& pl, int64_t sequences, int64_t heads, int64_t value_dim);

struct DeltaStepArgs {
  StepArgs s;
  const float* beta;
};
hipError_t launch_delta_step(const DeltaStepArgs& a);

// ------------------------------------------------------------------ passes
struct DeltaParams {
  const void *q, *k, *v;
  const float *g, *beta;
  const float* state_in;    // or null
  void* o;
  float* state_out;         // or null
  char* systems;            // (chunk, head): inverse, scores; backward: inverse, transposed inverse and scores
  float* seg_state;         // (part, head, K, V): what a segment adds, after the carry the state before it
  float* seg_map;           // (part, head, KP, KP): the segment's map of the state before it
  float* chunk_state;       // (chunk, head, tile, KP, 64): the state before every chunk, 0 outside K and V
  float* errors;            // (chunk, head, tile, C, 64): E, 0 behind the chunk's tokens and outside V
  SequenceMap map;          // segments
  SequenceMap chunk_map;    // segments of one chunk
  int64_t q_stride[3], k_stride[3], v_stride[3], g_stride[3], b_stride[3];
  int tiles;                // of 64 value columns in the chunks' arrays
  int groups, heads, K, V, vtiles, ktiles;  // tiles of the pass's columns of values; of the segment maps' columns
  uint32_t blocks;          // workgroups; of a walk: units of a segment and head, each with its tiles
  float scale;
  bool split;               // segments start from seg_state
  bool cut;                 // parts are the slots of sequences of several segments alone; else of all
  bool last_maps;           // segment maps of the sequences' last segments too, for the way back
  int64_t system_stride;    // bytes of a chunk's and head's systems
};
DeltaParams delta_params(const DeltaArgs& a, const DeltaPlan& pl);
// The systems of all chunks.
hipError_t launch_delta_systems(const DeltaParams& p, const DeltaPlan& pl, int dtype, hipStream_t st);
// seg_state and seg_map of all segments but their sequence's last, then seg_state as the states before all of them.
hipError_t launch_delta_segments(DeltaParams p, const DeltaPlan& pl, int dtype, hipStream_t st);
// chunk_state and errors.
hipError_t launch_delta_states(DeltaParams p, const DeltaPlan& pl, int dtype, hipStream_t st);
// seg: what segments add to the state (backwards: to its gradient) becomes the states before (the gradients behind) them.
struct CarryParams {
  float* seg;            // (part, head, K, V)
  const float* seg_map;  // (part, head, KP, KP)
  const float* from;     // (sequence, head, K, V) or null
  SequenceMap map;
  bool cut;
  int heads, K, V, vtiles;
  uint32_t blocks;
};
// back: the same of the states' gradients, or null.
hipError_t launch_delta_carry(CarryParams p, const CarryParams* back, const DeltaPlan& pl, hipStream_t st);
// Bytes of one chunk's and head's systems.
int64_t system_bytes(const DeltaPlan& pl, int dtype);

namespace tok {

// A segment's part.
__device__ __forceinline__ int64_t part_number(const SequenceMap& m, bool cut, const Segment& g) {
  const uint32_t seg_len = (uint32_t)m.seg_len, seg = (uint32_t)g.begin / seg_len;
  if (!m.cu) return (int64_t)g.s * m.nseg + seg;
  return (int64_t)((cut ? 2 : 1) * (uint32_t)g.start / seg_len) + (cut ? 0 : g.s) + seg;
}

// c[x] += a[x] b for x in from .. to - 1, both operands in parts: those whose share of the product lies under the last
// part's (p + q >= N) are left out, the smallest come first, and products of different x stand next to each other.
template <int FROM, int TO, int N, int M, typename E>
__device__ __forceinline__ void mma_parts(const Frag<E> (&a)[M][N], const Frag<E> (&b)[N], f32x4 (&c)[M]) {
#pragma unroll
  for (int s = N - 1; s >= 0; --s)
#pragma unroll
    for (int p = 0; p <= s; ++p)
#pragma unroll
      for (int x = FROM; x < TO; ++x) c[x] = mma(a[x][p], b[s - p], c[x]);
}

// What a chunk's cumulative decays G give for each of its tokens.
template <int C>
struct Rates {
  __attribute__((aligned(16))) float since[C], left[C], beta[C];  // exp(G), exp(G_last - G)
  __device__ __forceinline__ static f32x4 four(const float* x) { return *reinterpret_cast<const f32x4*>(x); }
};
// One wave: lane t holds token t's log decay and beta (0 behind the end).
template <int C>
__device__ __forceinline__ void scan_rates(float g, float beta, Rates<C>& m) {
  const int lane = threadIdx.x & 63;
  const double s = wave_scan((double)clamp_log_decay(g) * 1.4426950408889634074);
  const double last = __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(s), C - 1),
                                       __builtin_amdgcn_readlane(__double2loint(s), C - 1));
  if (lane < C) {
    m.since[lane] = __builtin_amdgcn_exp2f((float)s);
    m.left[lane] = __builtin_amdgcn_exp2f((float)(last - s));
    m.beta[lane] = beta;
  }
}

// Workgroups go round the eight XCDs, each with an L2 of its own: a unit's tiles are eight workgroups apart, on one XCD at
// about the same time, so that what they share is read from memory once.  False behind the last unit.
constexpr uint32_t kXcds = 8;
__host__ __device__ constexpr int64_t spread_blocks(int64_t units, int tiles) { return (units + kXcds - 1) / kXcds * kXcds * tiles; }
__device__ __forceinline__ bool spread(uint32_t block, uint32_t units, uint32_t tiles, uint32_t& unit, uint32_t& tile) {
  const uint32_t round = block / (kXcds * tiles), rest = block - round * (kXcds * tiles);
  tile = rest / kXcds;
  unit = round * kXcds + rest % kXcds;
  return unit < units;
}

// Part q of fragment `at` of a chunk's systems.
template <typename E>
__device__ __forceinline__ Frag<E> system_frag(const char* sys, int at, int q) {
  Frag<E> f;
  __builtin_memcpy(&f, __builtin_assume_aligned(sys + (at * Systems<E, 32>::kParts + q) * Systems<E, 32>::kFragBytes +
                                                    (threadIdx.x & 63) * (8 * sizeof(E)), 16), sizeof(f));
  return f;
}
// A chunk's systems on their way from memory, BYTES by THREADS threads; stored as fragments in parts.  Split here, fp32 takes
// two thirds of the parts' bytes in memory (16 x 2048 tokens of 16 heads of 128: 393 us, with parts in memory 412).  Every
// thread has whole pieces, and no condition that only some threads meet stands around them, on purpose: the compiler has
// stored spilled registers before it let all threads go on behind one, and read them back for all.
template <typename E, int BYTES, int THREADS>
struct SystemLoad {
  static constexpr int kPieces = BYTES / 16 / THREADS;
  static_assert(kPieces * 16 * THREADS == BYTES, "a thread's pieces are whole");
  f32x4 x[kPieces];
  __device__ __forceinline__ void load(const char* from) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) x[i] = *reinterpret_cast<const f32x4*>(from + (threadIdx.x + i * THREADS) * 16);
  }
  __device__ __forceinline__ void store(char* sys) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = threadIdx.x + i * THREADS;  // half of a lane's eight values
      if constexpr (sizeof(E) == 4) {
        *reinterpret_cast<f32x4*>(sys + piece * 16) = x[i];
      } else {
        f32x4 rest = x[i];
#pragma unroll
        for (int q = 0; q < Systems<E, 32>::kParts; ++q) {
          const uint32_t w[2] = {pack_bf16(rest[0], rest[1]), pack_bf16(rest[2], rest[3])};
          __builtin_memcpy(__builtin_assume_aligned(sys + ((piece / 128 * Systems<E, 32>::kParts + q) * 128 + piece % 128) * 8, 8), w, 8);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            rest[2 * r] -= __uint_as_float(w[r] << 16);
            rest[2 * r + 1] -= __uint_as_float(w[r] & 0xffff0000u);
          }
        }
      }
    }
  }
};

// Four consecutive elements of a row of which the first n are there (the others are 0).
__device__ __forceinline__ f32x4 load4(const float* p, int n) {
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if (n >= 4) {
    const Bytes16 w = *reinterpret_cast<const Bytes16*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) x[i] = p[i];
  }
  return x;
}
__device__ __forceinline__ f32x4 load4(const uint16_t* p, int n) {
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if (n >= 4) {
    const Bytes8 w = *reinterpret_cast<const Bytes8*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] = bf16_bits_to_f32(w.w[i] & 0xffffu);
      x[2 * i + 1] = __uint_as_float(w.w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) x[i] = load1(p + i);
  }
  return x;
}

// p, uniform, moved by a lane's own bytes: one register of an address, and what is added by constants goes into the
// instruction (a sum of 32-bit indexes does not, and takes two registers for each).
template <typename T>
__device__ __forceinline__ T* by_bytes(T* p, uint32_t bytes) {
  return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + bytes);
}

// Two result tiles stacked along their rows as the eight inner values of an operand.
__device__ __forceinline__ void stack(const f32x4& a, const f32x4& b, float (&u)[8]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    u[r] = a[r];
    u[4 + r] = b[r];
  }
}

}  // namespace tok
}  // namespace ss2d
