// Norms of queries and keys for each head, and the rotation by the token's position in the same pass; the gradients.
//
//   xhat = x rstd,  rstd = 1 / sqrt(mean(x^2) + eps),  y = R xhat weight,
// R turning the pairs of the first `rotated` channels by the position's angles (its transpose turns them back):
//   dxhat = weight R' dy,  dx = rstd (dxhat - xhat mean(dxhat xhat)),  dweight = sum over rows of (R' dy) xhat.
//
// Bound by memory: every value is read once and written once.  A row (one token's head) is held in registers by up to
// 64 threads between the sum over it and the output.  A thread has eight channels as two quads a, b: of rotating
// channels the two quads whose values are pairs, wherever the pairs' halves lie, so a pair never crosses threads.
// Table rows and weights are shared by all heads of a token, or all rows, and come from the caches.  16384 tokens of 16 + 16
// heads of 128 in bf16: 51 us, 5.3 TB/s; gradients 80, 5.0 TB/s, and 4.5 for the sums of the weights' parts.
#include <type_traits>

#include "ss2d_delta.h"
#include "ss2d_qk_norm.h"

namespace ss2d {
namespace {

using namespace tok;

struct QkParams {
  QkSide side[2];  // queries, keys
  const float* table;
  const int32_t* positions;
  float* partial;  // gradients: (workgroup, dim)
  uint32_t tokens, length, table_rows;  // all tokens; of a sequence
  int heads[2];
  int runs[2];     // runs of heads of a token
  int dim, rotated, pair_pieces, interleaved;
  int blocks[2];   // gradients: workgroups of each side
  float eps, share;  // share: 1 / dim
};

// A thread's channels: quads at a and b, of which na and nb exist; pairs: they rotate.
struct Piece {
  int a, b, na, nb, pair;
  bool turns, zip;
};
__device__ __forceinline__ Piece piece_of(const QkParams& p, int t) {
  Piece x;
  x.turns = t < p.pair_pieces;
  x.zip = x.turns && p.interleaved;
  x.pair = 4 * t;
  if (x.turns && !p.interleaved) {
    x.a = 4 * t;
    x.b = p.rotated / 2 + 4 * t;
    x.na = x.nb = min(4, p.rotated / 2 - 4 * t);
  } else {
    const int end = x.turns ? p.rotated : p.dim;
    x.a = x.turns ? 8 * t : p.rotated + 8 * (t - p.pair_pieces);
    x.b = x.a + 4;
    x.na = max(0, min(4, end - x.a));
    x.nb = max(0, min(4, end - x.b));
  }
  return x;
}
// WHOLE: every thread has eight channels, and the ends are not asked for.
template <bool WHOLE, typename S>
__device__ __forceinline__ void load_piece(const S* row, const Piece& x, f32x4& a, f32x4& b) {
  a = load4(row + x.a, WHOLE ? 4 : x.na);
  b = load4(row + x.b, WHOLE ? 4 : x.nb);
  if (x.zip) {
    const f32x4 u = {a[0], a[2], b[0], b[2]}, v = {a[1], a[3], b[1], b[3]};
    a = u;
    b = v;
  }
}
template <bool WHOLE, typename S>
__device__ __forceinline__ void store_piece(S* row, const Piece& x, f32x4 a, f32x4 b) {
  if (x.zip) {
    const f32x4 u = {a[0], b[0], a[1], b[1]}, v = {a[2], b[2], a[3], b[3]};
    a = u;
    b = v;
  }
  if (WHOLE || x.na > 0) store4(row + x.a, WHOLE ? 4 : x.na, a);
  if (WHOLE || x.nb > 0) store4(row + x.b, WHOLE ? 4 : x.nb, b);
}
// Sum over the THREADS threads that share a row: within 16 lanes by permutations that cost no LDS access.
template <int THREADS>
__device__ __forceinline__ float row_sum(float v) {
  constexpr int kPairs = 0xb1, kHalves = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;  // of a quad, of eight, of a row
  v += dpp<kPairs>(v);
  v += dpp<kHalves>(v);
  if (THREADS >= 8) v += dpp<kHalfMirror>(v);
  if (THREADS >= 16) v += dpp<kMirror>(v);
  if (THREADS >= 32) v += __shfl_xor(v, 16);
  if (THREADS >= 64) v += __shfl_xor(v, 32);
  return v;
}
// A token's place: its sequence and its number there.
struct Place {
  uint32_t token, sequence, at;
  __device__ __forceinline__ Place(const QkParams& p, uint32_t t) : token(t), sequence(0), at(t) {
    if (p.length < p.tokens) {
      sequence = t / p.length;
      at = t - sequence * p.length;
    }
  }
  __device__ __forceinline__ int64_t offset(const int64_t (&stride)[3]) const {
    return sequence * stride[0] + at * stride[1];
  }
};
// Cosines and sines of a token's pairs.
template <bool WHOLE>
__device__ __forceinline__ void angles(const QkParams& p, const Piece& x, const Place& at, f32x4& c, f32x4& s) {
  int64_t row = p.positions ? (int64_t)p.positions[at.token] : (int64_t)at.at;
  row = row < 0 ? 0 : row >= p.table_rows ? p.table_rows - 1 : row;
  const float* from = p.table + row * p.rotated + x.pair;
  const int n = WHOLE ? 4 : min(4, p.rotated / 2 - x.pair);
  c = load4(from, n);
  s = load4(from + p.rotated / 2, n);
}

// THREADS threads take a run of RUN heads of one token, all loads before the first sum.
template <typename S, int THREADS, int RUN, bool WHOLE>
__global__ __launch_bounds__(256) void qk_norm_kernel(QkParams p) {
  const uint32_t item = (uint32_t)block_id() * (256 / THREADS) + threadIdx.x / THREADS;
  const uint32_t runs = p.runs[0] + p.runs[1], token = item / runs;
  if (token >= p.tokens) return;  // whole groups of threads; no barrier follows
  uint32_t run = item - token * runs;
  const int side = run >= (uint32_t)p.runs[0];
  if (side) run -= p.runs[0];
  const QkSide& z = p.side[side];
  const int head = run * RUN, last = p.heads[side] - 1;
  const Place at(p, token);
  const Piece x = piece_of(p, threadIdx.x % THREADS);
  f32x4 a[RUN], b[RUN], c, s, wa, wb;
  const S* from = static_cast<const S*>(z.x) + at.offset(z.x_stride);
#pragma unroll
  for (int i = 0; i < RUN; ++i) load_piece<WHOLE>(from + min(head + i, last) * z.x_stride[2], x, a[i], b[i]);
  if (x.turns) angles<WHOLE>(p, x, at, c, s);
  if (z.weight) load_piece<WHOLE>(z.weight, x, wa, wb);
  S* to = static_cast<S*>(z.y) + at.offset(z.y_stride);
#pragma unroll
  for (int i = 0; i < RUN; ++i) {
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) sq = fmaf(a[i][j], a[i][j], fmaf(b[i][j], b[i][j], sq));
    const float rstd = rsqrtf(row_sum<THREADS>(sq) * p.share + p.eps);
    f32x4 u = a[i] * rstd, v = b[i] * rstd;
    if (z.weight) {
      u *= wa;
      v *= wb;
    }
    if (x.turns) {
      const f32x4 w = u * c - v * s;
      v = u * s + v * c;
      u = w;
    }
    if (head + i <= last) store_piece<WHOLE>(to + (head + i) * z.y_stride[2], x, u, v);
  }
}

// Workgroups 0 .. blocks[0] - 1 take the queries' runs of heads, the others the keys'; each leaves one part of the
// weight's gradient.
template <typename S, int THREADS, int RUN, bool WHOLE>
__global__ __launch_bounds__(256) void qk_norm_backward_kernel(QkParams p) {
  constexpr int ITEMS = 256 / THREADS;
  __shared__ f32x4 parts[2][4][THREADS];
  const int side = (int)blockIdx.x >= p.blocks[0], block = (int)blockIdx.x - (side ? p.blocks[0] : 0);
  const QkSide& z = p.side[side];
  const int heads = p.heads[side];
  const uint32_t runs = p.runs[side], step = p.blocks[side] * ITEMS, items = p.tokens * runs;
  const Piece x = piece_of(p, threadIdx.x % THREADS);
  f32x4 wa = {1.f, 1.f, 1.f, 1.f}, wb = wa, da = {0.f, 0.f, 0.f, 0.f}, db = da;
  if (z.weight) load_piece<WHOLE>(z.weight, x, wa, wb);
  for (uint32_t item = block * ITEMS + threadIdx.x / THREADS; item < items; item += step) {
    const uint32_t token = item / runs;
    const int head = (item - token * runs) * RUN;
    const Place at(p, token);
    const S* from = static_cast<const S*>(z.x) + at.offset(z.x_stride);
    const S* dfrom = static_cast<const S*>(z.dy) + at.offset(z.y_stride);
    f32x4 a[RUN], b[RUN], ga[RUN], gb[RUN], c, s;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      const int h = min(head + i, heads - 1);
      load_piece<WHOLE>(from + h * z.x_stride[2], x, a[i], b[i]);
      load_piece<WHOLE>(dfrom + h * z.y_stride[2], x, ga[i], gb[i]);
    }
    if (x.turns) angles<WHOLE>(p, x, at, c, s);
    S* to = static_cast<S*>(z.y) + ((int64_t)token * heads + head) * p.dim;
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      if (x.turns) {
        const f32x4 u = ga[i] * c + gb[i] * s;
        gb[i] = gb[i] * c - ga[i] * s;
        ga[i] = u;
      }
      const f32x4 ha = ga[i] * wa, hb = gb[i] * wb;
      float sq = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sq = fmaf(a[i][j], a[i][j], fmaf(b[i][j], b[i][j], sq));
        dot = fmaf(a[i][j], ha[j], fmaf(b[i][j], hb[j], dot));
      }
      sq = row_sum<THREADS>(sq);
      dot = row_sum<THREADS>(dot);
      const float rstd = rsqrtf(sq * p.share + p.eps);
      const float mean = dot * rstd * p.share;
      a[i] *= rstd;
      b[i] *= rstd;
      if (head + i < heads) {
        da += ga[i] * a[i];
        db += gb[i] * b[i];
        store_piece<WHOLE>(to + i * p.dim, x, rstd * (ha - a[i] * mean), rstd * (hb - b[i] * mean));
      }
    }
  }
  if (z.dweight) {
#pragma unroll
    for (int m = THREADS; m < 64; m <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        da[i] += __shfl_xor(da[i], m);
        db[i] += __shfl_xor(db[i], m);
      }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane < THREADS) {
      parts[0][wave][lane] = da;
      parts[1][wave][lane] = db;
    }
    __syncthreads();
    if (threadIdx.x < THREADS) {
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        da += parts[0][w][lane];
        db += parts[1][w][lane];
      }
      store_piece<WHOLE>(p.partial + (int64_t)blockIdx.x * p.dim, x, da, db);
    }
  }
}

// dweight[c] = sum over a side's workgroups' parts: 32 channels by 32 ranges of parts per workgroup, eight loads in
// flight per thread, the ranges' sums added in order.  blockIdx.y: the side.
constexpr int kSumCols = 32, kSumRanges = 32;
__global__ __launch_bounds__(kSumCols * kSumRanges) void qk_sum_partials(QkParams p) {
  __shared__ float sums[kSumRanges][kSumCols + 1];
  const int side = blockIdx.y, col = threadIdx.x % kSumCols, range = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + col, parts = p.blocks[side];
  if (!p.side[side].dweight) return;
  const float* from = p.partial + (side ? (int64_t)p.blocks[0] * p.dim : 0);
  float s = 0.f;
  if (c < p.dim)
    for (int i = range; i < parts; i += 8 * kSumRanges) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = i + j * kSumRanges < parts ? from[(int64_t)(i + j * kSumRanges) * p.dim + c] : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
  sums[range][col] = s;
  __syncthreads();
  if (range == 0 && c < p.dim) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumRanges; ++i) s += sums[i][col];
    p.side[side].dweight[c] = s;
  }
}

QkParams params_of(const QkArgs& a, int run) {
  QkParams p{};
  for (int i = 0; i < 2; ++i) p.side[i] = a.side[i];
  p.table = a.table;
  p.positions = a.positions;
  p.partial = a.partial;
  p.tokens = (uint32_t)(a.sequences * a.length);
  p.length = (uint32_t)a.length;
  p.table_rows = (uint32_t)a.table_rows;
  for (int i = 0; i < 2; ++i) {
    p.heads[i] = (int)a.heads[i];
    p.runs[i] = (int)((a.heads[i] + run - 1) / run);
  }
  p.dim = (int)a.dim;
  p.rotated = a.table ? (int)a.rotated : 0;
  p.pair_pieces = (p.rotated + 7) / 8;
  p.interleaved = a.interleaved;
  p.eps = a.eps;
  p.share = 1.0f / (float)a.dim;
  return p;
}
// Threads per row: a power of two of at least its pieces of eight channels.
int threads_of(int64_t dim, int64_t rotated) {
  const int pieces = (int)((rotated + 7) / 8 + (dim - rotated + 7) / 8);
  int t = 4;
  while (t < pieces) t *= 2;
  return t;
}
// Heads in a run, and the gradients' workgroups of both sides at most: 16384 tokens of 16 + 16 heads of 128 in bf16, us of
// runs of 1, 2 and 4 heads 65, 52, 48; gradients of runs of 1, 2 and 4 by 1024 to 4096 workgroups 89 to 103, 88 to 98 and
// 89 (the fewer the better).  A run shares its token's angles and has more loads in flight; where rows are few, runs of 1
// are no faster (64 and 512 tokens: 6.4 and 5.2 us, in runs of 4 7.6 and 4.7).
constexpr int kRun = 4, kBackRun = 2;
constexpr int64_t kMost = 1024;
void share(int64_t tokens, const int64_t (&heads)[2], int threads, int run, int (&blocks)[2]) {
  int64_t items[2];
  for (int i = 0; i < 2; ++i) items[i] = tokens * ((heads[i] + run - 1) / run);
  for (int i = 0; i < 2; ++i) {
    const int64_t all = (items[i] + 256 / threads - 1) / (256 / threads);
    const int64_t most = kMost * items[i] / (items[0] + items[1]);
    blocks[i] = (int)(all < most ? all : most < 1 ? 1 : most);
  }
}

// Calls f with the threads per row and whether each has eight channels as constants.
template <typename F>
void with_threads(const QkParams& p, F f) {
  using std::integral_constant;
  const int t = threads_of(p.dim, p.rotated);
  auto of = [&](auto threads) {
    if (p.dim == 8 * t && p.rotated % 8 == 0)
      f(threads, integral_constant<bool, true>());
    else
      f(threads, integral_constant<bool, false>());
  };
  switch (t) {
    case 4: of(integral_constant<int, 4>()); break;
    case 8: of(integral_constant<int, 8>()); break;
    case 16: of(integral_constant<int, 16>()); break;
    case 32: of(integral_constant<int, 32>()); break;
    default: of(integral_constant<int, 64>());
  }
}

template <typename S>
void launch_forward(const QkArgs& a, hipStream_t st) {
  const QkParams p = params_of(a, kRun);
  const int t = threads_of(p.dim, p.rotated);
  const int64_t items = (int64_t)p.tokens * (p.runs[0] + p.runs[1]);
  const dim3 grid = grid_of((items + 256 / t - 1) / (256 / t), 256), block(256);
  with_threads(p, [&](auto threads, auto whole) { qk_norm_kernel<S, threads(), kRun, whole()><<<grid, block, 0, st>>>(p); });
}
template <typename S>
void launch_backward(const QkArgs& a, hipStream_t st) {
  QkParams p = params_of(a, kBackRun);
  const int t = threads_of(p.dim, p.rotated);
  share(p.tokens, a.heads, t, kBackRun, p.blocks);
  const dim3 grid((unsigned)(p.blocks[0] + p.blocks[1])), block(256);
  with_threads(p, [&](auto threads, auto whole) {
    qk_norm_backward_kernel<S, threads(), kBackRun, whole()><<<grid, block, 0, st>>>(p);
  });
  if (p.side[0].dweight || p.side[1].dweight)
    qk_sum_partials<<<dim3((unsigned)((p.dim + kSumCols - 1) / kSumCols), 2), dim3(kSumCols * kSumRanges), 0, st>>>(p);
}

}  // namespace

size_t qk_norm_backward_workspace_bytes(int64_t tokens, const int64_t (&heads)[2], int64_t dim, int64_t rotated) {
  int blocks[2];
  share(tokens, heads, threads_of(dim, rotated), kBackRun, blocks);
  return (size_t)(blocks[0] + blocks[1]) * (size_t)dim * 4;
}

hipError_t launch_qk_norm(const QkArgs& a) {
  a.dtype == 1 ? launch_forward<uint16_t>(a, a.stream) : launch_forward<float>(a, a.stream);
  return hipGetLastError();
}

hipError_t launch_qk_norm_backward(const QkArgs& a) {
  a.dtype == 1 ? launch_backward<uint16_t>(a, a.stream) : launch_backward<float>(a, a.stream);
  return hipGetLastError();
}

}  // namespace ss2d
