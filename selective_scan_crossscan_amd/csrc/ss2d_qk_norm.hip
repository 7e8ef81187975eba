// Norms of queries and keys for each head, and the rotation by the token's position in the same pass; the gradients.
//
//   xhat = x rstd,  rstd = 1 / sqrt(mean(x^2) + eps),  y = R xhat weight,
// R turning the pairs of the first `rotated` channels by the position's angles (its transpose turns them back):
//   dxhat = weight R' dy,  dx = rstd (dxhat - xhat mean(dxhat xhat)),  dweight = sum over rows of (R' dy) xhat.
//
// Bound by memory: every value is read once and written once.  A row (one token's head) is held in registers by up to
// 64 threads between the sum over it and the output.  A thread has eight channels as two quads a, b: of rotating
// channels the two quads whose values are pairs, wherever the pairs' halves lie, so a pair never crosses threads.
// Table rows and weights are shared by all heads of a token, or all rows, and come from the caches.
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
  int64_t tokens, length, table_rows;  // all tokens; of a sequence
  int heads[2];
  int dim, rotated, pair_pieces, interleaved;
  int blocks[2];   // gradients: workgroups of each side
  uint32_t rows;
  float eps;
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
template <typename S>
__device__ __forceinline__ void load_piece(const S* row, const Piece& x, f32x4& a, f32x4& b) {
  a = load4(row + x.a, x.na);
  b = load4(row + x.b, x.nb);
  if (x.zip) {
    const f32x4 u = {a[0], a[2], b[0], b[2]}, v = {a[1], a[3], b[1], b[3]};
    a = u;
    b = v;
  }
}
template <typename S>
__device__ __forceinline__ void store_piece(S* row, const Piece& x, f32x4 a, f32x4 b) {
  if (x.zip) {
    const f32x4 u = {a[0], b[0], a[1], b[1]}, v = {a[2], b[2], a[3], b[3]};
    a = u;
    b = v;
  }
  if (x.na > 0) store4(row + x.a, x.na, a);
  if (x.nb > 0) store4(row + x.b, x.nb, b);
}
template <int THREADS>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < THREADS; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
// Cosines and sines of a token's pairs.
__device__ __forceinline__ void angles(const QkParams& p, const Piece& x, int64_t token, f32x4& c, f32x4& s) {
  int64_t at = p.positions ? p.positions[token] : token % p.length;
  at = at < 0 ? 0 : at >= p.table_rows ? p.table_rows - 1 : at;
  const float* row = p.table + at * p.rotated + x.pair;
  const int n = min(4, p.rotated / 2 - x.pair);
  c = load4(row, n);
  s = load4(row + p.rotated / 2, n);
}
__device__ __forceinline__ int64_t offset(const int64_t (&stride)[3], const QkParams& p, int64_t token, int head) {
  const int64_t s = token / p.length;
  return s * stride[0] + (token - s * p.length) * stride[1] + head * stride[2];
}

template <typename S, int THREADS>
__global__ __launch_bounds__(256) void qk_norm_kernel(QkParams p) {
  const uint32_t row = (uint32_t)block_id() * (256 / THREADS) + threadIdx.x / THREADS;
  if (row >= p.rows) return;  // whole rows; no barrier follows
  const uint32_t heads = p.heads[0] + p.heads[1];
  const int64_t token = row / heads;
  const int side = row % heads >= (uint32_t)p.heads[0], head = row % heads - (side ? p.heads[0] : 0);
  const QkSide& z = p.side[side];
  const Piece x = piece_of(p, threadIdx.x % THREADS);
  f32x4 a, b, c, s, wa, wb;
  load_piece(static_cast<const S*>(z.x) + offset(z.x_stride, p, token, head), x, a, b);
  if (x.turns) angles(p, x, token, c, s);
  if (z.weight) load_piece(z.weight, x, wa, wb);
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) sq = fmaf(a[i], a[i], fmaf(b[i], b[i], sq));
  const float rstd = 1.0f / sqrtf(row_sum<THREADS>(sq) / (float)p.dim + p.eps);
  a *= rstd;
  b *= rstd;
  if (z.weight) {
    a *= wa;
    b *= wb;
  }
  if (x.turns) {
    const f32x4 u = a * c - b * s;
    b = a * s + b * c;
    a = u;
  }
  store_piece(static_cast<S*>(z.y) + offset(z.y_stride, p, token, head), x, a, b);
}

// One wave per workgroup; workgroups 0 .. blocks[0] - 1 take the queries' rows, the others the keys'.
template <typename S, int THREADS>
__global__ __launch_bounds__(64) void qk_norm_backward_kernel(QkParams p) {
  constexpr int ROWS = 64 / THREADS;
  const int side = (int)blockIdx.x >= p.blocks[0], block = (int)blockIdx.x - (side ? p.blocks[0] : 0);
  const QkSide& z = p.side[side];
  const int heads = p.heads[side];
  const int64_t rows = p.tokens * heads, step = (int64_t)p.blocks[side] * ROWS;
  const Piece x = piece_of(p, threadIdx.x % THREADS);
  f32x4 wa = {1.f, 1.f, 1.f, 1.f}, wb = wa, da = {0.f, 0.f, 0.f, 0.f}, db = da;
  if (z.weight) load_piece(z.weight, x, wa, wb);
  for (int64_t row = (int64_t)block * ROWS + threadIdx.x / THREADS; row < rows; row += step) {
    const int64_t token = row / heads;
    const int head = (int)(row - token * heads);
    f32x4 a, b, ga, gb;
    load_piece(static_cast<const S*>(z.x) + offset(z.x_stride, p, token, head), x, a, b);
    load_piece(static_cast<const S*>(z.dy) + offset(z.y_stride, p, token, head), x, ga, gb);
    if (x.turns) {
      f32x4 c, s;
      angles(p, x, token, c, s);
      const f32x4 u = ga * c + gb * s;
      gb = gb * c - ga * s;
      ga = u;
    }
    const f32x4 ha = ga * wa, hb = gb * wb;
    float sq = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sq = fmaf(a[i], a[i], fmaf(b[i], b[i], sq));
      dot = fmaf(a[i], ha[i], fmaf(b[i], hb[i], dot));
    }
    sq = row_sum<THREADS>(sq);
    dot = row_sum<THREADS>(dot);
    const float rstd = 1.0f / sqrtf(sq / (float)p.dim + p.eps);
    const float mean = dot * rstd / (float)p.dim;
    a *= rstd;
    b *= rstd;
    da += ga * a;
    db += gb * b;
    store_piece(static_cast<S*>(z.y) + row * p.dim, x, rstd * (ha - a * mean), rstd * (hb - b * mean));
  }
  if (z.dweight) {
#pragma unroll
    for (int m = THREADS; m < 64; m <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        da[i] += __shfl_xor(da[i], m);
        db[i] += __shfl_xor(db[i], m);
      }
    if (threadIdx.x < THREADS) store_piece(p.partial + (int64_t)blockIdx.x * p.dim, x, da, db);
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

QkParams params_of(const QkArgs& a) {
  QkParams p{};
  for (int i = 0; i < 2; ++i) p.side[i] = a.side[i];
  p.table = a.table;
  p.positions = a.positions;
  p.partial = a.partial;
  p.tokens = a.sequences * a.length;
  p.length = a.length;
  p.table_rows = a.table_rows;
  p.heads[0] = (int)a.heads[0];
  p.heads[1] = (int)a.heads[1];
  p.dim = (int)a.dim;
  p.rotated = a.table ? (int)a.rotated : 0;
  p.pair_pieces = (p.rotated + 7) / 8;
  p.interleaved = a.interleaved;
  p.rows = (uint32_t)(p.tokens * (a.heads[0] + a.heads[1]));
  p.eps = a.eps;
  return p;
}
// Threads per row: a power of two of at least its pieces of eight channels.
int threads_of(const QkParams& p) {
  const int pieces = p.pair_pieces + (p.dim - p.rotated + 7) / 8;
  int t = 4;
  while (t < pieces) t *= 2;
  return t;
}
// Workgroups of each side, as many of both as there are rows, at most kMost together.
constexpr int64_t kMost = 2048;
void share(int64_t tokens, int64_t hq, int64_t hk, int rows_each, int (&blocks)[2]) {
  const int64_t h[2] = {hq, hk};
  for (int i = 0; i < 2; ++i) {
    const int64_t all = (tokens * h[i] + rows_each - 1) / rows_each, most = kMost * h[i] / (hq + hk);
    blocks[i] = (int)(all < most ? all : most < 1 ? 1 : most);
  }
}

template <typename S>
void launch_forward(const QkParams& p, hipStream_t st) {
  const int t = threads_of(p);
  const dim3 grid = grid_of(((int64_t)p.rows + 256 / t - 1) / (256 / t), 256), block(256);
  switch (t) {
    case 4: qk_norm_kernel<S, 4><<<grid, block, 0, st>>>(p); break;
    case 8: qk_norm_kernel<S, 8><<<grid, block, 0, st>>>(p); break;
    case 16: qk_norm_kernel<S, 16><<<grid, block, 0, st>>>(p); break;
    case 32: qk_norm_kernel<S, 32><<<grid, block, 0, st>>>(p); break;
    default: qk_norm_kernel<S, 64><<<grid, block, 0, st>>>(p);
  }
}
template <typename S>
void launch_backward(const QkParams& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.blocks[0] + p.blocks[1])), block(64);
  switch (threads_of(p)) {
    case 4: qk_norm_backward_kernel<S, 4><<<grid, block, 0, st>>>(p); break;
    case 8: qk_norm_backward_kernel<S, 8><<<grid, block, 0, st>>>(p); break;
    case 16: qk_norm_backward_kernel<S, 16><<<grid, block, 0, st>>>(p); break;
    case 32: qk_norm_backward_kernel<S, 32><<<grid, block, 0, st>>>(p); break;
    default: qk_norm_backward_kernel<S, 64><<<grid, block, 0, st>>>(p);
  }
  if (p.side[0].dweight || p.side[1].dweight)
    qk_sum_partials<<<dim3((unsigned)((p.dim + kSumCols - 1) / kSumCols), 2), dim3(kSumCols * kSumRanges), 0, st>>>(p);
}

}  // namespace

size_t qk_norm_backward_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t dim) {
  int blocks[2];
  share(tokens, q_heads, k_heads, 1, blocks);  // as if each row had a wave: an upper bound
  return (size_t)(blocks[0] + blocks[1]) * (size_t)dim * 4;
}

hipError_t launch_qk_norm(const QkArgs& a) {
  const QkParams p = params_of(a);
  a.dtype == 1 ? launch_forward<uint16_t>(p, a.stream) : launch_forward<float>(p, a.stream);
  return hipGetLastError();
}

hipError_t launch_qk_norm_backward(const QkArgs& a) {
  QkParams p = params_of(a);
  share(p.tokens, a.heads[0], a.heads[1], 64 / threads_of(p), p.blocks);
  a.dtype == 1 ? launch_backward<uint16_t>(p, a.stream) : launch_backward<float>(p, a.stream);
  return hipGetLastError();
}

}  // namespace ss2d
