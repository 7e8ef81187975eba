// Root-mean-square norm of rows with the residual's addition, and its gradients.
//
//   r = x + residual,  y = r rstd weight,  rstd = 1 / sqrt(mean(r^2) + eps);
//   8-bit output: per 128 channels s = max(max|y| / 448, 2^-126), q = e4m3(y / s);
//   dx = dresidual + rstd (weight dy - xhat mean(weight dy xhat)),  xhat = r rstd,
//   dweight = sum over rows of dy xhat.
//
// Bound by memory: every value is read once and written once.  A row is held in
// registers, eight consecutive channels per thread, between the sum over it and
// the output, so no value is read twice.  A row gets the threads of up to 64 that
// it needs (several rows per wave) up to 512 channels and otherwise one workgroup
// of four waves up to 2048 channels, eight up to 8192 (the gradients' 16 behind 4096)
// and 16 behind (the gradients' eight, with registers for four times eight channels:
// 16 waves spilled, 113 us against 71 for 2048 rows of 16384), which also keeps a single row's latency at one load, one sum and one
// store.  The sums are fp32.
// 16384 rows of 2048 in bf16 with a residual: 47 us on inputs that change from call to
// call, 5.8 TB/s; 38 on the same ones, part of which the last-level cache holds.  The
// gradients 58 us, 4.6 TB/s, and 53.
//
// Threads per row, us for 4 and 16384 rows (bf16 with a residual, one launch after another in a graph, four sets of
// inputs): 512 channels
// 64 threads 2.6, 12.1, 256 threads 2.9, 21.4; 1024 channels 64 4.2, 25.4, 256
// 2.7, 25.6; 2048 channels 64 4.2, 49.9, 256 2.8, 42.3, 512 2.9, 54.1; 4096
// channels 256 3.3, 98, 512 3.0, 92, 1024 3.3, 116; 8192 channels 512 3.6, 191,
// 1024 3.6, 200.  2^23 values in rows of 59 channels: 8 threads 15.7, 64 50.4; of
// 64: 8 11.9, 64 38.7; of 128: 16 11.9, 64 21.8; of 256: 32 12.1, 64 14.2.
#include "ss2d_token_ops.h"

namespace ss2d {
namespace {

using namespace tok;

// Sum over the THREADS threads that share a row (`red`: one float per wave).
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if (THREADS < 64) {
#pragma unroll
    for (int m = 1; m < THREADS; m <<= 1) v += __shfl_xor(v, m);
    return v;
  }
  v = wave_sum(v);
  if (THREADS > 64) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) v += red[i];
  }
  return v;
}

// Threads of a workgroup: one row's, or 256 for the rows of a wave each or less.
constexpr int block_threads(int per_row) { return per_row <= 64 ? 256 : per_row; }

template <typename S, int THREADS, int NV, bool FP8>
__global__ __launch_bounds__(block_threads(THREADS)) void rms_norm_kernel(
    const S* x, const S* residual, const float* __restrict__ weight, S* residual_out, void* yv,
    float* __restrict__ scales, float eps, int64_t rows, int dim) {
  __shared__ float red[THREADS > 64 ? THREADS / 64 : 1];
  const int t = threadIdx.x % THREADS;
  const int64_t row = block_id() * (block_threads(THREADS) / THREADS) + threadIdx.x / THREADS;
  if (row >= rows) return;  // whole rows, and only where a row is within a wave: no barrier follows there
  const int64_t at = row * dim;
  float v[NV][8], w[NV][8];
  float sq = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * THREADS) * 8;
    load8(x + at + c, dim - c, dim >= 8, v[j]);
    if (weight) load8(weight + c, dim - c, dim >= 8, w[j]);
    if (residual) {
      float r[8];
      load8(residual + at + c, dim - c, dim >= 8, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] += r[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(v[j][i], v[j][i], sq);
  }
  const float rstd = 1.0f / sqrtf(row_sum<THREADS>(sq, red) / (float)dim + eps);
  // 8 bits: rstd as a power of two and a factor in [1, 2)
  const bool finite = rstd < __builtin_inff();
  const float power = finite ? __uint_as_float(__float_as_uint(rstd) & 0x7f800000u) : rstd;
  const float factor = finite ? __uint_as_float((__float_as_uint(rstd) & 0x007fffffu) | 0x3f800000u) : 1.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * THREADS) * 8;
    if (residual_out) store8(residual_out + at + c, dim - c, v[j]);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[j][i] *= FP8 ? power : rstd;
      if (weight) v[j][i] *= w[j][i];
      if (FP8) amax = fmaxf(amax, fabsf(v[j][i]));  // a NaN is passed over here and stays one below
    }
    if (!FP8) {
      store8(static_cast<S*>(yv) + at + c, dim - c, v[j]);
    } else {
      // 16 consecutive threads hold one block of 128 channels.  v is y / factor, which cancels out of
      // y / s = v 448 / max|v|: fewer roundings before the one to 8 bits, and one division per block.  The power of two
      // costs no rounding and keeps v within a factor of two of y, so the quotient stays in range: a scale over
      // 2^-126 has max|v| over 224 x 2^-126, and 448 / max|v| under 2^127
#pragma unroll
      for (int m = 1; m < 16; m <<= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
      constexpr float kLeast = 1.17549435e-38f;  // 2^-126
      const float top = amax * factor / 448.0f;
      const bool least = !(top > kLeast);  // nearly nothing, or NaN
      const float s = least ? kLeast : top, k = least ? factor : 448.0f / amax, k2 = least ? 1.0f / kLeast : 1.0f;
      const int blocks = (dim + kScaleBlock - 1) / kScaleBlock;
      if ((threadIdx.x & 15) == 0 && c < dim) scales[row * blocks + c / kScaleBlock] = s;
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z = v[j][i] * k2 * k;
        u[i] = z > 448.f ? 448.f : z < -448.f ? -448.f : z;  // keeps NaN
      }
      uint32_t q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(u[4 * i], u[4 * i + 1], 0, false);
        q[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(u[4 * i + 2], u[4 * i + 3], p, true);
      }
      uint8_t* y = static_cast<uint8_t*>(yv) + at + c;
      if (dim - c >= 8) {
        __builtin_memcpy(y, q, 8);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < dim - c) y[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

// Each workgroup takes rows blockIdx.x, blockIdx.x + gridDim.x, ... (a wave the
// 64 / THREADS rows of its groups at a time) and keeps its part of the weight's
// gradient in registers; norm_sum_partials adds the parts.
template <typename S, int THREADS, int NV>
__global__ __launch_bounds__(THREADS < 64 ? 64 : THREADS) void rms_norm_backward_kernel(
    const S* __restrict__ r, const float* __restrict__ weight, const S* dy, const S* dresidual, S* dx,
    float* __restrict__ partial, float eps, int64_t rows, int dim) {
  __shared__ float red[THREADS > 64 ? 2 * THREADS / 64 : 1];
  constexpr int ROWS = THREADS < 64 ? 64 / THREADS : 1;
  const int t = threadIdx.x % THREADS;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (t + j * THREADS) * 8;
    if (weight) load8(weight + c, dim - c, dim >= 8, w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!weight) w[j][i] = 1.f;
      dw[j][i] = 0.f;
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS; row < rows; row += (int64_t)gridDim.x * ROWS) {
    const int64_t at = row * dim;
    float x[NV][8], g[NV][8];
    float sq = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + j * THREADS) * 8;
      load8(r + at + c, dim - c, dim >= 8, x[j]);
      load8(dy + at + c, dim - c, dim >= 8, g[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sq = fmaf(x[j][i], x[j][i], sq);
        dot = fmaf(x[j][i], g[j][i] * w[j][i], dot);
      }
    }
    sq = row_sum<THREADS>(sq, red);
    dot = row_sum<THREADS>(dot, red + (THREADS > 64 ? THREADS / 64 : 0));
    const float rstd = 1.0f / sqrtf(sq / (float)dim + eps);
    const float mean = dot * rstd / (float)dim;  // mean of weight dy xhat
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + j * THREADS) * 8;
      float d[8];
      if (dresidual) load8(dresidual + at + c, dim - c, dim >= 8, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = x[j][i] * rstd;
        dw[j][i] = fmaf(g[j][i], xh, dw[j][i]);
        const float v = rstd * (w[j][i] * g[j][i] - xh * mean);
        d[i] = dresidual ? d[i] + v : v;
      }
      store8(dx + at + c, dim - c, d);
    }
  }
  if (partial) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (t + j * THREADS) * 8;
#pragma unroll
      for (int m = THREADS; m < 64; m <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] += __shfl_xor(dw[j][i], m);
      if (threadIdx.x < THREADS) store8(partial + (int64_t)blockIdx.x * dim + c, dim - c, dw[j]);
    }
  }
}

// dweight[c] = sum over the workgroups' parts: 32 channels by 32 ranges of parts
// per workgroup, eight loads in flight per thread, the ranges' sums added in order.
constexpr int kSumCols = 32, kSumRanges = 32;
__global__ __launch_bounds__(kSumCols * kSumRanges) void norm_sum_partials(const float* __restrict__ partial,
                                                                           float* __restrict__ dw, int parts, int dim) {
  __shared__ float sums[kSumRanges][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, range = threadIdx.x / kSumCols, c = blockIdx.x * kSumCols + col;
  float s = 0.f;
  if (c < dim)
    for (int p = range; p < parts; p += 8 * kSumRanges) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = p + i * kSumRanges;
        v[i] = q < parts ? partial[(int64_t)q * dim + c] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  sums[range][col] = s;
  __syncthreads();
  if (range == 0 && c < dim) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumRanges; ++i) s += sums[i][col];
    dw[c] = s;
  }
}

template <typename S, int THREADS, int NV>
void launch_norm_t(const NormArgs& a) {
  const int per = block_threads(THREADS) / THREADS;
  const dim3 block(block_threads(THREADS)), grid = grid_of((a.rows + per - 1) / per, block.x);
  if constexpr (THREADS >= 16) {  // a scale's threads
    if (a.scales) {
      rms_norm_kernel<S, THREADS, NV, true><<<grid, block, 0, a.stream>>>(
          (const S*)a.x, (const S*)a.residual, a.weight, (S*)a.residual_out, a.y, a.scales, a.eps, a.rows, (int)a.dim);
      return;
    }
  }
  rms_norm_kernel<S, THREADS, NV, false><<<grid, block, 0, a.stream>>>(
      (const S*)a.x, (const S*)a.residual, a.weight, (S*)a.residual_out, a.y, nullptr, a.eps, a.rows, (int)a.dim);
}

template <typename S>
hipError_t launch_norm_s(const NormArgs& a) {
  // 8 bits: at least the 16 threads that share a scale
  if (a.dim <= 64 && !a.scales)
    launch_norm_t<S, 8, 1>(a);
  else if (a.dim <= 128)
    launch_norm_t<S, 16, 1>(a);
  else if (a.dim <= 256)
    launch_norm_t<S, 32, 1>(a);
  else if (a.dim <= 512)
    launch_norm_t<S, 64, 1>(a);
  else if (a.dim <= 2048)
    launch_norm_t<S, 256, 1>(a);
  else if (a.dim <= 4096)
    launch_norm_t<S, 512, 1>(a);
  else if (a.dim <= 8192)
    launch_norm_t<S, 512, 2>(a);
  else
    launch_norm_t<S, 1024, 2>(a);
  return hipGetLastError();
}

// The gradients' threads per row, each with `pieces` times eight channels, and their workgroups at most, each of one
// row or of as many as a wave has groups of threads.  16 waves per CU (2048 channels with 8, 16 and 32 waves 75, 54 and
// 58 us, 4096 channels 154, 110 and 112), 8 where a wave has whole rows (2^23 values in bf16, 8 against 16: rows of 64
// 20.6 us and 23.3, of 512 21.6 and 25.1, of 59 26.9 and 26.6, of 414 29.1 and 28.4) and behind 8192 channels, whose
// registers leave a CU one workgroup of eight (2048 rows of 16384 by 256, 512 and 1024 workgroups: bf16 70, 78 and 94
// us, fp32 124, 122 and 141).
struct BackwardShape {
  int threads, pieces, most;
  int64_t blocks(int64_t rows) const {  // no more than there are rows
    const int per = threads < 64 ? 64 / threads : 1;
    const int64_t all = (rows + per - 1) / per;
    return all < most ? all : most;
  }
};
BackwardShape backward_shape(int64_t dim) {
  if (dim <= 64) return {8, 1, 2048};
  if (dim <= 128) return {16, 1, 2048};
  if (dim <= 256) return {32, 1, 2048};
  if (dim <= 512) return {64, 1, 2048};
  if (dim <= 2048) return {256, 1, 1024};
  if (dim <= 4096) return {512, 1, 512};
  if (dim <= 8192) return {1024, 1, 256};
  return {512, 4, 256};
}

template <typename S, int THREADS, int NV>
void launch_norm_backward_t(const NormBackwardArgs& a, int64_t blocks) {
  rms_norm_backward_kernel<S, THREADS, NV><<<dim3((unsigned)blocks), dim3(THREADS < 64 ? 64 : THREADS), 0, a.stream>>>(
      (const S*)a.r, a.weight, (const S*)a.dy, (const S*)a.dresidual, (S*)a.dx, a.dweight ? a.partial : nullptr, a.eps,
      a.rows, (int)a.dim);
}

template <typename S>
hipError_t launch_norm_backward_s(const NormBackwardArgs& a) {
  const BackwardShape shape = backward_shape(a.dim);
  const int64_t blocks = shape.blocks(a.rows);
  switch (shape.threads) {
    case 8: launch_norm_backward_t<S, 8, 1>(a, blocks); break;
    case 16: launch_norm_backward_t<S, 16, 1>(a, blocks); break;
    case 32: launch_norm_backward_t<S, 32, 1>(a, blocks); break;
    case 64: launch_norm_backward_t<S, 64, 1>(a, blocks); break;
    case 256: launch_norm_backward_t<S, 256, 1>(a, blocks); break;
    case 1024: launch_norm_backward_t<S, 1024, 1>(a, blocks); break;
    default:
      if (shape.pieces == 1)
        launch_norm_backward_t<S, 512, 1>(a, blocks);
      else
        launch_norm_backward_t<S, 512, 4>(a, blocks);
  }
  if (a.dweight)
    norm_sum_partials<<<dim3((unsigned)((a.dim + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumRanges), 0, a.stream>>>(
        a.partial, a.dweight, (int)blocks, (int)a.dim);
  return hipGetLastError();
}

}  // namespace

int64_t norm_backward_blocks(int64_t rows, int64_t dim) { return backward_shape(dim).blocks(rows); }

hipError_t launch_rms_norm(const NormArgs& a) {
  return a.dtype == 1 ? launch_norm_s<uint16_t>(a) : launch_norm_s<float>(a);
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a) {
  return a.dtype == 1 ? launch_norm_backward_s<uint16_t>(a) : launch_norm_backward_s<float>(a);
}

}  // namespace ss2d
