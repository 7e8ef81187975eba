// Internal interface of the token-sequence operators (include/ss2d_tokens.h):
// launch arguments, already validated by ss2d_tokens_api.hip, and the device
// helpers their kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ss2d {

constexpr int kMaxKeyDim = 256;
constexpr int kMaxValueDim = 1024;
constexpr int64_t kMaxTokenStride = (1 << 24) - 1;  // a factor of 24 bits; 64 tokens' offsets fit 32
constexpr int kMaxNormDim = 16384;
constexpr int kScaleBlock = 128;  // channels per scale of the 8-bit values

struct NormArgs {
  const void* x;
  const void* residual;   // or null
  const float* weight;    // or null
  void* residual_out;     // or null
  void* y;
  float* scales;          // or null: y in the storage type
  float eps;
  int64_t rows, dim;
  int dtype;
  hipStream_t stream;
};
hipError_t launch_rms_norm(const NormArgs& a);

struct NormBackwardArgs {
  const void* r;
  const float* weight;    // or null
  const void* dy;
  const void* dresidual;  // or null
  void* dx;
  float* dweight;         // or null
  float* partial;         // norm_backward_blocks(rows, dim) x dim, with dweight
  float eps;
  int64_t rows, dim;
  int dtype;
  hipStream_t stream;
};
hipError_t launch_rms_norm_backward(const NormBackwardArgs& a);
// Workgroups of the backward, each with a row of partial weight gradients.
int64_t norm_backward_blocks(int64_t rows, int64_t dim);

struct StepArgs {
  const void *q, *k, *v;
  const float* log_decay;
  float* state;
  const int32_t* index;  // or null
  void* o;
  int64_t rows, slots, groups, heads, key_dim, value_dim, q_row, k_row, v_row;
  float scale;
  int dtype;
  hipStream_t stream;
};
hipError_t launch_attention_step(const StepArgs& a);

struct MatmulArgs {
  const void* a;          // (m, k) e4m3
  const float* a_scales;  // (m, ceil(k / 128))
  const void* b;          // (n, k) e4m3
  const float* b_scales;  // (ceil(n / 128), ceil(k / 128))
  void* out;              // (m, n)
  int64_t m, n, k;
  int dtype;
  hipStream_t stream;
};
hipError_t launch_matmul_fp8(const MatmulArgs& a);

// A launch of `blocks` workgroups, along x and, where their threads pass 2^31, y too: an axis takes fewer than 2^32
// threads, and one with more runs a part of them without an error.  The axes may hold a few workgroups too many, which
// leave by block_id().
inline dim3 grid_of(int64_t blocks, int threads) {
  const int64_t most = ((int64_t)1 << 31) / threads, y = (blocks + most - 1) / most;
  return dim3((unsigned)((blocks + y - 1) / y), (unsigned)y);
}

// ------------------------------------------------------------------ device helpers
namespace tok {

// This workgroup's number in a grid_of.
__device__ __forceinline__ int64_t block_id() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

constexpr float kLog2e = 1.4426950408889634f;
// A decay under exp(-104) is 0 in fp32; sums of clamped logarithms stay finite.
constexpr float kMinLogDecay = -104.f;

__device__ __forceinline__ float clamp_log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }  // keeps NaN

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Two floats to two packed bf16, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// 16 bytes at an address that need only be aligned to its elements: gfx950's
// global memory takes such accesses as they are.
struct __attribute__((packed, aligned(2))) Bytes16 {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(2))) Bytes8 {
  uint32_t w[2];
};

// Eight elements p[0..7] of a row, of which the first n are there (the others are 0).  Across the row's end they come
// from the 16 bytes (32 in fp32) that end where it does, moved down: one load for any n.  Element by element it would
// double a ragged row's time (81000 rows of 414 channels in bf16: 111 us against 59).  `whole`: the row has eight
// elements at all; if not, they are gathered one by one.
__device__ __forceinline__ void load8(const float* p, int n, bool whole, float (&v)[8]) {
  if (n >= 8 || (n > 0 && whole)) {
    const int k = n >= 8 ? 0 : 8 - n;
    const Bytes16 a = *reinterpret_cast<const Bytes16*>(p - k), b = *reinterpret_cast<const Bytes16*>(p - k + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a.w[i]);
      v[4 + i] = __uint_as_float(b.w[i]);
    }
    if (k) {
#pragma unroll
      for (int m = 4; m; m >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k & m ? (i + m < 8 ? v[i + m] : 0.f) : v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const float f = p[j];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i == j ? f : v[i];
    }
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, int n, bool whole, float (&v)[8]) {
  uint64_t lo = 0, hi = 0;
  if (n >= 8 || (n > 0 && whole)) {
    const int k = n >= 8 ? 0 : 8 - n;
    const Bytes16 a = *reinterpret_cast<const Bytes16*>(p - k);
    lo = a.w[0] | (uint64_t)a.w[1] << 32;
    hi = a.w[2] | (uint64_t)a.w[3] << 32;
    if (k) {
      const int s = 16 * k;  // 16 .. 112
      lo = s < 64 ? lo >> s | hi << (64 - s) : hi >> (s - 64);
      hi = s < 64 ? hi >> s : 0;
    }
  } else {
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const uint64_t f = (uint64_t)p[j] << (16 * (j & 3));
      lo |= j < 4 ? f : 0;
      hi |= j < 4 ? 0 : f;
    }
  }
  const uint32_t w[4] = {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(w[i] & 0xffffu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    Bytes16 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a.w[i] = __float_as_uint(v[i]);
      b.w[i] = __float_as_uint(v[4 + i]);
    }
    *reinterpret_cast<Bytes16*>(p) = a;
    *reinterpret_cast<Bytes16*>(p + 4) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&v)[8]) {
  Bytes16 a;
#pragma unroll
  for (int i = 0; i < 4; ++i) a.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  if (n >= 8) {
    *reinterpret_cast<Bytes16*>(p) = a;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(i & 1 ? a.w[i / 2] >> 16 : a.w[i / 2]);
  }
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, 0.f); }

// v moved across lanes by a DPP pattern; lanes without a source, and rows outside
// ROWS, get 0.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, true));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp(double v) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROWS, 0xf, true);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROWS, 0xf, true);
  return __hiloint2double(hi, lo);
}
constexpr int kRowShr = 0x110, kRowRor = 0x120;  // + 1 .. 15: lanes of a row of 16 shifted up, rotated
constexpr int kBcast15 = 0x142, kBcast31 = 0x143;  // a row's (half's) last lane to the next row (half)

// Sum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp<kRowRor + 8>(v);
  v += dpp<kRowRor + 4>(v);
  v += dpp<kRowRor + 2>(v);
  return v + dpp<kRowRor + 1>(v);
}
// Sum over the lanes 16 apart, in every lane.
__device__ __forceinline__ float across_rows(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
// Sum over the 64 lanes of a wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) { return across_rows(row16_sum(v)); }

// Inclusive sum over the lanes up to this one.
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
  v += dpp<kRowShr + 1>(v);
  v += dpp<kRowShr + 2>(v);
  v += dpp<kRowShr + 4>(v);
  v += dpp<kRowShr + 8>(v);
  v += dpp<kBcast15, 0xa>(v);  // rows 1 and 3
  return v + dpp<kBcast31, 0xc>(v);  // rows 2 and 3
}

}  // namespace tok
}  // namespace ss2d
