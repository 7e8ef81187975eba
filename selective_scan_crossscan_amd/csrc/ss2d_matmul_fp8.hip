// Matrix product of e4m3 values with a scale per block of 128 (gfx950):
//
//   out[m, n] = sum_j sa[m, j] sb[n / 128, j] sum_{k in block j} a[m, k] b[n, k].
//
// For bf16 outputs every block of 128 inner indices is one
// v_mfma_f32_16x16x128_f8f6f4 per 16x16 outputs, from 0, and its result is added to
// the sum times the two scales: the scales change with every block, so they cannot
// be left to the end.  That instruction adds its products in groups of eight, in
// which it drops what lies below 2^-13 of the largest one (measured: beside 2^16,
// 2^3 is kept and 2^2 is not; between groups 2^-7 is kept): about 1.5e-5 of a
// block's sum for normal values, far under the output's rounding of 2^-8, but not
// good enough for an fp32 output.  There the values are converted to bf16, which
// is exact, and a block is four v_mfma_f32_16x16x32_bf16 (1e-8), at half the rate.  Tiles are
// formed transposed (rows n, columns m): a lane has one m, hence one product of
// scales per block for all its outputs of a column tile, and four consecutive n
// for its stores.  A fragment is 32 consecutive bytes of a row per lane, 16 rows
// by four quarters of a block, in both operands alike.
//
// Two kernels.  Products with enough outputs for tiles of 128x128 stage both
// operands through LDS, double buffered (5001 x 4096 x 4096: 102 us among
// other calls, 1646 TFLOP/s; 107 to 118 by itself).  Fewer are bound by reading b once: there a workgroup's waves split
// the inner dimension over one strip of 16 n, each streaming its part of b from
// global memory straight into fragments, and add their sums through LDS in a
// fixed order (3 x 6144 x 4096: 8.4 us, 3.0 TB/s).
#include "ss2d_token_ops.h"

namespace ss2d {
namespace {

using namespace tok;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

struct MatmulParams {
  const uint8_t *a, *b;
  const float *sa, *sb;
  void* out;
  int64_t M, N;
  int K, blocks;  // blocks: of 128 inner indices
  int mtiles, ntiles;
};

// A lane's 32 values of a block as an operand for outputs of type O.
template <typename O>
struct Operand;
template <>
struct Operand<uint16_t> {
  i32x8 v;
  __device__ __forceinline__ Operand() {}
  __device__ __forceinline__ explicit Operand(const i32x8& bytes) : v(bytes) {}
};
template <>
struct Operand<float> {
  bf16x8 v[4];
  __device__ __forceinline__ Operand() {}
  __device__ __forceinline__ explicit Operand(const i32x8& bytes) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bf16x2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes[2 * i + j], 1.f, false);
        const bf16x2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes[2 * i + j], 1.f, true);
        v[i][4 * j] = x[0];
        v[i][4 * j + 1] = x[1];
        v[i][4 * j + 2] = y[0];
        v[i][4 * j + 3] = y[1];
      }
  }
};

__device__ __forceinline__ f32x4 mfma_block(const Operand<uint16_t>& a, const Operand<uint16_t>& b) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, zero, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_block(const Operand<float>& a, const Operand<float>& b) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
  return d;
}

// Bytes p[0..15], of which the first n are there (the others are 0), at any address.
__device__ __forceinline__ i32x4 load_bytes16(const uint8_t* p, int n) {
  i32x4 r = {0, 0, 0, 0};
  if (n >= 16) {
    struct __attribute__((packed, aligned(1))) B16 {
      uint32_t w[4];
    };
    const B16 v = *reinterpret_cast<const B16*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (int)v.w[i];
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) r[i / 4] |= (int)p[i] << (8 * (i % 4));
  }
  return r;
}

template <typename O>
__device__ __forceinline__ void store_out(O* p, int64_t n, f32x4 v);
template <>
__device__ __forceinline__ void store_out(float* p, int64_t n, f32x4 v) {
  if (n >= 4) {
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}
template <>
__device__ __forceinline__ void store_out(uint16_t* p, int64_t n, f32x4 v) {
  const uint32_t w[2] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  if (n >= 4) {
    __builtin_memcpy(p, w, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
  }
}

// ------------------------------------------------------------------ tiles of 128 x 128
constexpr int kTile = 128;
constexpr int kScaleStep = 16;  // blocks of a's scales in LDS at a time

// Four waves, 64 x 64 outputs each; two workgroups share a CU.  An operand's 128
// rows of one block lie in LDS, double buffered, as 128-byte rows of eight 16-byte
// pieces, piece q of row r in place q ^ (r / 2 % 8): sixteen rows' reads of one piece
// then fall into different banks (two rows to the 64 banks, eight places each).  (Fragments straight from memory would spare half of
// LDS's traffic, but a wave's 16 rows by four pieces 32 bytes apart are 64 separate
// addresses: 232 us where this takes 108, 5001 x 4096 x 4096.)  The scales,
// one product per row and block, come through LDS as well, sixteen blocks at a time:
// read from memory where they are used, sixteen rows' lines for four bytes each, they
// cost a quarter of the time, and even b's alone made every step wait for the pieces
// on their way (loads are waited for in order).
// DMA: rows are 16-byte aligned and whole pieces long; pieces go from memory to LDS
// without registers, and those outside the operand read as 0 by the buffer's bounds.
// Otherwise they go through registers, byte by byte at a row's end.
template <typename O, bool DMA>
__global__ __launch_bounds__(256, 2) void matmul_fp8_tiles(MatmulParams p) {
  // Two buffers each, as variables of their own and with the steps written out for either: only so does the compiler see
  // that a step's reads are not of the pieces on their way, and not wait for those (136 us where this takes 108)
  __shared__ __attribute__((aligned(16))) uint8_t sm0[kTile * kScaleBlock], sm1[kTile * kScaleBlock];
  __shared__ __attribute__((aligned(16))) uint8_t sn0[kTile * kScaleBlock], sn1[kTile * kScaleBlock];
  __shared__ float scale[kTile * (kScaleStep + 1)];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63, g = lane >> 4,
            l = lane & 15;
  // Workgroups go round the eight XCDs, each with an L2 of its own: an XCD gets a band of columns of tiles and walks
  // down it row by row, so that a row of a is read once for the whole band and the band's rows of b stay in its L2.
  const int block = (int)block_id(), total = p.mtiles * p.ntiles;
  if (block >= total) return;
  const int xcd = block & 7, each = total >> 3, more = total & 7;
  const int at = xcd * each + min(xcd, more) + (block >> 3);
  const int width = (p.ntiles + 7) >> 3, band = at / (width * p.mtiles), rest = at - band * width * p.mtiles;
  const int here = min(width, p.ntiles - band * width);  // the last band may be narrower
  const int64_t m0 = (int64_t)(rest / here) * kTile, n0 = (int64_t)(band * width + rest % here) * kTile;
  const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
  const int rows_m = (int)min((int64_t)kTile, p.M - m0), rows_n = (int)min((int64_t)kTile, p.N - n0);
  const uint8_t *a = p.a + m0 * p.K, *b = p.b + n0 * p.K;

  // this thread's four pieces of an operand: rows and byte columns
  i32x4 stage_m[4], stage_n[4];
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)a, 0, (uint32_t)rows_m * (uint32_t)p.K, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)b, 0, (uint32_t)rows_n * (uint32_t)p.K, 0x00020000);
  auto fetch = [&](int kb, uint8_t* sm, uint8_t* sn) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int place = (wave * 4 + i) * 64 + lane, row = place >> 3, c = kb * kScaleBlock + ((place & 7) ^ ((row >> 1) & 7)) * 16;
      if (DMA) {
        const uint32_t at = c < p.K ? (uint32_t)row * (uint32_t)p.K + c : 1u << 30;  // past any operand's rows: 128 x 2^20 bytes
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(sm + (wave * 4 + i) * 1024), 16, at, 0, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(sn + (wave * 4 + i) * 1024), 16, at, 0, 0, 0);
      } else {
        stage_m[i] = load_bytes16(a + (int64_t)row * p.K + c, row < rows_m ? p.K - c : 0);
        stage_n[i] = load_bytes16(b + (int64_t)row * p.K + c, row < rows_n ? p.K - c : 0);
      }
    }
  };
  auto land = [&](uint8_t* sm, uint8_t* sn) __attribute__((always_inline)) {
    if (!DMA)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int place = (wave * 4 + i) * 64 + lane;
        *reinterpret_cast<i32x4*>(sm + place * 16) = stage_m[i];
        *reinterpret_cast<i32x4*>(sn + place * 16) = stage_n[i];
      }
  };
  const float* sbp = p.sb + (n0 / kScaleBlock) * p.blocks;
  // both scales' products for blocks kb .. kb + 15: a row's sixteen by sixteen lanes
  auto fetch_scales = [&](int kb) {
#pragma unroll
    for (int i = 0; i < kTile * kScaleStep / 256; ++i) {
      const int idx = threadIdx.x + i * 256, row = idx / kScaleStep, c = idx % kScaleStep;
      const int block = min(kb + c, p.blocks - 1);
      scale[row * (kScaleStep + 1) + c] = p.sa[(m0 + min(row, rows_m - 1)) * p.blocks + block] * sbp[block];
    }
  };
  auto fragment = [&](const uint8_t* s, int row) __attribute__((always_inline)) {
    const uint8_t* r = s + row * kScaleBlock;
    const i32x4 x = *reinterpret_cast<const i32x4*>(r + ((2 * g) ^ ((row >> 1) & 7)) * 16);
    const i32x4 y = *reinterpret_cast<const i32x4*>(r + ((2 * g + 1) ^ ((row >> 1) & 7)) * 16);
    return Operand<O>(__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[x][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // block kb from (sm, sn), the next one on its way into (tm, tn)
  auto step = [&](int kb, const uint8_t* sm, const uint8_t* sn, uint8_t* tm, uint8_t* tn) __attribute__((always_inline)) {
    if (kb % kScaleStep == 0) {
      if (kb > 0) __syncthreads();  // the scales before have been read
      fetch_scales(kb);
    }
    if (DMA) __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's pieces have landed
    __syncthreads();  // the block is whole, the other buffer has been read
    if (kb + 1 < p.blocks) fetch(kb + 1, tm, tn);
    float s[4];
    Operand<O> fm[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      s[t] = scale[(wm + t * 16 + l) * (kScaleStep + 1) + kb % kScaleStep];
      fm[t] = fragment(sm, wm + t * 16 + l);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const Operand<O> fn = fragment(sn, wn + x * 16 + l);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f32x4 d = mfma_block(fn, fm[t]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[x][t][r] = fmaf(d[r], s[t], acc[x][t][r]);
      }
    }
    if (kb + 1 < p.blocks) land(tm, tn);
  };
  fetch(0, sm0, sn0);
  land(sm0, sn0);
  for (int kb = 0; kb < p.blocks; kb += 2) {
    step(kb, sm0, sn0, sm1, sn1);
    if (kb + 1 < p.blocks) step(kb + 1, sm1, sn1, sm0, sn0);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t m = m0 + wm + t * 16 + l;
    if (m < p.M)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int64_t n = n0 + wn + x * 16 + 4 * g;
        store_out(static_cast<O*>(p.out) + m * p.N + n, p.N - n, acc[x][t]);
      }
  }
}

// ------------------------------------------------------------------ few rows
constexpr int kRowWaves = 8;

// MT column tiles (16 MT rows of a), one strip of 16 n; wave w takes blocks w, w + 8, ...
template <typename O, int MT>
__global__ __launch_bounds__(kRowWaves * 64) void matmul_fp8_rows(MatmulParams p) {
  __shared__ f32x4 sums[kRowWaves][MT][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const int64_t n0 = (int64_t)(blockIdx.x % p.ntiles) * 16, m0 = (int64_t)(blockIdx.x / p.ntiles) * (16 * MT);
  const bool has_n = n0 + l < p.N;
  const uint8_t* brow = p.b + (has_n ? (n0 + l) * p.K : 0);
  const float* sbp = p.sb + (n0 / kScaleBlock) * p.blocks;
  const uint8_t* arow[MT];
  const float* sap[MT];
  bool has_m[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t m = m0 + t * 16 + l;
    has_m[t] = m < p.M;
    arow[t] = p.a + (has_m[t] ? m * p.K : 0);
    sap[t] = p.sa + (has_m[t] ? m * p.blocks : 0);
  }
  auto row32 = [&](const uint8_t* row, bool has, int c) {
    const int n = has ? p.K - c : 0;
    const i32x4 x = load_bytes16(row + c, n), y = load_bytes16(row + c + 16, n - 16);
    return Operand<O>(__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < p.blocks; kb += kRowWaves) {
    const int c = kb * kScaleBlock + g * 32;
    const Operand<O> fn = row32(brow, has_n, c);
    const float sb = sbp[kb];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const Operand<O> fm = row32(arow[t], has_m[t], c);
      const float s = sap[t][kb] * sb;
      const f32x4 d = mfma_block(fn, fm);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(d[r], s, acc[t][r]);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
#pragma unroll
  for (int t0 = 0; t0 < MT; t0 += kRowWaves) {
    const int t = t0 + wave;
    if (t < MT) {
      f32x4 s = sums[0][t][lane];
#pragma unroll
      for (int w = 1; w < kRowWaves; ++w) s += sums[w][t][lane];
      const int64_t m = m0 + t * 16 + l, n = n0 + 4 * g;
      if (m < p.M && n < p.N) store_out(static_cast<O*>(p.out) + m * p.N + n, p.N - n, s);
    }
  }
}

template <typename O, int MT>
void launch_rows(MatmulParams p, hipStream_t st) {
  p.ntiles = (int)((p.N + 15) / 16);
  p.mtiles = (int)((p.M + 16 * MT - 1) / (16 * MT));
  matmul_fp8_rows<O, MT><<<dim3((unsigned)(p.ntiles * (int64_t)p.mtiles)), dim3(kRowWaves * 64), 0, st>>>(p);
}

template <typename O>
hipError_t launch_o(const MatmulArgs& x) {
  MatmulParams p{static_cast<const uint8_t*>(x.a), static_cast<const uint8_t*>(x.b), x.a_scales, x.b_scales, x.out,
                 x.m, x.n, (int)x.k, (int)((x.k + kScaleBlock - 1) / kScaleBlock), 0, 0};
  p.mtiles = (int)((x.m + kTile - 1) / kTile);
  p.ntiles = (int)((x.n + kTile - 1) / kTile);
  // Strips cost a step for every 16 x 16 outputs that a CU gets, tiles a walk over k at least, however few they are.
  // K = 4096, us of strips against tiles: 64 x 4096 15.9 (25.6), 80 x 4096 20.6 (25.7), 128 x 4096 28.5 (26.7),
  // 256 x 1024 15.6 (26.4), 512 x 1024 28.2 (26.3), 16 x 16384 22.9 (31.4), 48 x 16384 43.9 (32.4); fp32 outputs,
  // whose tiles take longer: 128 x 4096 29.1 (38.6), 256 x 4096 54.4 (38.8), 48 x 16384 46.6 (38.7).
  if (x.m * x.n >= (sizeof(O) == 2 ? 1 << 19 : 3 << 18)) {
    const dim3 grid = grid_of((int64_t)p.mtiles * p.ntiles, 256), block(256);
    // 16-byte copies into LDS; odd rows through registers (4096 cubed: 84 us against 118)
    if (x.k % 16 == 0 && (((uintptr_t)x.a | (uintptr_t)x.b) & 15) == 0)
      matmul_fp8_tiles<O, true><<<grid, block, 0, x.stream>>>(p);
    else
      matmul_fp8_tiles<O, false><<<grid, block, 0, x.stream>>>(p);
  } else if (x.m <= 16) {
    // Strips of 16, 32 or 64 rows at once; 4096 x 4096, us of the three: 16 rows 7.5, 9.2, 9.9; 32 rows 12.2, 10.2,
    // 11.7; 64 rows 20.9, 17.2, 15.6.
    launch_rows<O, 1>(p, x.stream);
  } else if (x.m <= 32) {
    launch_rows<O, 2>(p, x.stream);
  } else {
    launch_rows<O, 4>(p, x.stream);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_matmul_fp8(const MatmulArgs& x) {
  return x.dtype == 1 ? launch_o<uint16_t>(x) : launch_o<float>(x);
}

}  // namespace ss2d
