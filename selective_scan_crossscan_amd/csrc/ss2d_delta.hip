// The gated delta rule over prompts (ss2d_delta.h has the mathematics): the walk's kernels, the carry along segments, the
// plan and the launches.
//
// Few sequences and heads leave CUs idle, so sequences are then cut into segments.  What a segment does to the state is
// affine, h -> M h + u: u is the walk from 0, M (keys x keys) the walk from the identity with values 0, both by the same
// kernel, and a carry along the segments gives the states before them.
//
// us of 38144 packed tokens in six sequences, 16 heads of 128, bf16: systems 98, segments 344, carry 81, outputs 382; of
// 16 x 2048 tokens systems 90, outputs 329.
#include "ss2d_delta_walk.h"

namespace ss2d {
namespace {

constexpr int kCarryColumns = 32;

template <typename E, int C, int KP, DeltaPass PASS, bool TINY>
__global__ __launch_bounds__(256, TINY ? 1 : 2) void delta_walk(DeltaParams p) {
  __shared__ WalkTiles<E, C, KP, 64, PASS> lds;
  walk<E, C, KP, 64, PASS, TINY>(p, (uint32_t)block_id(), lds);
}

// One workgroup carries 32 value columns of a head along its sequence's segments: h <- M h + u forwards, h <- M' h + u
// backwards, h before (behind) each segment in the place of its u.  The first one's too: the last segment's workgroup may
// write the final state over the initial one before the first has begun.  A wave owns 16 (at 256 keys 32) rows of the
// result and reads those of M alone, the next segment's while this one's are multiplied; h goes round through LDS as
// fragments in parts: 3.5 us a segment of 128 keys, the latency of M's loads, the parts and the barrier one after the
// other.  (With 16 columns per wave and all of M read by each 10 us.)
template <int KP>
constexpr int kCarryThreads = KP == 256 ? 512 : KP * 4;
template <int KP>
struct CarryTiles {
  __attribute__((aligned(16))) uint32_t parts[2][KP / 32][kCarryColumns / 16][3][64][4];
};
template <int KP, bool REVERSE>
__device__ __forceinline__ void carry(const CarryParams& p, uint32_t block, CarryTiles<KP>& lds) {
  constexpr int NK = KP / 16, NW = NK < 8 ? NK : 8, OWN = NK / NW, NC = KP / 32, NV = kCarryColumns / 16, PF = 3;
  constexpr bool AHEAD = kAhead<KP>;  // the next segment's M and u wait in registers
  auto& parts = lds.parts;
  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const int tile = block % p.vtiles, head = block / p.vtiles % p.heads, unit = block / p.vtiles / p.heads;
  Segment first;  // a sequence's; the unit is its part, of equal lengths the sequence
  const int64_t slot = p.map.cu ? unit : (int64_t)unit * p.map.nseg;
  if (!find_segment(p.map, slot, first, p.cut) || first.begin > 0) return;
  const int s = first.s;
  const int64_t n = (first.len + p.map.seg_len - 1) / p.map.seg_len;  // segments
  if (n < 2) return;
  const int64_t kv = (int64_t)p.K * p.V;
  auto row = [&](int a, int r) { return (wave + a * NW) * 16 + 4 * g + r; };
  auto col = [&](int t) { return tile * kCarryColumns + t * 16 + l; };
  auto place = [&](int a, int t, int r) { return (int64_t)min(row(a, r), p.K - 1) * p.V + min(col(t), p.V - 1); };
  auto inside = [&](int a, int t, int r) { return row(a, r) < p.K && col(t) < p.V; };
  auto at = [&](int64_t i) { return (slot + (REVERSE ? n - 1 - i : i)) * p.heads + head; };
  f32x4 h[OWN][NV], add[OWN][NV];
  float m[OWN][AHEAD ? NC : 1][8];
  auto load_map = [&](int64_t i, int a, int c) {  // segment i's M, 32 columns of the wave's rows
    const float* map = p.seg_map + at(i) * (KP * KP);
    const int k = (wave + a * NW) * 16 + l;
    float(&to)[8] = m[a][AHEAD ? c : 0];
    if (REVERSE) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        to[r] = map[(c * 32 + 4 * g + r) * KP + k];
        to[4 + r] = map[(c * 32 + 16 + 4 * g + r) * KP + k];
      }
    } else {
      const float* x = map + k * KP + c * 32 + 4 * g;
      stack(*reinterpret_cast<const f32x4*>(x), *reinterpret_cast<const f32x4*>(x + 16), to);
    }
  };
  auto load = [&](int64_t i) {  // segment i's u, and M
    const float* u = p.seg + at(i) * kv;
#pragma unroll
    for (int a = 0; a < OWN; ++a) {
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) add[a][t][r] = u[place(a, t, r)];
      if (AHEAD)
#pragma unroll
        for (int c = 0; c < NC; ++c) load_map(i, a, c);
    }
  };
  auto put = [&](int64_t i) {  // h before (behind) segment i
    float* u = p.seg + at(i) * kv;
#pragma unroll
    for (int a = 0; a < OWN; ++a)
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (inside(a, t, r)) u[place(a, t, r)] = h[a][t][r];
  };
  load(0);
  const float* from = p.from ? p.from + ((int64_t)s * p.heads + head) * kv : nullptr;
#pragma unroll
  for (int a = 0; a < OWN; ++a)
#pragma unroll
    for (int t = 0; t < NV; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = from ? from[place(a, t, r)] : 0.f;
        h[a][t][r] = inside(a, t, r) ? x : 0.f;
      }
  for (int64_t i = 0; i < n; ++i) {
    if (i + 1 == n) {
      put(i);
      break;
    }
    auto& buffer = parts[i & 1];
#pragma unroll
    for (int a = 0; a < OWN; ++a)
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        const int k = wave + a * NW;
        f32x4 x = h[a][t];
#pragma unroll
        for (int q = 0; q < PF; ++q) {
          const uint32_t w[2] = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
          __builtin_memcpy(__builtin_assume_aligned(&buffer[k / 2][t][q][lane][2 * (k & 1)], 8), w, 8);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            x[2 * r] -= __uint_as_float(w[r] << 16);
            x[2 * r + 1] -= __uint_as_float(w[r] & 0xffff0000u);
          }
        }
      }
    Frag<uint16_t> f[AHEAD ? NC : 1][OWN][PF];
    if (AHEAD)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int a = 0; a < OWN; ++a) split_parts(m[a][c], f[AHEAD ? c : 0][a]);
    __builtin_amdgcn_sched_barrier(0);
    put(i);  // behind the uses of what was loaded before: a wait for those would be one for these stores too
#pragma unroll
    for (int a = 0; a < OWN; ++a)
#pragma unroll
      for (int t = 0; t < NV; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) h[a][t][r] = inside(a, t, r) ? add[a][t][r] : 0.f;
    __syncthreads();  // h is whole; the buffer is next written behind the next barrier
    if (AHEAD) load(i + 2 < n ? i + 1 : i);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (!AHEAD)
#pragma unroll
        for (int a = 0; a < OWN; ++a) {
          load_map(i, a, c);
          split_parts(m[a][0], f[0][a]);
        }
#pragma unroll
      for (int t = 0; t < NV; ++t) {
        Frag<uint16_t> b[PF];
#pragma unroll
        for (int q = 0; q < PF; ++q) __builtin_memcpy(&b[q], __builtin_assume_aligned(buffer[c][t][q][lane], 16), 16);
#pragma unroll
        for (int x = PF - 1; x >= 0; --x)
#pragma unroll
          for (int q = 0; q <= x; ++q)
#pragma unroll
            for (int a = 0; a < OWN; ++a) h[a][t] = mma(f[AHEAD ? c : 0][a][q], b[x - q], h[a][t]);
      }
      if (!AHEAD) __builtin_amdgcn_sched_barrier(0);
    }
    if (!AHEAD) load(i + 2 < n ? i + 1 : i);
  }
}

// The carry of the states, or of both ways' in one grid: each alone leaves CUs idle.
template <int KP, bool BOTH>
__global__ __launch_bounds__(kCarryThreads<KP>) void delta_carry(CarryParams p, CarryParams r) {
  __shared__ CarryTiles<KP> lds;
  const uint32_t block = (uint32_t)block_id(), n = p.blocks;
  if (block < n)
    carry<KP, false>(p, block, lds);
  else if (BOTH && block - n < n)
    carry<KP, true>(r, block - n, lds);
}

template <typename E, int C, DeltaPass PASS>
hipError_t launch_walk(DeltaParams p, const DeltaPlan& pl, hipStream_t st) {
  p.vtiles = (p.V + 63) / 64;
  p.ktiles = (pl.a.kp + 63) / 64;
  p.blocks = (uint32_t)((PASS == kSegments ? pl.parts : pl.a.slots) * p.heads);
  const int64_t blocks = spread_blocks(p.blocks, PASS == kSegments ? p.vtiles + p.ktiles : p.vtiles);
  with_keys(pl, [&](auto kp, auto tiny) {
    delta_walk<E, C, kp(), PASS, tiny()><<<grid_of(blocks, 256), dim3(256), 0, st>>>(p);
  });
  return hipGetLastError();
}

struct Regions {
  size_t systems, seg_state, seg_map, end;
};
Regions regions(const DeltaPlan& pl, int64_t heads, int64_t K, int64_t V, int dtype) {
  Regions r{};
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += ((size_t)bytes + 255) / 256 * 256;
    return here;
  };
  r.systems = take(pl.a.chunks * heads * system_bytes(pl, dtype));
  r.seg_state = take(pl.a.split ? pl.parts * heads * K * V * 4 : 0);
  r.seg_map = take(pl.a.split ? pl.parts * heads * pl.a.kp * pl.a.kp * 4 : 0);
  r.end = at;
  return r;
}

}  // namespace

// Chunks of 64 tokens (32 in fp32).  Sequences are cut so that there are about two workgroups per CU, packed ones, of which
// only some may be long, four; into three segments at least, as two would be walked twice for less than twice the speed.
// 16 heads of 128, us for 1, 2, 3 and 4 workgroups per CU: 8192 tokens in one sequence 255, 257, 298, 316, gradients of
// 2 x 4096 tokens 718, 622, 704, 688; for twice as many of each, 38144 tokens in six packed sequences 1075, 886, 960, 973.
DeltaPlan plan_delta(int64_t sequences, int64_t tokens, int64_t heads, int64_t key_dim, int64_t value_dim, bool packed,
                     int dtype, bool backward) {
  DeltaPlan pl;
  pl.backward = backward;
  AttentionPlan& a = pl.a;
  const int64_t few = dtype == 1 ? 8 : 4;  // values in 16 bytes
  a.tiny = key_dim < few || value_dim < few;
  a.kp = a.tiny ? (key_dim <= 32 ? 32 : 256) : key_dim <= 32 ? 32 : key_dim <= 64 ? 64 : key_dim <= 128 ? 128 : 256;
  a.vt = 64;
  a.vtiles = (int)((value_dim + 63) / 64);
  const int64_t chunk = a.chunk = dtype == 1 ? 64 : 32;
  const int64_t longest = packed ? tokens : tokens / sequences;
  const int64_t each = (packed && sequences > 1 ? 1024 : 512) / (heads * a.vtiles);  // segments of all sequences together
  int64_t parts = packed ? (each - sequences > each / 2 ? each - sequences : each / 2) : each / sequences;
  if (parts < 1) parts = 1;
  int64_t seg = (longest + parts - 1) / parts;
  if (seg < 4 * chunk) seg = 4 * chunk;
  seg = (seg + chunk - 1) / chunk * chunk;
  a.split = longest > 2 * seg;
  if (!a.split) seg = (longest + chunk - 1) / chunk * chunk;
  a.seg_len = seg;
  a.nseg = (int)((longest + seg - 1) / seg);
  a.slots = packed ? tokens / seg + sequences : sequences * a.nseg;
  // Packed sequences' kept segments are numbered as their slots are, or with many sequences those of the cut ones alone:
  // 1024 sequences of 64 tokens, 16 heads of 128, keep 68 MiB for them instead of 2080, 1395 us instead of 1646.
  pl.cut = packed && sequences > tokens / seg + 2;
  pl.parts = pl.cut ? 2 * tokens / seg + 2 : a.slots;
  a.chunks = packed ? tokens / chunk + sequences : sequences * ((longest + chunk - 1) / chunk);
  return pl;
}

int64_t delta_blocks(const DeltaPlan& pl, int64_t sequences, int64_t heads, int64_t value_dim) {
  const int64_t v = (value_dim + 63) / 64, k = (pl.a.kp + 63) / 64;
  const int64_t most = pl.a.slots > pl.parts ? pl.a.slots : pl.parts, walk = spread_blocks(most * heads, (int)(2 * v + k)),
                systems = pl.a.chunks * heads,
                carry = 2 * (sequences > pl.parts ? sequences : pl.parts) * heads * ((value_dim + kCarryColumns - 1) / kCarryColumns);
  return walk > systems ? (walk > carry ? walk : carry) : systems > carry ? systems : carry;
}

size_t delta_workspace_bytes(const DeltaPlan& pl, int64_t heads, int64_t key_dim, int64_t value_dim, int dtype) {
  return regions(pl, heads, key_dim, value_dim, dtype).end;
}

DeltaParams delta_params(const DeltaArgs& a, const DeltaPlan& pl) {
  DeltaParams p{};
  const AttentionArgs& f = a.f;
  p.q = f.q;
  p.k = f.k;
  p.v = f.v;
  p.g = f.log_decay;
  p.beta = a.beta;
  p.state_in = f.state_in;
  p.o = f.o;
  p.state_out = f.state_out;
  p.map = sequence_map(f, pl.a);
  p.chunk_map = p.map;
  p.chunk_map.seg_len = pl.a.chunk;
  p.chunk_map.nseg = (int)((f.tokens / f.sequences + pl.a.chunk - 1) / pl.a.chunk);
  for (int i = 0; i < 3; ++i) {
    p.q_stride[i] = f.q_stride[i];
    p.k_stride[i] = f.k_stride[i];
    p.v_stride[i] = f.v_stride[i];
    p.g_stride[i] = f.g_stride[i];
    p.b_stride[i] = a.beta_stride[i];
  }
  p.groups = (int)f.groups;
  p.heads = (int)f.heads;
  p.K = (int)f.key_dim;
  p.V = (int)f.value_dim;
  p.scale = f.scale;
  p.split = pl.a.split;
  p.cut = pl.cut;
  p.system_stride = system_bytes(pl, f.dtype);
  return p;
}

hipError_t launch_delta_segments(DeltaParams p, const DeltaPlan& pl, int dtype, hipStream_t st) {
  const hipError_t e = dtype == 1 ? launch_walk<uint16_t, 64, kSegments>(p, pl, st) : launch_walk<float, 32, kSegments>(p, pl, st);
  if (e != hipSuccess) return e;
  const CarryParams c{p.seg_state, p.seg_map, p.state_in, p.map, p.cut, p.heads, p.K, p.V, 0, 0};
  return launch_delta_carry(c, nullptr, pl, st);
}

hipError_t launch_delta_carry(CarryParams c, const CarryParams* back, const DeltaPlan& pl, hipStream_t st) {
  c.vtiles = (c.V + kCarryColumns - 1) / kCarryColumns;
  c.blocks = (uint32_t)((c.map.cu ? pl.parts : (int64_t)c.map.sequences) * c.heads * c.vtiles);
  CarryParams r = back ? *back : c;
  r.vtiles = c.vtiles;
  r.blocks = c.blocks;
  with_keys(pl, [&](auto kp, auto) {
    constexpr int threads = kCarryThreads<kp()>;
    const dim3 grid = grid_of(back ? 2 * (int64_t)c.blocks : c.blocks, threads), block(threads);
    if (back)
      delta_carry<kp(), true><<<grid, block, 0, st>>>(c, r);
    else
      delta_carry<kp(), false><<<grid, block, 0, st>>>(c, r);
  });
  return hipGetLastError();
}

hipError_t launch_delta_states(DeltaParams p, const DeltaPlan& pl, int dtype, hipStream_t st) {
  return dtype == 1 ? launch_walk<uint16_t, 64, kStates>(p, pl, st) : launch_walk<float, 32, kStates>(p, pl, st);
}

hipError_t launch_delta(const DeltaArgs& a, const DeltaPlan& pl) {
  const AttentionArgs& f = a.f;
  const Regions rg = regions(pl, f.heads, f.key_dim, f.value_dim, f.dtype);
  char* ws = static_cast<char*>(f.workspace);
  DeltaParams p = delta_params(a, pl);
  p.systems = ws + rg.systems;
  p.seg_state = reinterpret_cast<float*>(ws + rg.seg_state);
  p.seg_map = reinterpret_cast<float*>(ws + rg.seg_map);
  hipError_t e = launch_delta_systems(p, pl, f.dtype, f.stream);
  if (e == hipSuccess && pl.a.split) e = launch_delta_segments(p, pl, f.dtype, f.stream);
  if (e != hipSuccess) return e;
  return f.dtype == 1 ? launch_walk<uint16_t, 64, kOutputs>(p, pl, f.stream) : launch_walk<float, 32, kOutputs>(p, pl, f.stream);
}

}  // namespace ss2d
