// rope.cu -- rotary positions: the table of cosines and sines, the rotation of a [tokens, heads, head_dim] view and its
// transpose, and the append to the paged 4-bit cache that rotates K (and the step's queries) on the way.
//   (a, b) -> (a cos - b sin, b cos + a sin), pair i of a head: channels (i, i + rotary/2) or (2 i, 2 i + 1)
// Products and their sum are rounded each (no multiply-add): the result then does not depend on which of a pair's
// channels a thread computes, and is what elementary fp32 arithmetic gives.
#include <algorithm>
#include <cmath>

#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "launch.h"

namespace fp4 {
namespace {

// -------------------------------------------------------------- rope_table --
// An angle is position * frequency radians modulo a turn.  With the frequency as a 64-bit fraction of a turn (steps)
// the product modulo 2^64 is the angle itself, in units of 2^-64 of a turn, exact but for the fraction's own
// rounding times the position.  cos and sin in fp64, rounded once: the entries are those of the exact angle but for one in
// some million.  Runs once a model; bound by fp64: 131,072 positions of 64 pairs: see the document's table.
struct RopeSteps {
  uint64_t step[128];
};

__global__ void __launch_bounds__(256) rope_table_kernel(const RopeSteps s, int half, double scale, int64_t entries,
                                                         float2* __restrict__ table) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < entries; i += (int64_t)gridDim.x * 256) {
    const uint64_t pos = (uint64_t)(i / half);
    const uint64_t phase = pos * s.step[i - (int64_t)pos * half];
    double sn, cs;
    sincospi((double)(int64_t)phase * 0x1p-63, &sn, &cs);  // half turns in [-1, 1)
    table[i] = make_float2((float)(cs * scale), (float)(sn * scale));
  }
}

// (a, b) turned; sgn -1: the transpose
__device__ __forceinline__ void turn(float a, float b, float2 cs, float& u, float& v) {
  u = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  v = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// n table entries from an 8-byte aligned address (16-byte where the address allows)
template <int N>
__device__ __forceinline__ void load_cs(const float2* p, bool wide, float2 (&cs)[N]) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      cs[i] = make_float2(v.x, v.y);
      cs[i + 1] = make_float2(v.z, v.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) cs[i] = __ldg(p + i);
  }
}

// Whether the rotated channels of a head are whole 16-byte pieces (and, in halves, a pair's two lie in two pieces).
__host__ __device__ inline bool whole_pieces(const RopeDesc& r) {
  return r.interleaved ? r.rotary_dim % 8 == 0 : r.rotary_dim % 16 == 0;
}

// -------------------------------------------------------------------- rope --
// What one thread does of a token's heads [first, heads) in steps of `step`, unit `u` of each head.  Whole pieces: a unit
// is two pieces of a head's halves (eight pairs), or an interleaved piece (four pairs), then the pieces that stay as
// they are.  Its cosines are loaded once for all its heads, and kBatch heads are in flight.  Otherwise a unit is a pair
// (two-byte accesses), then a channel that stays.
constexpr int kBatch = 4;

template <bool INTERLEAVED>
__device__ __forceinline__ void rope_pieces(const HeadsView& x, const uint16_t* in, uint16_t* out, const float2* row,
                                            bool wide, float sign, int rotary, int u, int first, int step) {
  constexpr int N = INTERLEAVED ? 4 : 8;  // pairs of the unit
  const int turned = rotary / (INTERLEAVED ? 8 : 16);
  if (u >= turned) {  // a piece that stays
    const int c = rotary + 8 * (u - turned);
    for (int h = first; h < x.heads; h += step)
      *reinterpret_cast<uint4*>(out + h * x.out_head + c) = *reinterpret_cast<const uint4*>(in + h * x.in_head + c);
    return;
  }
  const int c0 = 8 * u, c1 = c0 + rotary / 2;
  float2 cs[N];
  load_cs<N>(row + N * u, wide, cs);
#pragma unroll
  for (int i = 0; i < N; ++i) cs[i].y *= sign;
  for (int h0 = first; h0 < x.heads; h0 += kBatch * step) {
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * step;
      if (h < x.heads) {
        a[i] = *reinterpret_cast<const uint4*>(in + h * x.in_head + c0);
        if (!INTERLEAVED) b[i] = *reinterpret_cast<const uint4*>(in + h * x.in_head + c1);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * step;
      if (h < x.heads) {
        float fa[8], fb[8], ga[8], gb[8];
        unpack8(a[i], fa);
        if (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < 4; ++j) turn(fa[2 * j], fa[2 * j + 1], cs[j], ga[2 * j], ga[2 * j + 1]);
        } else {
          unpack8(b[i], fb);
#pragma unroll
          for (int j = 0; j < 8; ++j) turn(fa[j], fb[j], cs[j], ga[j], gb[j]);
          *reinterpret_cast<uint4*>(out + h * x.out_head + c1) = pack8(gb);
        }
        *reinterpret_cast<uint4*>(out + h * x.out_head + c0) = pack8(ga);
      }
    }
  }
}

__device__ __forceinline__ void rope_pairs(const RopeDesc& r, const HeadsView& x, const uint16_t* in, uint16_t* out,
                                           const float2* row, float sign, int u, int first, int step) {
  const int half = r.rotary_dim / 2;
  if (u >= half) {
    const int c = r.rotary_dim + u - half;
    for (int h = first; h < x.heads; h += step) out[h * x.out_head + c] = in[h * x.in_head + c];
    return;
  }
  const int c0 = r.interleaved ? 2 * u : u, c1 = r.interleaved ? c0 + 1 : u + half;
  float2 cs = __ldg(row + u);
  cs.y *= sign;
  for (int h = first; h < x.heads; h += step) {
    const float a = __uint_as_float((uint32_t)in[h * x.in_head + c0] << 16);
    const float b = __uint_as_float((uint32_t)in[h * x.in_head + c1] << 16);
    float p, q;
    turn(a, b, cs, p, q);
    out[h * x.out_head + c0] = (uint16_t)f32_to_bf16_rn(p);
    out[h * x.out_head + c1] = (uint16_t)f32_to_bf16_rn(q);
  }
}

// Thread `i` of the rotation's: unit fastest, so that neighbouring lanes hold neighbouring pieces of a head, then
// `lanes` threads that take every lanes-th head, then the token.
__device__ __forceinline__ void rope_item(const RopeDesc& r, const HeadsView& x, const int32_t* positions, int64_t T,
                                          float sign, int units, int lanes, int64_t i, unsigned* err) {
  const unsigned per_token = (unsigned)units * (unsigned)lanes;
  const int64_t t = i <= UINT32_MAX ? (int64_t)((unsigned)i / per_token) : i / per_token;
  if (t >= T) return;
  const unsigned rem = (unsigned)(i - t * per_token);
  const int hl = (int)(rem / (unsigned)units), u = (int)(rem - (unsigned)hl * (unsigned)units);
  const int pos = __ldg(positions + t);
  if (pos < 0) return;  // a padding token
  if (pos >= r.positions) {
    if (rem == 0) record_error(err, kErrIndex);
    return;
  }
  const float2* row = r.table + (int64_t)pos * (r.rotary_dim / 2);
  const uint16_t* in = x.in + t * x.in_token;
  uint16_t* out = x.out + t * x.out_token;
  if (whole_pieces(r)) {
    const bool wide = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    if (r.interleaved)
      rope_pieces<true>(x, in, out, row, wide, sign, r.rotary_dim, u, hl, lanes);
    else
      rope_pieces<false>(x, in, out, row, wide, sign, r.rotary_dim, u, hl, lanes);
  } else {
    rope_pairs(r, x, in, out, row, sign, u, hl, lanes);
  }
}

constexpr int kRopeThreads = 128;

__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeDesc r, const HeadsView x,
                                                            const int32_t* __restrict__ positions, int64_t T, float sign,
                                                            int units, int lanes, unsigned* __restrict__ err) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  rope_item(r, x, positions, T, sign, units, lanes, (int64_t)blockIdx.x * kRopeThreads + threadIdx.x, err);
}

// ----------------------------------------------------------- kv_append_rope --
// The first blocks append, a thread a scale group as in kv_append: it reads its group and, of a K group, the channels
// that its own are paired with (which another thread of the same warp or its neighbour reads as its own: they
// come from L1), rotates in fp32, and applies the block rule to the fp32 values.  The blocks behind them rotate q.
// Channels [c0, c0 + 8) of a K head, rotated.
__device__ __forceinline__ void rotated8(const RopeDesc& r, const uint16_t* head, const float2* row, bool pieces, bool wide,
                                         int c0, float (&f)[8]) {
  const int half = r.rotary_dim / 2;
  unpack8(__ldg(reinterpret_cast<const uint4*>(head + c0)), f);
  if (c0 >= r.rotary_dim) return;
  if (pieces && r.interleaved) {
    float2 cs[4];
    load_cs<4>(row + c0 / 2, wide, cs);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float u, v;
      turn(f[2 * j], f[2 * j + 1], cs[j], u, v);
      f[2 * j] = u;
      f[2 * j + 1] = v;
    }
  } else if (pieces) {
    const bool first = c0 < half;
    float g[8];
    float2 cs[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(head + (first ? c0 + half : c0 - half))), g);
    load_cs<8>(row + (first ? c0 : c0 - half), wide, cs);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = first ? -cs[j].y : cs[j].y;  // a cos - b sin, or b cos + a sin
      f[j] = __fadd_rn(__fmul_rn(f[j], cs[j].x), __fmul_rn(g[j], s));
    }
  } else {
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + j;
      if (c >= r.rotary_dim) break;
      const bool first = r.interleaved ? !(c & 1) : c < half;
      const int i = r.interleaved ? c >> 1 : (first ? c : c - half);
      const int other = r.interleaved ? c ^ 1 : (first ? c + half : c - half);
      const float2 cs = __ldg(row + i);
      const float g = __uint_as_float((uint32_t)__ldg(head + other) << 16);
      f[j] = __fadd_rn(__fmul_rn(f[j], cs.x), __fmul_rn(g, first ? -cs.y : cs.y));
    }
  }
}

constexpr int kAppendThreads = 128;

template <int MODE>
__global__ void __launch_bounds__(kAppendThreads) kv_append_rope_kernel(
    const KvCacheDesc c, const RopeDesc r, const uint16_t* __restrict__ k, int64_t k_token, int64_t k_head,
    const uint16_t* __restrict__ v, int64_t v_token, int64_t v_head, const int64_t* __restrict__ slot_map,
    const int32_t* __restrict__ positions, int64_t T, const HeadsView q, int units, int lanes, unsigned append_blocks,
    unsigned* __restrict__ err) {
  constexpr int kGroup = MODE == 2 ? 16 : 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // k, v and q may come from the previous kernel
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x >= append_blocks) {
    rope_item(r, q, positions, T, 1.0f, units, lanes, (int64_t)(blockIdx.x - append_blocks) * kAppendThreads + threadIdx.x, err);
    return;
  }
  const unsigned groups = (unsigned)(c.head_dim / kGroup), per_token = groups * (unsigned)c.kv_heads * 2u;
  const int64_t idx = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
  const int64_t t = idx <= UINT32_MAX ? (int64_t)((unsigned)idx / per_token) : idx / per_token;
  if (t >= T) return;
  unsigned rem = (unsigned)(idx - t * per_token);
  const unsigned g = rem % groups;
  rem /= groups;
  const bool is_v = rem >= (unsigned)c.kv_heads;
  const unsigned h = is_v ? rem - (unsigned)c.kv_heads : rem;
  const int64_t slot = __ldg(slot_map + t);
  const int pos = __ldg(positions + t);
  if (slot < 0 || pos < 0) return;  // a padding token
  const int64_t page = (unsigned)slot / (unsigned)c.page_size;
  if (slot > INT32_MAX || page >= c.num_pages || pos >= r.positions) {
    if (rem == 0 && g == 0) record_error(err, kErrIndex);
    return;
  }
  const uint16_t* head = is_v ? v + t * v_token + h * v_head : k + t * k_token + h * k_head;
  const float2* row = r.table + (int64_t)pos * (r.rotary_dim / 2);
  const bool pieces = whole_pieces(r), wide = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
  float f[kGroup / 8][8];
  float b = 0.0f;
#pragma unroll
  for (int i = 0; i < kGroup / 8; ++i) {
    const int c0 = (int)g * kGroup + 8 * i;
    if (is_v)
      unpack8(__ldg(reinterpret_cast<const uint4*>(head + c0)), f[i]);
    else
      rotated8(r, head, row, pieces, wide, c0, f[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) b = fmaxf(b, fabsf(f[i][j]));
  }
  const float* gsp = is_v ? c.gs_v : c.gs_k;
  float mul;
  uint32_t sbyte;
  block_scale_rule_f32<MODE>(b, block_scale<MODE>(gsp), mul, sbyte);
  uint32_t words[kGroup / 8];
#pragma unroll
  for (int i = 0; i < kGroup / 8; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = __fmul_rn(f[i][j], mul);
    words[i] = e2m1x8_rn(f[i]);
  }
  const int64_t at = (page * c.kv_heads + h) * c.page_size + (slot - page * c.page_size);
  uint32_t* codes = (is_v ? c.v_codes : c.k_codes) + at * (c.head_dim / 8) + g * (kGroup / 8);
  if (MODE == 2)
    *reinterpret_cast<uint2*>(codes) = make_uint2(words[0], words[1]);
  else
    *reinterpret_cast<uint4*>(codes) = make_uint4(words[0], words[1], words[kGroup / 8 - 2], words[kGroup / 8 - 1]);
  (is_v ? c.v_scales : c.k_scales)[at * groups + g] = (uint8_t)sbyte;
}

// How many threads share a token's heads: one for every kBatch heads, as long as there are then threads enough for the
// GPU; else one a head.
int head_lanes(const DevInfo& d, int64_t T, int units, int heads) {
  const int some = (heads + kBatch - 1) / kBatch;
  return T * units * some >= (int64_t)d.sm_count * 1024 ? some : heads;
}

void pdl(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int64_t grid, int block, cudaStream_t s) {
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

int host_units(const RopeDesc& r, int dim, bool keep) {
  const int rest = keep ? dim - r.rotary_dim : 0;
  if (whole_pieces(r)) return r.rotary_dim / (r.interleaved ? 8 : 16) + rest / 8;
  return r.rotary_dim / 2 + rest;
}

}  // namespace

cudaError_t launch_rope_table(const DevInfo& d, const double* frequencies, int rotary_dim, double scale,
                              int64_t positions, float* table, cudaStream_t s) {
  // 1 / 2 pi in two parts, so that a frequency's fraction of a turn has all its 64 bits
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  RopeSteps steps = {};
  const int half = rotary_dim / 2;
  for (int i = 0; i < half; ++i) {
    const double f = frequencies[i], hi = f * kHi, lo = std::fma(f, kHi, -hi) + f * kLo;
    const double frac = hi - std::floor(hi);  // exact
    // (frac < 1, but may round to 1 where hi is a tiny negative number: then 2^64 is 0)
    const uint64_t top = frac >= 1.0 ? 0 : (uint64_t)std::ldexp(frac, 64);
    steps.step[i] = top + (uint64_t)(int64_t)std::ldexp(lo - std::floor(lo + 0.5), 64);
  }
  const int64_t entries = positions * half;
  const int64_t grid = std::min<int64_t>((entries + 255) / 256, (int64_t)d.sm_count * 16);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, grid, 256, s);
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, steps, half, scale, entries, reinterpret_cast<float2*>(table));
}

cudaError_t launch_rope(const DevInfo& d, const RopeDesc& r, const HeadsView& x, const int32_t* positions, int64_t T,
                        int backward, cudaStream_t s) {
  const int units = host_units(r, x.dim, x.in != x.out);
  const int lanes = head_lanes(d, T, units, x.heads);
  const int64_t grid = (T * units * lanes + kRopeThreads - 1) / kRopeThreads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, grid, kRopeThreads, s);
  return cudaLaunchKernelEx(&cfg, rope_kernel, r, x, positions, T, backward ? -1.0f : 1.0f, units, lanes, d.err);
}

cudaError_t launch_kv_append_rope(const DevInfo& d, const KvCacheDesc& c, const RopeDesc& r, const uint16_t* k,
                                  int64_t k_token, int64_t k_head, const uint16_t* v, int64_t v_token, int64_t v_head,
                                  const int64_t* slot_map, const int32_t* positions, int64_t T, const HeadsView& q,
                                  cudaStream_t s) {
  const int group = c.mode == FP4_MODE_NVFP4 ? 16 : 32;
  const int64_t append = (T * (int64_t)(c.head_dim / group) * c.kv_heads * 2 + kAppendThreads - 1) / kAppendThreads;
  int units = 0, lanes = 0;
  int64_t rotate = 0;
  if (q.heads > 0) {
    units = host_units(r, q.dim, q.in != q.out);
    lanes = head_lanes(d, T, units, q.heads);
    rotate = (T * units * lanes + kAppendThreads - 1) / kAppendThreads;
  }
  if (append + rotate > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, append + rotate, kAppendThreads, s);
  if (c.mode == FP4_MODE_NVFP4)
    return cudaLaunchKernelEx(&cfg, kv_append_rope_kernel<2>, c, r, k, k_token, k_head, v, v_token, v_head, slot_map,
                              positions, T, q, units, lanes, (unsigned)append, d.err);
  return cudaLaunchKernelEx(&cfg, kv_append_rope_kernel<1>, c, r, k, k_token, k_head, v, v_token, v_head, slot_map,
                            positions, T, q, units, lanes, (unsigned)append, d.err);
}

}  // namespace fp4
