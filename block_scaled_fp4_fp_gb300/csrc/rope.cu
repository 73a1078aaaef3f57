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
#include "packed.cuh"

namespace fp4 {
namespace {

// -------------------------------------------------------------- rope_table --
// An angle is position * frequency radians modulo a turn.  With the frequency as a 64-bit fraction of a turn (steps)
// the product modulo 2^64 is the angle itself, in units of 2^-64 of a turn, exact but for the fraction's own
// rounding times the position.  cos and sin in fp64, rounded once: the entries are those of the exact angle but for one in
// some million.  Runs once a model; bound by fp64: 131,072 positions of 64 pairs take 0.49 ms.
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

// n table entries from an 8-byte aligned address (16-byte where the address allows)
template <int N>
__device__ __forceinline__ void load_cs(const float2* p, float2 (&cs)[N]) {
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
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

__device__ __forceinline__ uint64_t pair_of(float lo, float hi) { return pair_of(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ uint64_t swapped(uint64_t v) { return pair_of((uint32_t)(v >> 32), (uint32_t)v); }
__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// Largest vector (8, 4 channels; 1: none) of which the rotated channels of a head are whole vectors and, in halves, a
// pair's two channels lie at the same place of two vectors.
__host__ __device__ inline int vector_of(const RopeDesc& r) {
  const int n = r.interleaved ? r.rotary_dim : r.rotary_dim / 2;
  return n % 8 == 0 ? 8 : n % 4 == 0 ? 4 : 1;
}

// -------------------------------------------------------------------- rope --
// What one thread does of a token's heads first, first + step, ..: unit `u` of each (no more of them than its batch:
// head_lanes).  A unit is two vectors of a head's halves, or an interleaved vector, then the vectors that stay as they
// are; its cosines are loaded once for all its heads, whose loads are all in flight.  Rotations that are no whole vectors
// (rotary/2 or, interleaved, rotary no multiple of 4) are done a pair at a time.  Whatever is written was read by the same
// thread before: in place is fine.
// Bound by HBM: 4096 tokens x 40 heads of 128 14.7 us in halves, 14.3 interleaved (5.9 and 6.0 TB/s); a quarter of heads of
// 96 in halves (vectors of four) 15.4 us, a pair at a time 108.
constexpr int kRopeBatchHalves = 4, kRopeBatchInterleaved = 8;

template <int N>
struct VecOf;
template <>
struct VecOf<8> {
  using T = uint4;
};
template <>
struct VecOf<4> {
  using T = uint2;
};

// The row of cosines of position `pos`; nullptr where the token is not to be written (padding, or past the table: reported)
__device__ __forceinline__ const float2* row_of(const RopeDesc& r, int pos, bool reports, unsigned* err) {
  if (pos < 0) return nullptr;
  if (pos >= r.positions) {
    if (reports) record_error(err, kErrIndex);
    return nullptr;
  }
  return r.table + (int64_t)pos * (r.rotary_dim / 2);
}

template <bool INTERLEAVED, int N>
__device__ __forceinline__ void rope_vectors(const RopeDesc& r, const HeadsView& x, const uint16_t* in, uint16_t* out, int pos,
                                             float sign, int u, int first, int step, unsigned* err) {
  using T = typename VecOf<N>::T;
  constexpr int NW = N / 2, B = INTERLEAVED ? kRopeBatchInterleaved : kRopeBatchHalves;  // words of a vector; heads, all in flight
  const int rotary = r.rotary_dim, turned = rotary / (INTERLEAVED ? N : 2 * N);
  const bool stays = u >= turned;
  const int c0 = stays ? rotary + N * (u - turned) : N * u, c1 = c0 + rotary / 2;
  // on their way while the position and its row are; past the last head its own first again (no branch a load: 4096 x 40 of 128
  // in halves 14.7 us, with one 15.4)
  T a[B], b[B];
#pragma unroll
  for (int i = 0; i < B; ++i) {
    const int h = first + i * step < x.heads ? first + i * step : first;
    a[i] = *reinterpret_cast<const T*>(in + h * x.in_head + c0);
    if (!INTERLEAVED && !stays) b[i] = *reinterpret_cast<const T*>(in + h * x.in_head + c1);
  }
  const float2* row = row_of(r, pos, u + first == 0, err);
  if (!row) return;
  uint64_t C[NW], S[NW];
  if (!stays) {
    float2 cs[INTERLEAVED ? NW : N];
    load_cs(row + (INTERLEAVED ? NW : N) * u, cs);
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      if (INTERLEAVED) {
        C[j] = pair_of(cs[j].x);
        S[j] = pair_of(-sign * cs[j].y, sign * cs[j].y);
      } else {
        C[j] = pair_of(cs[2 * j].x, cs[2 * j + 1].x);
        S[j] = pair_of(sign * cs[2 * j].y, sign * cs[2 * j + 1].y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < B; ++i) {
    const int h = first + i * step;
    if (h >= x.heads) break;
    T* o0 = reinterpret_cast<T*>(out + h * x.out_head + c0);
    T* o1 = reinterpret_cast<T*>(out + h * x.out_head + c1);
    if (stays) {
      *o0 = a[i];
      continue;
    }
    const uint32_t* aw = reinterpret_cast<const uint32_t*>(&a[i]);
    const uint32_t* bw = reinterpret_cast<const uint32_t*>(&b[i]);
    T ya, yb;
    uint32_t* yaw = reinterpret_cast<uint32_t*>(&ya);
    uint32_t* ybw = reinterpret_cast<uint32_t*>(&yb);
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const uint64_t p = widen(aw[j]);
      if (INTERLEAVED) {
        const uint64_t y = add2(mul2(p, C[j]), mul2(swapped(p), S[j]));
        yaw[j] = pack_bf16x2_rn(lo_of(y), hi_of(y));
      } else {
        const uint64_t q = widen(bw[j]), minus = pair_of(-lo_of(S[j]), -hi_of(S[j]));
        const uint64_t y0 = add2(mul2(p, C[j]), mul2(q, minus)), y1 = add2(mul2(q, C[j]), mul2(p, S[j]));
        yaw[j] = pack_bf16x2_rn(lo_of(y0), hi_of(y0));
        ybw[j] = pack_bf16x2_rn(lo_of(y1), hi_of(y1));
      }
    }
    *o0 = ya;
    if (!INTERLEAVED) *o1 = yb;
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
  const float2 cs = __ldg(row + u);
  const float sn = sign * cs.y;
  for (int h = first; h < x.heads; h += step) {
    const float a = bf16_at(in + h * x.in_head + c0), b = bf16_at(in + h * x.in_head + c1);
    out[h * x.out_head + c0] = (uint16_t)f32_to_bf16_rn(__fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, sn)));
    out[h * x.out_head + c1] = (uint16_t)f32_to_bf16_rn(__fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, sn)));
  }
}

// How a view is rotated: which of the above.  (kAny asks: for a kernel whose registers do not go by it.)
enum RopeKind { kHalves8, kInterleaved8, kHalves4, kInterleaved4, kByPairs, kAny };
__host__ __device__ inline RopeKind rope_kind(const RopeDesc& r) {
  const int n = vector_of(r);
  return n == 1 ? kByPairs : n == 8 ? (r.interleaved ? kInterleaved8 : kHalves8) : (r.interleaved ? kInterleaved4 : kHalves4);
}

// Thread `i` of the rotation's: unit fastest, so that neighbouring lanes hold neighbouring vectors of a head, then
// `lanes` threads that take every lanes-th head, then the token.
template <int KIND>
__device__ __forceinline__ void rope_item(const RopeDesc& r, const HeadsView& x, const int32_t* positions, int64_t T,
                                          float sign, int units, int lanes, int64_t i, unsigned* err) {
  const unsigned per_token = (unsigned)units * (unsigned)lanes;
  const int64_t t = i <= UINT32_MAX ? (int64_t)((unsigned)i / per_token) : i / per_token;
  if (t >= T) return;
  const unsigned rem = (unsigned)(i - t * per_token);
  const int hl = (int)(rem / (unsigned)units), u = (int)(rem - (unsigned)hl * (unsigned)units);
  const int pos = __ldg(positions + t);
  const uint16_t* in = x.in + t * x.in_token;
  uint16_t* out = x.out + t * x.out_token;
  switch (KIND == kAny ? rope_kind(r) : KIND) {
    case kHalves8: return rope_vectors<false, 8>(r, x, in, out, pos, sign, u, hl, lanes, err);
    case kInterleaved8: return rope_vectors<true, 8>(r, x, in, out, pos, sign, u, hl, lanes, err);
    case kHalves4: return rope_vectors<false, 4>(r, x, in, out, pos, sign, u, hl, lanes, err);
    case kInterleaved4: return rope_vectors<true, 4>(r, x, in, out, pos, sign, u, hl, lanes, err);
    default:
      if (const float2* row = row_of(r, pos, rem == 0, err)) rope_pairs(r, x, in, out, row, sign, u, hl, lanes);
  }
}

constexpr int kRopeThreads = 128;

template <int KIND>
__global__ void __launch_bounds__(kRopeThreads, 6) rope_kernel(const RopeDesc r, const HeadsView x,
                                                               const int32_t* __restrict__ positions, int64_t T, float sign,
                                                               int units, int lanes, unsigned* __restrict__ err) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  rope_item<KIND>(r, x, positions, T, sign, units, lanes, (int64_t)blockIdx.x * kRopeThreads + threadIdx.x, err);
}

// ----------------------------------------------------------- kv_append_rope --
// The first blocks append, the blocks behind them rotate q.  An appending thread has a unit of every lanes-th kv head
// of a token (kAppendBatch of them at most: head_lanes), of K and of V, its cosines loaded once for all its heads.  A unit is
//   kPairs   (halves of whole scale groups): two pieces of 8 channels of K's halves, which turn each other.  The lanes that
//            share two groups (2 of NVFP4, 4 of MXFP4) do the rule of one of them each and exchange multipliers;
//   kChunks  (interleaved): 16 channels of K;  both: 16 channels of V, and of K where it stays;
//   kPieces  (any other rotation): 8 channels; what they are paired with is read beside them.
// 17,500 tokens, 8 heads of 128: MXFP4 23 us, NVFP4 27 us, where the bytes take 15; with 32 query heads 62 and 67 us, 6.2
// and 5.8 TB/s.  A third of the SM's warps (80 registers) wait for loads; a scale group a thread, its partner read beside it,
// took 39 and 54 us, a piece a thread with the maximum shared by shuffles 47 and 64 (instructions).
constexpr int kAppendThreads = 128, kAppendBatch = 2;
enum AppendKind { kPairs, kChunks, kPieces };

// eight values' codes, their largest size
__device__ __forceinline__ uint32_t codes8(const uint64_t* f, float mul) {
  const uint64_t m2 = pair_of(mul);
  float y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t p = mul2(f[j], m2);
    y[2 * j] = lo_of(p);
    y[2 * j + 1] = hi_of(p);
  }
  return e2m1x8_rn(y);
}
__device__ __forceinline__ float largest8(const uint64_t* f) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max_abs3(m, lo_of(f[j]), hi_of(f[j]));
  return m;
}
__device__ __forceinline__ void widen8(uint4 v, uint64_t* f) {
  f[0] = widen(v.x);
  f[1] = widen(v.y);
  f[2] = widen(v.z);
  f[3] = widen(v.w);
}

// one cached row's codes and scales
struct CacheRow {
  uint32_t* codes;
  uint8_t* scales;
};

// 16 channels, the u-th of the row: a scale group of NVFP4, half of one of MXFP4 (the lane beside has the other)
template <int MODE>
__device__ __forceinline__ void store_chunk(const CacheRow& row, int u, const uint64_t (&f)[8], const BlockScale& rule,
                                            unsigned peers) {
  float m = fmaxf(largest8(f), largest8(f + 4)), mul;
  if (MODE == 1) m = fmaxf(m, __shfl_xor_sync(peers, m, 1));
  uint32_t sbyte;
  block_scale_rule_f32<MODE>(m, rule, mul, sbyte);
  reinterpret_cast<uint2*>(row.codes)[u] = make_uint2(codes8(f, mul), codes8(f + 4, mul));
  if (MODE == 2)
    row.scales[u] = (uint8_t)sbyte;
  else if (!(u & 1))
    row.scales[u >> 1] = (uint8_t)sbyte;
}

// pieces u and u + half / 8 of the row: lanes of even u do the rule of the first's group, of odd u of the second's
template <int MODE>
__device__ __forceinline__ void store_pair(const CacheRow& row, int u, int half, const uint64_t (&fa)[4],
                                           const uint64_t (&fb)[4], const BlockScale& rule, unsigned peers) {
  constexpr int G = MODE == 2 ? 16 : 32;
  const float ma = largest8(fa), mb = largest8(fb);
  const bool odd = u & 1;
  float m = fmaxf(odd ? mb : ma, __shfl_xor_sync(peers, odd ? ma : mb, 1)), mul;
  if (MODE == 1) m = fmaxf(m, __shfl_xor_sync(peers, m, 2));
  uint32_t sbyte;
  block_scale_rule_f32<MODE>(m, rule, mul, sbyte);
  const float other = __shfl_xor_sync(peers, mul, 1);
  row.codes[u] = codes8(fa, odd ? other : mul);
  row.codes[u + half / 8] = codes8(fb, odd ? mul : other);
  if (MODE == 2 || !(u & 2)) row.scales[(u * 8 + (odd ? half : 0)) / G] = (uint8_t)sbyte;
}

// How the channels [c0, c0 + 8) of a K head are turned: y = own C + other S
struct PieceTurn {
  enum Kind { kStays, kPartner, kSwap, kGather } kind;
  int c0, partner;  // the paired piece (kPartner)
  uint64_t C[4], S[4];

  __device__ __forceinline__ PieceTurn(const RopeDesc& r, const float2* row, int c) : kind(kStays), c0(c), partner(c) {
    if (c >= r.rotary_dim) return;
    const int half = r.rotary_dim / 2;
    if (vector_of(r) != 8) {
      kind = kGather;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float c2[2], s2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int ch = c0 + 2 * j + k;
          const bool first = r.interleaved ? k == 0 : ch < half;
          const float2 cs = ch < r.rotary_dim ? __ldg(row + (r.interleaved ? ch >> 1 : first ? ch : ch - half))
                                              : make_float2(1.0f, first ? 0.0f : -0.0f);
          c2[k] = cs.x;
          s2[k] = first ? -cs.y : cs.y;  // (a channel that stays: a 1 + 0 (-0), its zero's sign too)
        }
        C[j] = pair_of(c2[0], c2[1]);
        S[j] = pair_of(s2[0], s2[1]);
      }
    } else if (r.interleaved) {
      kind = kSwap;
      float2 cs[4];
      load_cs(row + c0 / 2, cs);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        C[j] = pair_of(cs[j].x);
        S[j] = pair_of(-cs[j].y, cs[j].y);
      }
    } else {
      kind = kPartner;
      const bool first = c0 < half;
      partner = first ? c0 + half : c0 - half;
      float2 cs[8];
      load_cs(row + (first ? c0 : c0 - half), cs);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        C[j] = pair_of(cs[2 * j].x, cs[2 * j + 1].x);
        S[j] = first ? pair_of(-cs[2 * j].y, -cs[2 * j + 1].y) : pair_of(cs[2 * j].y, cs[2 * j + 1].y);
      }
    }
  }
  // the channels that a head's own are paired with, where they are not its own
  __device__ __forceinline__ uint4 others(const RopeDesc& r, const uint16_t* head) const {
    if (kind == kPartner) return __ldg(reinterpret_cast<const uint4*>(head + partner));
    uint32_t w[4] = {0, 0, 0, 0};
    if (kind == kGather) {
      const int half = r.rotary_dim / 2;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int ch = c0 + j, at = r.interleaved ? ch ^ 1 : ch < half ? ch + half : ch - half;
        if (ch < r.rotary_dim) w[j >> 1] |= (uint32_t)__ldg(head + at) << (16 * (j & 1));
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void apply(uint64_t (&h)[4], uint4 other) const {
    if (kind == kStays) return;
    const uint32_t w[4] = {other.x, other.y, other.z, other.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = add2(mul2(h[j], C[j]), mul2(kind == kSwap ? swapped(h[j]) : widen(w[j]), S[j]));
  }
};

template <int MODE, int KIND>
__global__ void __launch_bounds__(kAppendThreads, 6) kv_append_rope_kernel(
    const KvCacheDesc c, const RopeDesc r, const uint16_t* __restrict__ k, int64_t k_token, int64_t k_head,
    const uint16_t* __restrict__ v, int64_t v_token, int64_t v_head, const int64_t* __restrict__ slot_map,
    const int32_t* __restrict__ positions, int64_t T, int append_lanes, const HeadsView q, int units, int lanes,
    unsigned append_blocks, unsigned* __restrict__ err) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // k, v and q may come from the previous kernel
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x >= append_blocks) {
    constexpr int kind = KIND == kPairs ? kHalves8 : KIND == kChunks ? kInterleaved8 : kAny;  // (whole groups are whole vectors)
    rope_item<kind>(r, q, positions, T, 1.0f, units, lanes, (int64_t)(blockIdx.x - append_blocks) * kAppendThreads + threadIdx.x, err);
    return;
  }
  constexpr int kUnit = KIND == kPieces ? 8 : 16;  // channels
  const unsigned U = (unsigned)c.head_dim / kUnit, per_token = U * (unsigned)append_lanes;
  const int64_t idx = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
  const int64_t t = idx <= UINT32_MAX ? (int64_t)((unsigned)idx / per_token) : idx / per_token;
  if (t >= T) return;
  const unsigned rem = (unsigned)(idx - t * per_token);
  const int hl = (int)(rem / U), u = (int)(rem - (unsigned)hl * U);
  const int64_t slot = __ldg(slot_map + t);
  const int pos = __ldg(positions + t);
  const int heads = c.kv_heads, half = r.rotary_dim / 2;
  const uint16_t* kt = k + t * k_token;
  const uint16_t* vt = v + t * v_token;
  // the heads' loads are on their way while the slot, the position and its row are
  const bool turned = KIND != kPieces && u < r.rotary_dim / 16;
  const int p0 = KIND == kPieces || (KIND == kPairs && turned) ? u : 2 * u;  // K's pieces
  const int p1 = KIND == kPairs && turned ? u + half / 8 : 2 * u + 1;
  uint4 ka[kAppendBatch][2], va[kAppendBatch][2];
#pragma unroll
  for (int i = 0; i < kAppendBatch; ++i) {
    const int h = hl + i * append_lanes;
    if (h >= heads) continue;
    const uint4* kh = reinterpret_cast<const uint4*>(kt + h * k_head);
    const uint4* vh = reinterpret_cast<const uint4*>(vt + h * v_head);
    ka[i][0] = __ldg(kh + p0);
    va[i][0] = __ldg(vh + (KIND == kPieces ? u : 2 * u));
    if (KIND != kPieces) {
      ka[i][1] = __ldg(kh + p1);
      va[i][1] = __ldg(vh + 2 * u + 1);
    }
  }
  if (slot < 0 || pos < 0) return;  // a padding token
  const unsigned page = (unsigned)slot / (unsigned)c.page_size;
  if (slot > INT32_MAX || page >= c.num_pages || pos >= r.positions) {
    if (rem == 0) record_error(err, kErrIndex);
    return;
  }
  const float2* row = r.table + (int64_t)pos * half;
  const BlockScale rule_k = block_scale<MODE>(c.gs_k), rule_v = block_scale<MODE>(c.gs_v);
  // (num_pages * kv_heads * page_size < 2^31)
  const int at0 = (int)page * heads * c.page_size + (int)((unsigned)slot - page * (unsigned)c.page_size);
  const int words = c.head_dim / 8, groups = c.head_dim / (MODE == 2 ? 16 : 32);
  auto cached = [&](uint32_t* codes, uint8_t* scales, int h) {
    const int64_t at = at0 + h * c.page_size;
    return CacheRow{codes + at * words, scales + at * groups};
  };
  // (the lanes that share a group are neighbours with the same token and heads: they come to its exchange together)
  constexpr int kLanes = MODE == 2 ? 2 : 4;
  const unsigned peers = ((1u << kLanes) - 1) << ((threadIdx.x & 31) & ~(kLanes - 1));
  if constexpr (KIND == kPieces) {
    const PieceTurn turn(r, row, 8 * u);
    uint4 other[kAppendBatch];
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i)
      if (const int h = hl + i * append_lanes; h < heads) other[i] = turn.others(r, kt + h * k_head);
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      const int h = hl + i * append_lanes;
      if (h >= heads) continue;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint64_t f[4];
        widen8(which ? va[i][0] : ka[i][0], f);
        if (!which) turn.apply(f, other[i]);
        float m = largest8(f), mul;
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(peers, m, o));
        uint32_t sbyte;
        block_scale_rule_f32<MODE>(m, which ? rule_v : rule_k, mul, sbyte);
        const CacheRow to = which ? cached(c.v_codes, c.v_scales, h) : cached(c.k_codes, c.k_scales, h);
        to.codes[u] = codes8(f, mul);
        if (u % kLanes == 0) to.scales[u / kLanes] = (uint8_t)sbyte;
      }
    }
  } else {
    const unsigned two = 3u << ((threadIdx.x & 31) & ~1);
    float2 cs[8];
    uint64_t C[4], S[4], M[4];
    if (turned) {
      load_cs(row + 8 * u, cs);
      if (KIND == kPairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          C[j] = pair_of(cs[2 * j].x, cs[2 * j + 1].x);
          S[j] = pair_of(cs[2 * j].y, cs[2 * j + 1].y);
          M[j] = pair_of(-cs[2 * j].y, -cs[2 * j + 1].y);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      const int h = hl + i * append_lanes;
      if (h >= heads) continue;
      const CacheRow to = cached(c.k_codes, c.k_scales, h);
      uint64_t f[8];
      widen8(ka[i][0], f);
      widen8(ka[i][1], f + 4);
      if (KIND == kPairs && turned) {
        uint64_t fa[4], fb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          fa[j] = add2(mul2(f[j], C[j]), mul2(f[4 + j], M[j]));
          fb[j] = add2(mul2(f[4 + j], C[j]), mul2(f[j], S[j]));
        }
        store_pair<MODE>(to, u, half, fa, fb, rule_k, peers);
      } else {
        if (turned) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            f[j] = add2(mul2(f[j], pair_of(cs[j].x)), mul2(swapped(f[j]), pair_of(-cs[j].y, cs[j].y)));
        }
        store_chunk<MODE>(to, u, f, rule_k, two);
      }
      widen8(va[i][0], f);
      widen8(va[i][1], f + 4);
      store_chunk<MODE>(cached(c.v_codes, c.v_scales, h), u, f, rule_v, two);
    }
  }
}

// The kind of append: see kv_append_rope_kernel.  (A warp holds whole groups of four units where a head has them.)
AppendKind append_kind(const KvCacheDesc& c, const RopeDesc& r) {
  const int group = c.mode == FP4_MODE_NVFP4 ? 16 : 32;
  if (r.interleaved) return r.rotary_dim % 16 == 0 ? kChunks : kPieces;
  return r.rotary_dim / 2 % group == 0 && c.head_dim % (2 * group) == 0 ? kPairs : kPieces;
}

// How many threads share a token's heads: one for every `batch` heads, which is what a thread takes at most (in vectors), where
// there are then threads enough for the GPU, up to one a head where there are not (1001 tokens x 64 heads of 64: 5 us, with
// one a head 11).
int head_lanes(const DevInfo& d, int64_t T, int units, int heads, int batch) {
  const int64_t some = (heads + batch - 1) / batch, wanted = (int64_t)d.sm_count * 512 / (T * units);
  return (int)std::max<int64_t>(some, std::min<int64_t>(heads, wanted));
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

// units of a head that the rotation of a view is made of (rope_item), and the threads that share a token's heads
void rope_shape(const DevInfo& d, const RopeDesc& r, const HeadsView& x, int64_t T, int& units, int& lanes) {
  const int rest = x.in != x.out ? x.dim - r.rotary_dim : 0, n = vector_of(r);
  units = n == 1 ? r.rotary_dim / 2 + rest : r.rotary_dim / (r.interleaved ? n : 2 * n) + rest / n;
  lanes = head_lanes(d, T, units, x.heads, r.interleaved ? kRopeBatchInterleaved : kRopeBatchHalves);
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
  int units, lanes;
  rope_shape(d, r, x, T, units, lanes);
  const int64_t grid = (T * units * lanes + kRopeThreads - 1) / kRopeThreads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, grid, kRopeThreads, s);
  auto go = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, r, x, positions, T, backward ? -1.0f : 1.0f, units, lanes, d.err);
  };
  switch (rope_kind(r)) {
    case kHalves8: return go(rope_kernel<kHalves8>);
    case kInterleaved8: return go(rope_kernel<kInterleaved8>);
    case kHalves4: return go(rope_kernel<kHalves4>);
    case kInterleaved4: return go(rope_kernel<kInterleaved4>);
    default: return go(rope_kernel<kByPairs>);
  }
}

cudaError_t launch_kv_append_rope(const DevInfo& d, const KvCacheDesc& c, const RopeDesc& r, const uint16_t* k,
                                  int64_t k_token, int64_t k_head, const uint16_t* v, int64_t v_token, int64_t v_head,
                                  const int64_t* slot_map, const int32_t* positions, int64_t T, const HeadsView& q,
                                  cudaStream_t s) {
  const AppendKind kind = append_kind(c, r);
  const int per_head = c.head_dim / (kind == kPieces ? 8 : 16);
  const int append_lanes = head_lanes(d, T, per_head, c.kv_heads, kAppendBatch);
  const int64_t append = (T * per_head * append_lanes + kAppendThreads - 1) / kAppendThreads;
  int units = 0, lanes = 0;
  int64_t rotate = 0;
  if (q.heads > 0) {
    rope_shape(d, r, q, T, units, lanes);
    rotate = (T * units * lanes + kAppendThreads - 1) / kAppendThreads;
  }
  if (append + rotate > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, append + rotate, kAppendThreads, s);
  auto go = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, c, r, k, k_token, k_head, v, v_token, v_head, slot_map, positions, T,
                              append_lanes, q, units, lanes, (unsigned)append, d.err);
  };
  if (c.mode == FP4_MODE_NVFP4)
    return kind == kPairs    ? go(kv_append_rope_kernel<2, kPairs>)
           : kind == kChunks ? go(kv_append_rope_kernel<2, kChunks>)
                             : go(kv_append_rope_kernel<2, kPieces>);
  return kind == kPairs    ? go(kv_append_rope_kernel<1, kPairs>)
         : kind == kChunks ? go(kv_append_rope_kernel<1, kChunks>)
                           : go(kv_append_rope_kernel<1, kPieces>);
}

}  // namespace fp4
