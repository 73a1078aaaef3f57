// kv_decode.cu -- attention of a few query rows over the paged 4-bit cache: the
// serving form for single tokens (and for a handful of tokens a request), where the
// cache is read once and its bytes are the work.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(s_rj - m_r),   s_rj = c_r q_r . k_j
// with c_r = softmax_scale log2(e) gs_k, over the keys j that row r may see.  A row r is
// one (query token, head of the kv head's group); R = 8 NB rows share a pass over
// the keys of their kv head.
//
// Scores on the 5th-generation tensor cores, K never dequantized: a tile of 128
// keys is the block-scaled FP4 A operand of tcgen05.mma.kind::mxf4nvf4 (one key per
// accumulator lane, its E4M3/E8M0 scales applied by the hardware), and the R query
// rows are the B operand, each written as kTerms = 8 FP4 terms in radix 8,
//     q = 2^e0 (sum_t d_t 2^(6-3t) + rest),  d_t in {-4..4},  max|q| / 2^e0 in [128, 256),
// exact but for |rest| <= 2^-16, 2^-23 of the row's largest element, fp32's own precision of it.
// (With six, 2^-17, a channel of q a thousand times its others moved scores by 0.05.)
// Terms t and t + 3, t < 3, of row r add up in column t R + r, terms 6 and 7 in column 3 R + r,
// in units of 2^-18 (E4M3 has no scale small enough for them): two MMAs a step of 64 channels,
// ~143 cycles each whatever N is.  The thread that owns a key sums a row's four columns in
// registers: no score crosses a lane.  (A column a term and one MMA cost the consumers 27 more
// instructions per 32 keys and eight rows; one column and an MMA a term would take the tensor
// cores longer than the tile's DRAM time.)  Dequantizing K instead would cost an instruction stream as long as
// V's, the larger half of what the SM issues.
//
// Values in registers: a warp owns 32 keys of the tile (its tensor-memory lane
// quadrant) from scores to output.  V's codes come from shared memory in the
// m16n8k16 A-fragment order (channels as rows, keys as columns: neighbouring keys'
// codes are merged into bytes by one LOP3 and become f16 pairs by the hardware's
// e2m1x2 converter, times their scales: exact in f16), the probabilities go through
// 512 bytes of shared memory and ldmatrix.trans, and the mma.sync sums stay in
// registers.  (tcgen05 would want V as 16-bit shared-memory tiles: 512 bytes of
// shared memory traffic a key more, which alone is as long as the key's DRAM time.)
// With up to sixteen rows (NB = 2) a warp takes both blocks of eight in turn and dequantizes V once for
// them; more rows are more passes over the cache, the later ones out of L2.  (Four blocks a
// pass, with a quadrant's softmax and channels split over four warps that meet in a barrier each
// tile, was slower than two passes: 100 us against 72 for 16 requests x 4 tokens x 8 heads a group.)
// Every quadrant of every group keeps its own running reference m, sum and output:
// they meet only at the end of a (request, kv head).
//
// Range.  p = 2^(s - m) is rounded to f16 (2^-11, while p is at least 2^-14; 2^-8, as in bf16, at 2^-17, where f16 is
// subnormal).  m is set kHead below the largest score and moves only when a score passes it by kMax,
// so that p stays below f16's largest value.  A warp whose tile holds a p below 2^-kTiny (not zero: down to
// 2^-126) multiplies that tile in bf16 instead: codes to bf16 by shifts and masks (twice the
// instructions of the converter), p with bf16's range.  Sharp score distributions pay this; every p counts with
// eight bits in either, also where V is zero at the keys of the large ones.  (64 requests x 8,000, 16 rows a head:
// 192 us; 197 with a reference one power of two higher and the bound at 2^-16, 193 with that and 2^-23.)
// MXFP4's E8M0 scales have the range of fp32, f16 has not: a thread's V values are
// held relative to 2^E, E the largest scale exponent so far of the channel group it owns;
// a tile with scales 2^20 below it takes the bf16 form too.
//
// Work split.  The tiles of all (request, kv head, row block) are dealt out evenly
// to the CTAs (one an SM) as one sequence (the lengths are on the device: every CTA
// sums them itself).  A piece that does not cover its (request, kv head) leaves
// (m, l, o) in the workspace; the last CTA to arrive there joins the pieces in
// order, so the result does not depend on who is last.
//
//   consumers   kGroups groups of four warps; group g takes the CTA's tiles i with i % kGroups == g
//   then one warp each:
//   K, V        a tile's codes (swizzled by the row's length) and scales by cp.async into a ring each, pages looked
//               up a tile ahead.  (A TMA box or bulk copy costs its thread ~140 cycles to issue, and a tile of
//               16-slot pages takes 32 of them: as long as the tile's DRAM time.)
//   MMA         moves a tile's K scales into the 32x16-byte order tcgen05.cp reads, issues that copy and the MMAs
//   queries     query rows as FP4 terms, one segment ahead
//
// Bound by HBM: 2 D (1/2 + 1/g) bytes a key and kv head.  Of the 96 requests below the tiles take 225 of 268 us (473 ns
// each; their bytes take 410; issue active 53 %, no unit near its limit), the rest are the items' ends (about 4 us each,
// five a CTA) and the chain of plan, first queries, first tiles and joins (about 10 us), which is what one request
// pays.  Measured, heads of 128:
//   96 requests of 4k..20k, 40 query heads on 8, MXFP4    268 us, 4.7 TB/s
//   32 requests of 1..8k, 64 on 8, NVFP4                   46 us, 3.3 TB/s
//   1 request of 131k, 64 on 8, NVFP4                      40 us, 3.8 TB/s
//   16 requests x 4 tokens, 64 on 8, NVFP4                 65 us (two passes; a pass costs its instructions)
//   1 request of 997, 40 on 40, NVFP4                      11 us
#include <algorithm>
#include <type_traits>

#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "kv_common.cuh"
#include "kv_split.h"
#include "launch.h"

namespace fp4 {
namespace {

constexpr int kTerms = 8;
constexpr int kCols = 4;                 // score columns of a row
constexpr int kChains = kTerms / kCols;  // terms added into each
constexpr float kLastUnit = 0x1p-18f;    // unit of the last column
// term of chain ch in column c
__host__ __device__ constexpr int term_of(int ch, int c) { return c < 3 ? 3 * ch + c : 6 + ch; }
constexpr int kTile = 128;  // keys per tile: the MMA's M
constexpr int kMaxStages = 12;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHead = 8.0f;   // a new reference m is the largest score less this (log2)
constexpr float kMax = 15.0f;   // and moves when a score passes it by this: p <= 2^15
constexpr float kTiny = 17.0f;  // scores further below m than this need bf16's range
constexpr float kNone = -1e30f; // m before any score: exp2 of a hidden key's -inf less this is 0, of this less a score too

template <int MODE, int D, int NB>
struct Dec {
  static constexpr int kR = 8 * NB;                          // query rows
  static constexpr int kN = (kCols * kR + 15) / 16 * 16;     // MMA N (rows past kCols kR feed columns nothing reads)
  static constexpr int kGroup = MODE == 2 ? 16 : 32;
  static constexpr int kSB = D / kGroup;                     // scale bytes of a row
  static constexpr int kWords = kSB < 4 ? 1 : kSB / 4;       // and its 32-bit words
  static constexpr int kRowB = D / 2;                        // code bytes of a row
  static constexpr uint32_t kSwz = D == 64 ? 0x10 : D == 128 ? 0x30 : 0x70;
  static constexpr uint32_t kCodes = kTile * kRowB;
  static constexpr uint32_t kScales = kTile * kSB;
  // consumer warps: as many as their output fragments (D NB / 4 registers a thread) leave registers for
  static constexpr int kWarps = D * NB <= 128 ? 12 : 8;
  static constexpr int kGroups = kWarps / 4;
  static constexpr int kBufs = kGroups < 2 ? 2 : kGroups;    // score buffers
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kThreads = kConsumers + 128;
  static constexpr int kCh = D / 8;                     // channels of a consumer thread
  static constexpr int kPieces = D * NB / 8;                 // float2 of its output
  static constexpr uint32_t kQChain = (kN * kRowB + 1023) / 1024 * 1024;
  static constexpr uint32_t kQBytes = kChains * kQChain;
  static constexpr int kSStride = (kN + 31) / 32 * 32;       // tensor-memory columns between score buffers
  static constexpr uint32_t kSfa = kBufs * kSStride;         // K scales, kBufs buffers of 16 columns
  static constexpr uint32_t kSfb = kSfa + 16 * kBufs;        // term scales, 4 columns a chain
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSfb + 4 * kChains <= kTmemCols && kN <= 128, "tensor memory");
  // shared memory: [K codes][V codes][queries x 2][K scales as tcgen05.cp reads them][outputs of half the sets]
  // [probabilities][K scales][V scales][row data][barriers]
  static constexpr int kSets = kGroups * 4;                  // quadrants with their own m, l, output
  static constexpr uint32_t kSfaBytes = kWords * 512;
  static constexpr uint32_t kOutBytes = kWarps / 2 * kPieces * 32 * 8;
  static constexpr uint32_t kPBytes = kSets * NB * 512;
  // score factors, key ranges and output rows x 2, m, -m and l of the sets, joined m and l, factors of moved
  // references, segments x 2
  static constexpr uint32_t kRowBytes =
      2 * 3 * kR * 4 + 2 * kR * 16 + kSets * kR * 12 + 2 * kR * 4 + kSets * kR * 4 + 80;  // (a multiple of 8)
  static constexpr uint32_t kFixed =
      2 * kQBytes + kBufs * kSfaBytes + kOutBytes + kPBytes + kRowBytes + 1024 + 1024;
  static constexpr uint32_t kBudget = 226u * 1024u;
  // Two rings: a K tile is read once its scores are issued, a V tile is held until its group is through
  // with it, so of the tiles that fit V gets more.
  static constexpr int kFit = (int)((kBudget - kFixed) / (kCodes + kScales));
  static constexpr int kStK0 = (kFit - kGroups + 1) / 2, kStK = kStK0 > kMaxStages ? kMaxStages : kStK0;
  static constexpr int kStV0 = kFit - kStK, kStV = kStV0 > kMaxStages ? kMaxStages : kStV0;
  static constexpr uint32_t kSmem = kFixed + (kStK + kStV) * (kCodes + kScales);
  static_assert(kStK >= 2 && kStV >= 2 && kSmem <= kBudget, "shared memory");
  // a group's parity wait on a stage must not be two phases ahead of it
  static_assert(kStV >= kGroups, "the V ring holds a tile of every group");
  // What an item costs a CTA besides its tiles, in tiles: starting on new queries, draining the groups, joining the
  // sets and writing the rows take about 4 us, a tile 0.4 to 1.8 us (measured).  Counted when the work is
  // dealt out, so that a CTA with many short requests does not finish last.
  static constexpr int kItemCost = NB == 1 ? 8 : 5;
  static constexpr int kSlot = kR * D + 2 * kR;              // floats of a workspace piece (output, m, l)
};

// byte of the term scale 2^(7-3t), of terms 6 and 7 times 2^18 (see the FP4 GEMV's terms: exact in both formats)
template <int MODE>
__device__ __forceinline__ uint32_t term_scale(int t) {
  const int e = 7 - 3 * (t < 6 ? t : t - 6);
  if (MODE == 1) return (uint32_t)(127 + e);
  return e >= -6 ? (uint32_t)((e + 7) << 3) : (1u << (e + 9));
}

// four bytes of two e2m1 codes -> four f16 pairs
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// e2m1 code I (0..3) of each 16-bit half -> bf16 pair of the code's value times 2^-126: sign to bit 15, the
// exponent and mantissa bits to the lowest exponent bits and the highest mantissa bit (code 1 is subnormal there too)
template <int I>
__device__ __forceinline__ uint32_t e2m1_to_bf16(uint32_t n) {
  const uint32_t sign = I == 3 ? n : n << (12 - 4 * I);
  const uint32_t mag = I <= 1 ? n << (6 - 4 * I) : n >> (4 * I - 6);
  return (sign & 0x80008000u) | (mag & 0x01C001C0u);
}
// two f16 -> two bf16, times 2^8
__device__ __forceinline__ uint32_t f16x2_to_bf16x2_256(uint32_t h) {
  return pack_bf16x2_rn(f16_lo_to_f32(h) * 256.0f, f16_hi_to_f32(h) * 256.0f);
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
// shared-memory reads by 32-bit address
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint32_t v;
  asm volatile("{\n\t.reg .b16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void named_sync(int id) { asm volatile("bar.sync %0, %1;" :: "r"(id), "n"(N) : "memory"); }

// The keys of a thread's fragment column pair c, of the slab's 16: base(c) + offset(i), i = 0..3
// (columns 2c, 2c + 1, 2c + 8, 2c + 9).  Any order serves as long as the probabilities
// follow it; these make a warp's V loads touch every bank once per phase under the
// row's swizzle.
template <int D>
__device__ __forceinline__ int key_of(int c, int i) {
  if (D == 64) return c + 4 * i;
  if (D == 128) return (c & 1) + 4 * (c >> 1) + ((i & 1) << 1) + ((i >> 1) << 3);
  return 2 * c + (i & 1) + ((i >> 1) << 3);
}

// One request as this kernel deals it out.
struct Req {
  int q0, qlen, total, first;  // first token row, query count, keys, first visible key
  int tiles, lo_tile, blocks;  // tiles per pass, first tile, row blocks
  int cost;                    // units of an item: its tiles, and the fixed cost
  __device__ __forceinline__ int64_t units(int kv_heads) const {
    return tiles > 0 ? (int64_t)cost * blocks * kv_heads : 0;
  }
};

__device__ __forceinline__ Req load_req(const KvAttentionArgs& a, int b, int group, int R, int item_cost) {
  Req r;
  r.q0 = __ldg(a.query_start + b);
  r.qlen = __ldg(a.query_start + b + 1) - r.q0;
  r.total = __ldg(a.total_lens + b);
  r.total = max(min(r.total, a.max_pages * a.cache.page_size), 0);
  if (r.qlen > a.max_query_len || r.q0 < 0 || (int64_t)r.q0 + r.qlen > a.tokens) r.qlen = 0;
  r.first = a.window > 0 ? max(0, r.total - r.qlen + 1 - a.window) : 0;
  r.lo_tile = r.first / kTile;
  r.blocks = r.qlen > 0 ? (int)((unsigned)(r.qlen * group + R - 1) / (unsigned)R) : 0;
  r.tiles = r.total > 0 && r.qlen > 0 ? (r.total + kTile - 1) / kTile - r.lo_tile : 0;
  r.cost = r.tiles + item_cost;
  return r;
}

// A CTA's walk over its share of the sequence: request by request, in it kv head by kv head, in it row block
// by row block; each of these items is its tiles and then some units that hold no work.
struct Walk {
  const KvAttentionArgs* a;
  int group, R, item_cost, b, item, off;
  int64_t at, end;  // position in the sequence
  Req r;
  // the current segment
  int h, rb, ta, tb;
  int64_t start;  // where the item's tile 0 sits in the sequence
  __device__ __forceinline__ void begin(const KvAttentionArgs& args, int g, int rows, int fixed, int b0, int item0,
                                        int off0, int64_t f0, int64_t f1) {
    a = &args;
    group = g;
    R = rows;
    item_cost = fixed;
    b = b0;
    at = f0;
    end = f1;
    item = item0;
    off = off0;
    r = load_req(args, b, group, R, item_cost);
  }
  __device__ __forceinline__ bool next() {
    for (;;) {
      if (at >= end) return false;
      while (r.tiles == 0 || item == a->cache.kv_heads * r.blocks) {
        if (++b >= a->batch) return false;
        r = load_req(*a, b, group, R, item_cost);
        item = 0;
      }
      h = item / r.blocks;
      rb = item - h * r.blocks;
      start = at - off;
      const int to = (int)min((int64_t)r.cost, off + (end - at));
      ta = min(off, r.tiles);
      tb = min(to, r.tiles);
      at += to - off;
      off = 0;
      ++item;
      if (ta < tb) return true;
    }
  }
};

// A segment as the query warp hands it to the MMA warp and the consumers (in shared memory).
struct Seg {
  int ta, tb;                  // ta = tb: the CTA's share is done
  int total, first;            // the request's
  int lo_tile, tiles, lo_max, hi_min;
  int64_t start;  // where the item's tile 0 sits in the sequence
};

// |v| < 256 -> v's eight radix-8 digits in -4..4 as e2m1 codes of half of each, the lowest, of 2^-15, in the lowest nibble.
// With four added to every digit they are three bits each (the highest four) of an integer; spread to a nibble each,
// a digit below 4 (u) is the code of -(4 - u), one from 4 on that of u - 4.
__device__ __forceinline__ uint32_t radix8_codes(float v) {
  uint32_t w = (uint32_t)__float2int_rn(v * 32768.0f) + 04444'4444u;
  w = (w & 0xFFFu) | ((w & 0x1FFF000u) << 4);
  w = (w & 0x003F003Fu) | ((w & 0x1FC00FC0u) << 2);
  w = (w & 0x07070707u) | ((w & 0x78383838u) << 1);
  const uint32_t below = ~((w >> 2) | (w >> 3)) & 0x11111111u;  // 4 - u = (u ^ 3) + 1; 8 for the sign
  return ((w & 0x33333333u) ^ (3u * below)) + 9u * below + ((w >> 1) & 0x40000000u);
}

// Query rows r0 .. r0 + N - 1 of a segment as FP4 terms in the B operands' order (a warp): term term_of(ch, c) of row r is
// row c R + r of chain ch.  Writes each row's score factor.
template <int MODE, int D, int NB, int N>
__device__ __forceinline__ void query_rows(const KvAttentionArgs& a, uint8_t* dst, const int64_t* row_q, float* row_c,
                                           int r0, int lane) {
  using C = Dec<MODE, D, NB>;
  constexpr int EL = D / 32;  // elements of a lane
  uint32_t x[N][EL / 2];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int64_t at = row_q[r0 + k];
    const uint16_t* src = a.q + at + lane * EL;
#pragma unroll
    for (int e = 0; e < EL / 2; ++e) x[k][e] = at >= 0 ? __ldg(reinterpret_cast<const uint32_t*>(src) + e) : 0u;
  }
  const float mult = a.scale * kLog2e * ((MODE == 2 && a.cache.gs_k) ? __ldg(a.cache.gs_k) : 1.0f);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t mb = 0;
#pragma unroll
    for (int e = 0; e < EL / 2; ++e) mb = __vmaxu2(mb, x[k][e] & 0x7FFF7FFFu);
    mb = __reduce_max_sync(0xffffffffu, max(mb & 0xFFFFu, mb >> 16));
    // 2^e0 = the largest element's power of two / 128 (2^-127 at least); a NaN or infinity makes every score NaN
    const uint32_t E = max(mb >> 7, 7u);
    const float pre = __uint_as_float((261u - min(E, 254u)) << 23);  // 2^-e0, e0 = E - 134
    if (lane == 0)
      row_c[r0 + k] = mb < 0x7F80u ? mult * (E >= 8u ? __uint_as_float((E - 7u) << 23) : 0x1p-127f) : __int_as_float(0x7FC00000);
    uint32_t even[EL / 2], odd[EL / 2];  // digits 0, 2, 4, 6 and 1, 3, 5, 7 of a pair of elements, a byte each
#pragma unroll
    for (int e = 0; e < EL / 2; ++e) {
      const uint32_t d0 = radix8_codes(bf16_lo(x[k][e]) * pre), d1 = radix8_codes(bf16_hi(x[k][e]) * pre);
      even[e] = (d0 & 0x0F0F0F0Fu) | ((d1 << 4) & 0xF0F0F0F0u);
      odd[e] = ((d0 >> 4) & 0x0F0F0F0Fu) | (d1 & 0xF0F0F0F0u);
    }
    const uint32_t at = (uint32_t)((r0 + k) * C::kRowB + lane * (EL / 2));
    uint8_t* row = dst + (at ^ ((at >> 3) & C::kSwz));
    static_assert(((C::kR * C::kRowB) & (C::kSwz << 3 | ((C::kSwz << 3) - 1))) == 0, "a column starts at the same place of the swizzle");
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      const int i = (7 - t) >> 1;  // term t is digit 7 - t
      const uint32_t* by = t & 1 ? even : odd;
      uint8_t* to = row + (t < 6 ? t % 3 : 3) * (C::kR * C::kRowB) + (t < 6 ? t / 3 : t - 6) * C::kQChain;
      const uint32_t two = __byte_perm(by[0], by[1 % (EL / 2)], i | (i + 4) << 4);
      if (EL == 2) *to = (uint8_t)(by[0] >> (8 * i));
      else if (EL == 4) *reinterpret_cast<uint16_t*>(to) = (uint16_t)two;
      else *reinterpret_cast<uint32_t*>(to) = __byte_perm(two, __byte_perm(by[2 % (EL / 2)], by[3 % (EL / 2)], i | (i + 4) << 4), 0x5410);
    }
  }
}

template <int MODE, int D, int NB>
__global__ void __launch_bounds__((Dec<MODE, D, NB>::kThreads), 1) kv_decode_kernel(
    const KvAttentionArgs a, int group, int* __restrict__ arrivals, float* __restrict__ pieces, int inject_timeout) {
  using C = Dec<MODE, D, NB>;
  constexpr int R = C::kR, SK = C::kStK, SV = C::kStV, BUFS = C::kBufs, SETS = C::kSets;
  constexpr int kThreads = C::kThreads, kConsumers = C::kConsumers;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  constexpr uint32_t offV = SK * C::kCodes, offQ = offV + SV * C::kCodes, offSfa = offQ + 2 * C::kQBytes, offOut = offSfa + BUFS * C::kSfaBytes,
                     offP = offOut + C::kOutBytes, offS = offP + C::kPBytes, offSv = offS + SK * C::kScales, offRow = offSv + SV * C::kScales,
                     offBar = (offRow + C::kRowBytes + 7) / 8 * 8;
  float* row_c = reinterpret_cast<float*>(smem + offRow);         // [2][R] score factor of a row
  int* row_lo = reinterpret_cast<int*>(row_c + 2 * R);            // [2][R] first key it sees
  int* row_hi = row_lo + 2 * R;                                   // [2][R] first key past those it sees
  int64_t* row_out = reinterpret_cast<int64_t*>(row_hi + 2 * R);  // [2][R] its place in out and lse, or -1
  int64_t* row_q = row_out + 2 * R;                               // [2][R] its place in q (elements), or -1
  float* set_m = reinterpret_cast<float*>(row_q + 2 * R);         // [SETS][R] running references
  float* set_n = set_m + SETS * R;                                // [SETS][R] their negatives
  float* set_l = set_n + SETS * R;                                // [SETS][R] sums
  float* join_m = set_l + SETS * R;                               // [R]
  float* join_l = join_m + R;                                     // [R]
  float* set_f = join_l + R;                                      // [SETS][R] a moved reference's factors
  Seg* segs = reinterpret_cast<Seg*>(set_f + SETS * R);           // [2]
  static_assert(2 * sizeof(Seg) == 80 && (C::kRowBytes - 80) % 8 == 0 && offRow % 16 == 0, "segment records");
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + offBar);   // a K tile has landed
  uint64_t* kempty = kfull + SK;                                  // and is done with
  uint64_t* vfull = kempty + SK;                                  // a V tile
  uint64_t* vempty = vfull + SV;
  uint64_t* sfull = vempty + SV;                                  // scores computed
  uint64_t* sempty = sfull + BUFS;                                // and read
  uint64_t* qfull = sempty + BUFS;                                   // query terms written
  uint64_t* qempty = qfull + 2;                                   // and done with
  uint64_t* sfirst = qempty + 2;                                  // the first segment is known
  uint64_t* tbar = sfirst + 1;                                    // tensor memory allocated, term scales stored
  uint64_t* never = tbar + 1;                                     // fault injection: nothing arrives here
  int64_t* plan = reinterpret_cast<int64_t*>(never + 1);          // this CTA's share [f0, f1); all units; CTAs
  int* plan_at = reinterpret_cast<int*>(plan + 5);                // its first item: request, item, tile
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(plan_at + 3);
  int* last_flag = reinterpret_cast<int*>(tmem_slot + 1);
  static_assert((2 * SK + 2 * SV + 2 * BUFS + 4 + 3) * 8 + 5 * 8 + 12 + 8 <= 1024, "barrier area");
  __shared__ int64_t scan[kThreads / 32 + 1];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < SK; ++s) {
      mbar_init(&kfull[s], 32);  // every lane of the loading warp
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(&vfull[s], 32);
      mbar_init(&vempty[s], 4);
    }
    for (int s = 0; s < BUFS; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&qfull[s], 32 + C::kWarps);
      mbar_init(&qempty[s], 1 + C::kWarps);
    }
    mbar_init(tbar, 1);
    mbar_init(sfirst, 32);
    mbar_init(never, 1);
    fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this CTA's share of the tiles of all requests (a block scan over the lengths)
  {
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) {
      const Req r = load_req(a, b, group, R, C::kItemCost);
      sum += r.units(a.cache.kv_heads);
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      all += scan[w];
    }
    before += incl - sum;
    const int64_t ctas = FewSplit::ctas(all, (int)gridDim.x);
    const bool has = (int64_t)blockIdx.x < ctas && all > 0;
    if (threadIdx.x == 0) {
      plan[0] = plan[1] = 0;
      plan[3] = all;
      plan[4] = ctas;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // the share's two boundaries; the thread whose requests hold one places it
      const int64_t f = has ? FewSplit::share(all, blockIdx.x + e, (int)ctas) : -1;
      if (e == 1 && f == all && threadIdx.x == 0) plan[1] = all;
      if (f >= before && f < before + sum) {
        int64_t off = f - before;
        int b = b0;
        for (;; ++b) {
          const Req r = load_req(a, b, group, R, C::kItemCost);
          const int64_t n = r.units(a.cache.kv_heads);
          if (off < n) {
            int item = (int)((unsigned)off / (unsigned)r.cost), at = 0;  // (off < 2^31: at most 16 million keys a request)
            if (n > INT32_MAX) item = (int)(off / r.cost);
            at = (int)(off - (int64_t)item * r.cost);
            const int move = FewSplit::move(at, r.cost);  // to an end of the item, if one is near
            plan[e] = f + move;
            if (e == 0) {
              plan_at[0] = b;
              plan_at[1] = move > 0 ? item + 1 : item;
              plan_at[2] = move != 0 ? 0 : at;
            }
            break;
          }
          off -= n;
        }
      }
    }
  }
  __syncthreads();
  const int64_t f0 = plan[0], f1 = plan[1], all_units = plan[3];
  const int ctas = (int)plan[4];
  bool failed = false;

  // requests that see no key give zeros; requests outside the contract are reported
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int q0 = __ldg(a.query_start + b), ql = __ldg(a.query_start + b + 1) - q0, n = __ldg(a.total_lens + b);
    const Req r = load_req(a, b, group, R, C::kItemCost);
    if (threadIdx.x == 0 && (ql < 0 || (ql > 0 && r.qlen == 0) || n > r.total)) record_error(a.err, kErrIndex);
    if (r.qlen > 0 && r.tiles == 0) {
      for (int64_t i = threadIdx.x; i < (int64_t)r.qlen * a.q_heads * (D / 8); i += kThreads)
        reinterpret_cast<uint4*>(a.out + (int64_t)r.q0 * a.q_heads * D)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int64_t i = threadIdx.x; i < (int64_t)r.qlen * a.q_heads; i += kThreads)
          a.lse[(int64_t)r.q0 * a.q_heads + i] = -INFINITY;
    }
  }
  if (f0 >= f1) return;  // (uniform) no tile for this CTA

  const int page_size = a.cache.page_size, page_shift = 31 - __clz(page_size);

  if (warp < C::kWarps + 2 && warp >= C::kWarps) {
    // -------------------------------------------------- loads: K, and V
    // Sixteen-byte asynchronous copies: a copy's row, chunk and page are the lane's own arithmetic, so a tile
    // costs the same few dozen instructions whatever the page size.  (Bulk and tensor copies, whose
    // operands are uniform registers, took ~140 cycles each to issue, and a tile of 16-row pages is 32 of them.)
    const bool is_v = warp == C::kWarps + 1;
    uint64_t* full = is_v ? vfull : kfull;
    uint64_t* empty = is_v ? vempty : kempty;
    const int stages = is_v ? SV : SK;
    const uint32_t ring = base + (is_v ? offV : 0), scale_ring = base + (is_v ? offSv : offS);
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(is_v ? a.cache.v_codes : a.cache.k_codes);
    const uint8_t* scales = is_v ? a.cache.v_scales : a.cache.k_scales;
    constexpr int CPR = C::kRowB / 16, RPI = 32 / CPR;  // chunks of a row, rows (512 bytes) of an instruction
    constexpr int SPI = 512 / C::kSB;                   // keys whose scales an instruction moves
    const int tile_shift = 7 - page_shift;              // log2 of a tile's pages
    const int srow = lane * 16 / C::kSB;
    // a lane's place in 512 bytes of codes, under the row swizzle; where its period is 1024 bytes (D = 256) the
    // second 512 have their own
    const uint32_t at = lane * 16, at0 = at ^ ((at >> 3) & C::kSwz), at1 = (at + 512) ^ (((at + 512) >> 3) & C::kSwz);
    codes += lane * 16;
    int s = 0, round = 0;
    Walk w;
    w.begin(a, group, R, C::kItemCost, plan_at[0], plan_at[1], plan_at[2], f0, f1);
    while (w.next()) {
      // Cache rows of the table's next 32 pages, a page a lane, and the 32 after them on their way: one
      // table load's latency a tile would bound the ring.
      const int32_t* table = a.block_table + (int64_t)w.b * a.table_stride;
      const int last = (w.r.total - 1) >> page_shift;
      int batch = (w.r.lo_tile + w.ta) << tile_shift;
      int nxt = __ldg(table + min(batch + lane, last));
      int cur = 0, left = 0;
      for (int t = w.ta; t < w.tb; ++t) {
        const int j0 = (w.r.lo_tile + t) * kTile;
        // pages of the tile that hold visible keys (a window's first page, the request's last)
        const int pa = max(w.r.first - j0, 0) >> page_shift;
        const int pb = (min(w.r.total - j0, kTile) + page_size - 1) >> page_shift;
        const int first_pg = (w.r.lo_tile + t) << tile_shift;
        if (left == 0) {  // (a tile's pages never straddle two batches: both are powers of two)
          if (first_pg != (w.r.lo_tile + w.ta) << tile_shift) batch += 32;
          const int pg = batch + lane;
          if ((nxt < 0 || nxt >= a.cache.num_pages) && pg <= last && pg >= w.r.first >> page_shift) {
            record_error(a.err, kErrIndex);
            nxt = 0;
          }
          cur = (max(nxt, 0) * a.cache.kv_heads + w.h) << page_shift;
          nxt = __ldg(table + min(batch + 32 + lane, last));
          left = 32 >> tile_shift;
        }
        --left;
        if (round > 0) mbar_wait(&empty[s], (round - 1) & 1, a.err, failed);
        const uint32_t dc = ring + s * C::kCodes, ds = scale_ring + s * C::kScales;
        const int idx = first_pg - batch;  // the tile's first page in the batch
        auto pages = [&](auto ipp) {       // instructions of a page
          constexpr int IPP = decltype(ipp)::value, NP = kTile / RPI / IPP;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const int row = __shfl_sync(0xffffffffu, cur, idx + p);
            if (p >= pa && p < pb) {
              const uint8_t* src = codes + (int64_t)row * C::kRowB;
              const uint32_t dst = dc + p * (IPP * 512);
#pragma unroll
              for (int i = 0; i < IPP; ++i) cp_async16(dst + i * 512 + (i & 1 ? at1 - 512 : at0), src + i * 512);
            }
          }
        };
        switch (page_shift) {
          case 4: pages(std::integral_constant<int, 16 / RPI>()); break;
          case 5: pages(std::integral_constant<int, 32 / RPI>()); break;
          case 6: pages(std::integral_constant<int, 64 / RPI>()); break;
          default: pages(std::integral_constant<int, 128 / RPI>()); break;
        }
#pragma unroll
        for (int i = 0; i < (kTile + SPI - 1) / SPI; ++i) {
          const int r = i * SPI + srow, p = min(r, kTile - 1) >> page_shift;
          const int row = __shfl_sync(0xffffffffu, cur, idx + p) + (r & (page_size - 1));
          if (r < kTile && p >= pa && p < pb) cp_async16(ds + r * C::kSB, scales + (int64_t)row * C::kSB);
        }
        // arrives when this lane's copies have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(&full[s])) : "memory");
        if (++s == stages) { s = 0; ++round; }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy may still be writing shared memory when the CTA exits
  } else if (warp == C::kWarps + 2) {
    // ------------------------------------------------- K scales, MMA issue
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(tmem_slot)), "n"(C::kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    // the query terms' scales, column n / 32 of lane n % 32 of a chain, copied to every lane quadrant from the
    // first kilobyte of the output area, idle until the first segment ends
#pragma unroll
    for (int ch = 0; ch < kChains; ++ch) {
      uint32_t v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = 32 * c + lane;
        v[c] = n < kCols * R ? term_scale<MODE>(term_of(ch, n / R)) * 0x01010101u : 0u;
      }
      reinterpret_cast<uint4*>(smem + offOut)[32 * ch + lane] = make_uint4(v[0], v[1], v[2], v[3]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncwarp();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t leader = elect_one_sync();
    if (leader) {
      if (inject_timeout) {
        bool injected = false;  // separate flag: the injected expiry must not stop later waits
        mbar_wait(never, 0, a.err, injected, 2000000LL);
      }
#pragma unroll
      for (int ch = 0; ch < kChains; ++ch) tc_cp_sf(tmem + C::kSfb + 4 * ch, desc_sf(base + offOut + 512 * ch));
      mbar_arrive(tbar);  // publishes tmem_slot to the consumers
    }
    constexpr uint32_t idesc0 = (1u << 7) | (1u << 10) | ((uint32_t)(C::kN >> 3) << 17) | (MODE == 1 ? 1u << 23 : 0u) |
                                ((128u >> 4) << 24);
    constexpr uint32_t layout = D == 64 ? 6u : D == 128 ? 4u : 2u;  // 32-, 64-, 128-byte swizzle
    int s = 0, round = 0, it = 0;
    for (int seg = 0;; ++seg) {
      const int qb = seg & 1;
      mbar_wait(&qfull[qb], (seg >> 1) & 1, a.err, failed);
      const int n = failed ? 0 : segs[qb].tb - segs[qb].ta;
      if (n <= 0) break;
      for (int i = 0; i < n; ++i, ++it) {
        const int buf = it % BUFS;
        // the scores of tile it - BUFS have been read, so its MMAs and scale copy are done
        if (it >= BUFS) mbar_wait(&sempty[buf], (it / BUFS - 1) & 1, a.err, failed);
        mbar_wait(&kfull[s], round & 1, a.err, failed);
        // lane n % 32, word n / 32: key n's scale word j, for every k-step group j
        const uint8_t* lin = smem + offS + s * C::kScales;
        uint32_t v[4][C::kWords];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint8_t* src = lin + (32 * c + lane) * C::kSB;
          if (C::kSB == 2) v[c][0] = *reinterpret_cast<const uint16_t*>(src);
          else if (C::kSB == 4) v[c][0] = *reinterpret_cast<const uint32_t*>(src);
          else
#pragma unroll
            for (int j = 0; j < C::kWords; j += 2) {
              const uint2 x = *reinterpret_cast<const uint2*>(src + 4 * j);
              v[c][j] = x.x;
              v[c][(j + 1) % C::kWords] = x.y;
            }
        }
        uint4* dst = reinterpret_cast<uint4*>(smem + offSfa + buf * C::kSfaBytes) + lane;
#pragma unroll
        for (int j = 0; j < C::kWords; ++j) dst[32 * j] = make_uint4(v[0][j], v[1][j], v[2][j], v[3][j]);
        // both these and the copied codes, seen through the barrier, become visible to the tensor core
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (leader) {
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < C::kWords; ++j)
            tc_cp_sf(tmem + C::kSfa + 16 * buf + 4 * j, desc_sf(base + offSfa + buf * C::kSfaBytes + 512 * j));
          const uint64_t ad = desc_k(base + s * C::kCodes, 8 * C::kRowB, layout);
          const uint64_t bd = desc_k(base + offQ + qb * C::kQBytes, 8 * C::kRowB, layout);
#pragma unroll
          for (int ch = 0; ch < kChains; ++ch)
#pragma unroll
            for (int ks = 0; ks < D / 64; ++ks) {
              const int word = MODE == 2 ? ks : ks / 2;
              const uint32_t id = MODE == 2 ? 0u : 2u * (ks & 1);
              mma_fp4<MODE>(tmem + C::kSStride * buf, ad + 2 * ks, bd + ch * (C::kQChain >> 4) + 2 * ks,
                            idesc0 | (id << 29) | (id << 4), tmem + C::kSfa + 16 * buf + 4 * word,
                            tmem + C::kSfb + 4 * ch, ch > 0 || ks > 0);
            }
          tc_commit(&sfull[buf]);
          tc_commit(&kempty[s]);
          if (i + 1 == n) tc_commit(&qempty[qb]);
        }
        __syncwarp();
        if (++s == SK) { s = 0; ++round; }
      }
    }
  } else if (warp == C::kWarps + 3) {

    // ------------------------------------------------------------ queries
    if (blockIdx.x == 0 && lane == 0) report_expired(a);
    Walk w;
    w.begin(a, group, R, C::kItemCost, plan_at[0], plan_at[1], plan_at[2], f0, f1);
    for (int seg = 0;; ++seg) {
      const int qb = seg & 1;
      if (seg >= 2) mbar_wait(&qempty[qb], ((seg >> 1) - 1) & 1, a.err, failed);
      if (!w.next()) {
        if (lane == 0) segs[qb].ta = segs[qb].tb = 0;
        __syncwarp();
        if (seg == 0) mbar_arrive(sfirst);  // (a share that holds nothing but fixed costs)
        else if (lane < C::kWarps) mbar_arrive(&qfull[qb]);
        mbar_arrive(&qfull[qb]);
        break;
      }
      {  // lane r: the keys row r sees and where it goes (R <= 32); rows past the block are not used
        const int rr = w.rb * R + lane, i = rr / group;
        const bool real = lane < R && rr < w.r.qlen * group;
        const int pos = w.r.total - w.r.qlen + i;
        const int hi = real ? max(pos + 1, 0) : INT32_MAX;
        const int lo = real && a.window > 0 ? max(pos + 1 - a.window, 0) : 0;
        if (lane < R) {
          row_hi[qb * R + lane] = hi;
          row_lo[qb * R + lane] = lo;
          const int head = w.h * group + rr - i * group;
          row_out[qb * R + lane] = real ? (int64_t)(w.r.q0 + i) * a.q_heads + head : -1;
          row_q[qb * R + lane] = real ? (int64_t)(w.r.q0 + i) * a.q_token + (int64_t)head * a.q_head : -1;
        }
        const int hi_min = __reduce_min_sync(0xffffffffu, hi), lo_max = __reduce_max_sync(0xffffffffu, lo);
        if (lane == 0) segs[qb] = Seg{w.ta, w.tb, w.r.total, w.r.first, w.r.lo_tile, w.r.tiles, lo_max, hi_min, w.start};
      }
      __syncwarp();
      if (seg == 0) {
        mbar_arrive(sfirst);  // the consumers write the first segment's terms: it takes this warp several times as long
      } else {
#pragma unroll 1
        for (int r0 = 0; r0 < R; r0 += 4) query_rows<MODE, D, NB, 4>(a, smem + offQ + qb * C::kQBytes, row_q + qb * R, row_c + qb * R, r0, lane);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (seg > 0 && lane < C::kWarps) mbar_arrive(&qfull[qb]);  // in the consumers' place
      mbar_arrive(&qfull[qb]);
    }
  } else {
    // ----------------------------------------------------------- consumers
    const int grp = warp >> 2, quad = warp & 3, set = warp;
    const int g = lane >> 2, c = lane & 3;
    mbar_wait(tbar, 0, a.err, failed);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot + ((uint32_t)(32 * quad) << 16);
    const uint32_t pbuf = base + offP + set * (NB * 512);
    const uint32_t pread =
        pbuf + (uint32_t)(((lane >> 4) * 16 + key_of<D>((lane & 7) >> 1, (lane & 1) + ((lane >> 3) & 1) * 2)) * 16);
    float* mm = set_m + set * R;
    float* factors = set_f + set * R;
    const float gsv = (MODE == 2 && a.cache.gs_v) ? __ldg(a.cache.gs_v) : 1.0f;
    constexpr int CH = C::kCh, VB = CH / 2;                          // channels, code bytes of a thread's key
    constexpr int SPT = MODE == 2 && CH > 16 ? CH / 16 : 1;           // its scales
    // Where its keys' codes and scales lie in a stage.  Keys i of a slab differ by 128 bytes of codes (i & 1: the
    // bit the row swizzle folds onto bit 4) and by eight rows (i >> 1).
    const uint32_t vc = (uint32_t)((32 * quad + key_of<D>(c, 0)) * C::kRowB + g * VB);
    const uint32_t vc0 = vc ^ ((vc >> 3) & C::kSwz), vc1 = (vc0 + 128) ^ 16;
    const uint32_t vsc = (uint32_t)((32 * quad + key_of<D>(c, 0)) * C::kSB + g * CH / C::kGroup);
    constexpr int KSTEP = 128 / C::kRowB;  // keys between i = 0 and i = 1
    const uint64_t unit2 = pack2(__float_as_uint(kLastUnit), __float_as_uint(kLastUnit));
    float* mn = set_n + set * R;
    const uint32_t mn_a = smem_u32(mn);
    // the first segment's query terms
    mbar_wait(sfirst, 0, a.err, failed);
#pragma unroll 1
    for (int r = warp; r < R && !failed && segs[0].ta < segs[0].tb; r += C::kWarps)
      query_rows<MODE, D, NB, 1>(a, smem + offQ, row_q, row_c, r, lane);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(&qfull[0]);
    int s = 0, round = 0, it = 0;
    for (int seg = 0;; ++seg) {
      const int qb = seg & 1;
      mbar_wait(&qfull[qb], (seg >> 1) & 1, a.err, failed);
      const int n_tiles = failed ? 0 : segs[qb].tb - segs[qb].ta;
      if (n_tiles <= 0) break;
      float acc[CH / 2][NB][4] = {};
      uint64_t l2[NB][4] = {};  // sums of rows (8 nb + 2 i, + 1)
      int vexp = -127;  // MXFP4: V is held relative to 2^vexp
      if (lane < R) {
        mm[lane] = kNone;
        mn[lane] = -kNone;
      }
      __syncwarp();
      const uint32_t rc_a = smem_u32(row_c + qb * R);
      const int key0 = (segs[qb].lo_tile + segs[qb].ta) * kTile;
      const int lo_max = segs[qb].lo_max, hi_min = segs[qb].hi_min;
      int o = (grp + C::kGroups - it % C::kGroups) % C::kGroups;  // this group's first tile of the segment
      s += o;
      for (; o < n_tiles; o += C::kGroups, s += C::kGroups) {
        while (s >= SV) { s -= SV; ++round; }
        const int j0 = key0 + o * kTile;
        // masks only in tiles that hold an end of some row's keys
        const bool edge = j0 < lo_max || j0 + kTile > hi_min;
        const int j = j0 + 32 * quad + lane;  // this lane's key
        const int buf = (it + o) % BUFS;
        mbar_wait(&vfull[s], round & 1, a.err, failed);
        const uint32_t codes = base + offV + s * C::kCodes;
        uint32_t vs[2][4];  // V scale bytes of the thread's eight keys (two each where SPT == 2)
        {
          const uint32_t sa = base + offSv + s * C::kScales + vsc;
#pragma unroll
          for (int slab = 0; slab < 2; ++slab)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t at = sa + (16 * slab + KSTEP * (i & 1) + 8 * (i >> 1)) * C::kSB;
              vs[slab][i] = SPT == 2 ? lds16(at) : lds8(at);
            }
        }
        mbar_wait(&sfull[buf], ((it + o) / BUFS) & 1, a.err, failed);
        tc_fence_after();
        if (edge) {
#pragma unroll
          for (int slab = 0; slab < 2; ++slab)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // keys no row sees may hold anything: their scale becomes a finite one (p is zero)
              const int key = j0 + 32 * quad + 16 * slab + key_of<D>(c, i);
              if (key >= segs[qb].total || key < segs[qb].first) vs[slab][i] = MODE == 2 ? 0 : (uint32_t)(vexp + 127);
            }
        }
        unsigned wide = 0;  // blocks of rows whose probabilities are bf16
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          // ---- scores of this lane's key, two rows a register pair
          uint64_t t2[4], x2[4], f2[4];
          {
            uint32_t d[kCols][8];
#pragma unroll
            for (int k = 0; k < kCols; ++k) tmem_ld8(tmem + (uint32_t)(C::kSStride * buf + k * R + 8 * nb), d[k]);
            const uint4 f0 = lds128(rc_a + 32 * nb), f1 = lds128(rc_a + 32 * nb + 16);
            const uint4 n0 = lds128(mn_a + 32 * nb), n1 = lds128(mn_a + 32 * nb + 16);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            if (nb == NB - 1) {
              tc_fence_before();
              if (lane == 0) mbar_arrive(&sempty[buf]);  // a later tile may overwrite them
            }
            f2[0] = pack2(f0.x, f0.y), f2[1] = pack2(f0.z, f0.w), f2[2] = pack2(f1.x, f1.y), f2[3] = pack2(f1.z, f1.w);
            const uint64_t n2[4] = {pack2(n0.x, n0.y), pack2(n0.z, n0.w), pack2(n1.x, n1.y), pack2(n1.z, n1.w)};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              t2[r] = add2(add2(pack2(d[0][2 * r], d[0][2 * r + 1]), pack2(d[1][2 * r], d[1][2 * r + 1])),
                           fma2(pack2(d[3][2 * r], d[3][2 * r + 1]), unit2, pack2(d[2][2 * r], d[2][2 * r + 1])));
              x2[r] = fma2(t2[r], f2[r], n2[r]);
            }
          }
          float x[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) unpack2(x2[r], x[2 * r], x[2 * r + 1]);
          unsigned hidden = 0;
          if (edge) {
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (j >= row_hi[qb * R + 8 * nb + r] || j < row_lo[qb * R + 8 * nb + r]) {
                hidden |= 1u << r;
                x[r] = -INFINITY;
              }
          }
          // ---- softmax of eight rows
          const float high = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
          if (__any_sync(0xffffffffu, high > kMax)) {  // move the references that a score has passed (or that are not set)
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              float t[2], f[2], l[2];
              unpack2(t2[r >> 1], t[0], t[1]);
              unpack2(f2[r >> 1], f[0], f[1]);
              unpack2(l2[nb][r >> 1], l[0], l[1]);
              const float sc = hidden >> r & 1 ? -INFINITY : t[r & 1] * f[r & 1];
              const float top = warp_max(sc), m = mm[8 * nb + r];
              const float n = top > m + kMax ? top - kHead : m, scale = exp2f(m - n);
              l[r & 1] *= scale;
              l2[nb][r >> 1] = pack2(__float_as_uint(l[0]), __float_as_uint(l[1]));
              x[r] = sc - n;
              __syncwarp();
              if (lane == 0) {
                mm[8 * nb + r] = n;
                mn[8 * nb + r] = -n;
                factors[8 * nb + r] = scale;
              }
            }
            __syncwarp();
            const float2 f = *reinterpret_cast<const float2*>(factors + 8 * nb + 2 * c);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
              acc[i][nb][0] *= f.x;
              acc[i][nb][1] *= f.y;
              acc[i][nb][2] *= f.x;
              acc[i][nb][3] *= f.y;
            }
          }
          const float low = fminf(fminf(fminf(x[0], x[1]), fminf(x[2], x[3])), fminf(fminf(x[4], x[5]), fminf(x[6], x[7])));
          bool tiny = false;  // probabilities outside f16's range in this tile
          if (__any_sync(0xffffffffu, low < -kTiny)) {
#pragma unroll
            for (int r = 0; r < 8; ++r) tiny |= x[r] < -kTiny && x[r] > -126.0f;
            tiny = __any_sync(0xffffffffu, tiny);
          }
#pragma unroll
          for (int r = 0; r < 8; ++r) x[r] = exp2_approx(x[r]);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            l2[nb][r] = add2(l2[nb][r], pack2(__float_as_uint(x[2 * r]), __float_as_uint(x[2 * r + 1])));
          uint32_t pk[4];
          if (!tiny) {
#pragma unroll
            for (int r = 0; r < 4; ++r) pk[r] = pack_f16x2(x[2 * r], x[2 * r + 1]);
          } else {
            wide |= 1u << nb;
#pragma unroll
            for (int r = 0; r < 4; ++r) pk[r] = pack_bf16x2_rn(x[2 * r] * 256.0f, x[2 * r + 1] * 256.0f);
          }
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                       :: "r"(pbuf + nb * 512 + lane * 16), "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3]) : "memory");
        }
        __syncwarp();
        // ---- the probabilities as B fragments: keys 0-15 of the warp, keys 16-31
        uint32_t pb[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(pb[nb][0]), "=r"(pb[nb][1]), "=r"(pb[nb][2]), "=r"(pb[nb][3])
                       : "r"(pread + nb * 512) : "memory");
        uint32_t below[2][4];  // MXFP4: how far each key's scale lies below 2^vexp
        if (MODE == 1) {
          uint32_t far = 0;  // (a scale above it wraps to a large distance)
          auto distances = [&]() {
            far = 0;
#pragma unroll
            for (int slab = 0; slab < 2; ++slab)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                below[slab][i] = (uint32_t)(vexp + 127) - vs[slab][i];
                far = max(far, below[slab][i]);
              }
          };
          distances();
          if (__any_sync(0xffffffffu, far > 20u)) {
            int hi = 0;
#pragma unroll
            for (int slab = 0; slab < 2; ++slab)
#pragma unroll
              for (int i = 0; i < 4; ++i) hi = max(hi, (int)vs[slab][i]);
            hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
            hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, 2)) - 127;
            const int n = max(hi, vexp);
            const float f = exp2f((float)max(vexp - n, -200));
            vexp = n;
#pragma unroll
            for (int i = 0; i < CH / 2; ++i)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][nb][k] *= f;
            distances();
            if (__any_sync(0xffffffffu, far > 20u)) {  // V outside f16's range: everything in bf16
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                if (!(wide >> nb & 1))
#pragma unroll
                  for (int k = 0; k < 4; ++k) pb[nb][k] = f16x2_to_bf16x2_256(pb[nb][k]);
              wide = (1u << NB) - 1;
            }
          }
        }
        // ---- o += p V, sixteen keys at a time
#pragma unroll
        for (int slab = 0; slab < 2; ++slab) {
          uint32_t wd[4][CH / 8];  // the four keys' codes of the thread's channels
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t at = codes + (i & 1 ? vc1 : vc0) + (16 * slab + 8 * (i >> 1)) * C::kRowB;
            if (VB == 4) {
              wd[i][0] = lds32(at);
            } else if (VB == 8) {
              const uint2 v = lds64(at);
              wd[i][0] = v.x;
              wd[i][1 % (CH / 8)] = v.y;
            } else {
              const uint4 v = lds128(at);
              wd[i][0] = v.x;
              wd[i][1 % (CH / 8)] = v.y;
              wd[i][2 % (CH / 8)] = v.z;
              wd[i][3 % (CH / 8)] = v.w;
            }
          }
          if (wide != (1u << NB) - 1) {
            uint32_t s2[SPT][2];  // scales of key pairs (0, 1) and (2, 3) as f16
#pragma unroll
            for (int k = 0; k < SPT; ++k)
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const uint32_t x0 = (vs[slab][2 * p] >> (8 * k)) & 0xFFu, x1 = (vs[slab][2 * p + 1] >> (8 * k)) & 0xFFu;
                if (MODE == 2) {
                  const uint16_t both = (uint16_t)(x0 | (x1 << 8));
                  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2[k][p]) : "h"(both));
                } else {
                  // 2^(E - vexp) by its fp32 bits: E is within [-20, 0] of vexp here
                  s2[k][p] = pack_f16x2(__uint_as_float((127u - below[slab][2 * p]) << 23),
                                        __uint_as_float((127u - below[slab][2 * p + 1]) << 23));
                }
              }
#pragma unroll
            for (int q = 0; q < CH / 8; ++q) {
              const int k = SPT == 2 ? q / 2 : 0;
              uint32_t ev[2][4], od[2][4];  // two keys' codes in a byte: even channels, odd channels
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const uint32_t x = wd[2 * p][q], y = wd[2 * p + 1][q];
                e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), ev[p]);
                e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), od[p]);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t af[4] = {mul_f16x2(ev[0][i], s2[k][0]), mul_f16x2(od[0][i], s2[k][0]),
                                        mul_f16x2(ev[1][i], s2[k][1]), mul_f16x2(od[1][i], s2[k][1])};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  if (NB == 1 || !(wide >> nb & 1)) mma_f16(acc[4 * q + i][nb], af, pb[nb][2 * slab], pb[nb][2 * slab + 1]);
              }
            }
          }
          if (wide) {
            uint32_t s2[SPT][2];  // scales times 2^118 as bf16: V times 2^-8, p carries 2^8
#pragma unroll
            for (int k = 0; k < SPT; ++k)
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const uint32_t x0 = (vs[slab][2 * p] >> (8 * k)) & 0xFFu, x1 = (vs[slab][2 * p + 1] >> (8 * k)) & 0xFFu;
                if (MODE == 2)
                  s2[k][p] = pack_bf16x2_rn(e4m3_to_f32(x0) * 0x1p118f, e4m3_to_f32(x1) * 0x1p118f);
                else
                  s2[k][p] = pack_bf16x2_rn(exp2i_f32(max((int)x0 - 9 - vexp, -126)),
                                            exp2i_f32(max((int)x1 - 9 - vexp, -126)));
              }
#pragma unroll
            for (int q = 0; q < CH / 8; ++q) {
              const int k = SPT == 2 ? q / 2 : 0;
              const uint32_t n0[2] = {__byte_perm(wd[0][q], wd[1][q], 0x5410), __byte_perm(wd[0][q], wd[1][q], 0x7632)};
              const uint32_t n1[2] = {__byte_perm(wd[2][q], wd[3][q], 0x5410), __byte_perm(wd[2][q], wd[3][q], 0x7632)};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t x = n0[i >> 1], y = n1[i >> 1];
                const uint32_t af[4] = {
                    mul_bf16x2(i & 1 ? e2m1_to_bf16<2>(x) : e2m1_to_bf16<0>(x), s2[k][0]),
                    mul_bf16x2(i & 1 ? e2m1_to_bf16<3>(x) : e2m1_to_bf16<1>(x), s2[k][0]),
                    mul_bf16x2(i & 1 ? e2m1_to_bf16<2>(y) : e2m1_to_bf16<0>(y), s2[k][1]),
                    mul_bf16x2(i & 1 ? e2m1_to_bf16<3>(y) : e2m1_to_bf16<1>(y), s2[k][1])};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  if (NB == 1 || (wide >> nb & 1)) mma_bf16(acc[4 * q + i][nb], af, pb[nb][2 * slab], pb[nb][2 * slab + 1]);
              }
            }
          }
        }
        __syncwarp();  // every lane's loads of the stage (and of the probabilities) are done
        if (lane == 0) mbar_arrive(&vempty[s]);
      }
      s -= o - n_tiles;  // where the segment's last tile leaves the ring
      while (s < 0) { s += SV; --round; }
      it += n_tiles;

      // ---- the segment's end: join the sets
      const Seg e = segs[qb];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float l0, l1;
        unpack2(l2[r >> 3][(r >> 1) & 3], l0, l1);
        float v = r & 1 ? l1 : l0;
#pragma unroll
        for (int x = 16; x; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
        if (lane == 0) set_l[set * R + r] = v;
      }
      named_sync<kConsumers>(1);
      float* set_f = reinterpret_cast<float*>(smem + offP);  // a set's factor to the joint reference, over the joint sum
      if (threadIdx.x < SETS * R) {
        const int r = threadIdx.x % R;
        float m = -INFINITY, v = 0.f;
#pragma unroll
        for (int k = 0; k < SETS; ++k) m = fmaxf(m, set_m[k * R + r]);
#pragma unroll
        for (int k = 0; k < SETS; ++k) v += set_l[k * R + r] * exp2f(set_m[k * R + r] - m);
        set_f[threadIdx.x] = v == 0.f ? 0.f : exp2f(set_m[threadIdx.x] - m) / v;
        if (threadIdx.x < R) {
          join_m[r] = m;
          join_l[r] = v;
        }
      }
      named_sync<kConsumers>(1);
      // Outputs on the joint reference, divided by the joint sum (V may be near fp32's largest values, whose undivided
      // sums would pass it); the second half of the sets hands its own to the first (half the space).
      float2* dump = reinterpret_cast<float2*>(smem + offOut) + (set % (SETS / 2)) * (C::kPieces * 32) + lane;
      const float ve = MODE == 1 ? exp2i_f32(vexp) : 1.0f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 8 * nb + 2 * c + h;
          const float f = set_f[set * R + r] * ve;
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) {
            acc[i][nb][h] *= f;
            acc[i][nb][2 + h] *= f;
            if (set >= SETS / 2) dump[((i * NB + nb) * 2 + h) * 32] = make_float2(acc[i][nb][h], acc[i][nb][2 + h]);
          }
        }
      named_sync<kConsumers>(1);
      if (set < SETS / 2)
#pragma unroll
        for (int i = 0; i < CH / 2; ++i)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2& u = dump[((i * NB + nb) * 2 + h) * 32];
              u = make_float2(u.x + acc[i][nb][h], u.y + acc[i][nb][2 + h]);
            }
      named_sync<kConsumers>(1);
      constexpr int X = C::kPieces * 32;                          // float2 of the output
      constexpr int XN = (X + kConsumers - 1) / kConsumers;            // of a thread
      // element x: row 8 nb + 2 c + h, channels kCh g + 2 i, + 1
      auto row_of = [](int x) { return 8 * ((x >> 6) % NB) + 2 * (x & 3) + ((x >> 5) & 1); };
      auto total = [&](int x) {
        const float2* src = reinterpret_cast<const float2*>(smem + offOut) + x;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < SETS / 2; ++k) {
          const float2 u = src[k * X];
          v.x += u.x;
          v.y += u.y;
        }
        return v;
      };
      auto store = [&](int x, float2 v, float jm, float ls) {
        const int r = row_of(x), ch = CH * ((x & 31) >> 2) + 2 * ((x >> 6) / NB);
        const int64_t at = row_out[qb * R + r];
        if (at < 0) return;
        *reinterpret_cast<uint32_t*>(a.out + at * D + ch) = pack_bf16x2_rn(v.x * gsv, v.y * gsv);
        if (a.lse && ch == 0) a.lse[at] = ls == 0.f ? -INFINITY : (jm + log2f(ls)) * 0.6931471805599453f;
      };
      auto release = [&]() {  // the segment's query rows, key ranges and output rows are done with
        __syncwarp();
        if (lane == 0) mbar_arrive(&qempty[qb]);
      };
      if (e.ta == 0 && e.tb == e.tiles) {
        for (int x = threadIdx.x; x < X; x += kConsumers) store(x, total(x), join_m[row_of(x)], join_l[row_of(x)]);
        release();
        continue;
      }
      // A piece: into the workspace; the CTA that completes the item's count joins its pieces.  A CTA
      // starts inside at most one item (its piece 0) and ends inside at most one that it began (piece 1).
      const int c0 = FewSplit::first(all_units, e.start, ctas), c1 = FewSplit::last(all_units, e.start, e.tiles, C::kItemCost, ctas);
      auto piece = [&](int k) { return pieces + (int64_t)(2 * k + (k == c0)) * C::kSlot; };
      float* mine = piece(blockIdx.x);
      for (int x = threadIdx.x; x < X; x += kConsumers) __stcg(reinterpret_cast<float2*>(mine) + x, total(x));
      if (threadIdx.x < R) {
        __stcg(mine + 2 * X + threadIdx.x, join_m[threadIdx.x]);
        __stcg(mine + 2 * X + R + threadIdx.x, join_l[threadIdx.x]);
      }
      named_sync<kConsumers>(1);
      if (threadIdx.x == 0) {
        __threadfence();  // the barrier has ordered every thread's stores before it
        int* arrived = arrivals + 8 * c0;
        const int n = atomicAdd(arrived, 1);
        *last_flag = n == c1 - c0;
        if (n == c1 - c0) *arrived = 0;  // ready for the next call
        __threadfence();
      }
      named_sync<kConsumers>(1);
      if (!*last_flag) {
        release();
        continue;
      }
      // Every piece's m and l into shared memory (a chunk of pieces at a time) while this thread's outputs of them
      // are on their way; references only grow from chunk to chunk.
      constexpr int KC = NB == 1 ? 32 : 16;
      static_assert(3 * KC * R * 4 + R * 4 <= (int)C::kPBytes, "a chunk's m, l and factors fit the probabilities' space");
      float* cm = reinterpret_cast<float*>(smem + offP);
      float* cl = cm + KC * R;
      float* cf = cl + KC * R;  // weights: the sums on the chunk's reference, times 2^-24 (against overflow, as above)
      float* cr = cf + KC * R;  // that reference
      float2 v[XN] = {};
      float jm[XN], jl[XN];
#pragma unroll
      for (int i = 0; i < XN; ++i) jm[i] = kNone, jl[i] = 0.f;
      for (int k0 = c0; k0 <= c1; k0 += KC) {
        const int nk = min(KC, c1 + 1 - k0);
        for (int x = threadIdx.x; x < nk * R; x += kConsumers) {
          const float* src = piece(k0 + x / R) + 2 * X + x % R;
          cm[x] = __ldcg(src);
          cl[x] = __ldcg(src + R);
        }
#pragma unroll
        for (int i = 0; i < XN; ++i) {
          const int x = min((int)threadIdx.x + i * kConsumers, X - 1);
          float2 u[KC];
#pragma unroll
          for (int k = 0; k < KC; ++k) u[k] = __ldcg(reinterpret_cast<const float2*>(piece(k0 + min(k, nk - 1))) + x);
          if (i == 0) {
            named_sync<kConsumers>(1);
            for (int y = threadIdx.x; y < nk * R; y += kConsumers) {
              float m = kNone;
#pragma unroll 8
              for (int k = 0; k < nk; ++k) m = fmaxf(m, cm[k * R + y % R]);
              cf[y] = cl[y] * exp2f(cm[y] - m) * 0x1p-24f;
              if (y < R) cr[y] = m;
            }
            named_sync<kConsumers>(1);
          }
          const int r = row_of(x);
          const float m = fmaxf(jm[i], cr[r]), fo = exp2f(jm[i] - m), fn = exp2f(cr[r] - m);
          float2 w = make_float2(0.f, 0.f);
          float wl = 0.f;
#pragma unroll
          for (int k = 0; k < KC; ++k)
            if (k < nk) {
              const float g = cf[k * R + r];
              w.x += u[k].x * g;
              w.y += u[k].y * g;
              wl += g;
            }
          v[i] = make_float2(v[i].x * fo + w.x * fn, v[i].y * fo + w.y * fn);
          jl[i] = jl[i] * fo + wl * fn;
          jm[i] = m;
        }
        named_sync<kConsumers>(1);
      }
#pragma unroll
      for (int i = 0; i < XN; ++i) {
        const int x = threadIdx.x + i * kConsumers;
        const float inv = jl[i] == 0.f ? 0.f : 1.0f / jl[i];
        if (x < X) store(x, make_float2(v[i].x * inv, v[i].y * inv), jm[i], jl[i] * 0x1p24f);
      }
      release();
    }
  }
  if (failed) mark_expired(a);
  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarps + 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(*tmem_slot), "n"(C::kTmemCols)
                 : "memory");
  }
}

template <int MODE, int D, int NB>
cudaError_t launch(const DevInfo& d, const KvAttentionArgs& a, cudaStream_t s) {
  using C = Dec<MODE, D, NB>;
  const int group = a.q_heads / a.cache.kv_heads;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(d, kv_decode_kernel<MODE, D, NB>, (int)C::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  static_assert(kKvCtas <= 160, "FewSplit multiplies by the CTA count in 32 bits");
  cfg.gridDim = dim3((unsigned)std::min(kKvCtas, d.sm_count));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  return cudaLaunchKernelEx(&cfg, kv_decode_kernel<MODE, D, NB>, a, group, reinterpret_cast<int*>(ws + kKvArrivals),
                            reinterpret_cast<float*>(ws + kKvResults), a.inject_timeout);
}

template <int MODE, int D>
cudaError_t launch_rows(const DevInfo& d, const KvAttentionArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.max_query_len * (a.q_heads / a.cache.kv_heads);
  if (rows <= 8 || D == 256) return launch<MODE, D, 1>(d, a, s);
  return launch<MODE, D, D == 256 ? 1 : 2>(d, a, s);
}

}  // namespace

// Two pieces a CTA, of 8 or 16 rows.
size_t kv_decode_ws_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_query_len) {
  const int64_t rows = max_query_len * (q_heads / kv_heads), R = rows <= 8 || head_dim == 256 ? 8 : 16;
  return kKvResults + (size_t)(2 * kKvCtas * (R * head_dim + 2 * R) * 4);
}

bool kv_decode_supported(int head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }

cudaError_t launch_kv_decode(const DevInfo& d, const KvAttentionArgs& a, cudaStream_t s) {
  const int D = a.cache.head_dim;
  if (a.cache.mode == FP4_MODE_NVFP4)
    return D == 64 ? launch_rows<2, 64>(d, a, s) : D == 128 ? launch_rows<2, 128>(d, a, s) : launch_rows<2, 256>(d, a, s);
  return D == 64 ? launch_rows<1, 64>(d, a, s) : D == 128 ? launch_rows<1, 128>(d, a, s) : launch_rows<1, 256>(d, a, s);
}

}  // namespace fp4
