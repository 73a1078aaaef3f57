// kv_prefill.cu -- causal attention of many query rows over the paged 4-bit cache: the
// serving form for prompts and prompt chunks, where the tensor cores' rate is the bound.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(s_rj - m_r),   s_rj = c q_r . k_j
// with c = softmax_scale log2(e) gs_k, over the keys row r may see.  A row r is one (query
// token, head of the kv head's group), heads fastest, so that the rows of a tile
// see nearly the same keys.
//
// A CTA (one an SM) owns an item: 256 rows of one request and kv head as two tiles of 128
// (the MMA's M, one row per accumulator lane), and walks the keys 128 at a time:
//   S_i = Q_i K^T    tcgen05.mma.kind::f16 (bf16), both operands in shared memory
//   O_i += P_i V     P_i in tensor memory, in the columns S_i leaves; V as it is stored, keys as
//                    rows (an MN-major B operand)
// Scores, P and outputs stay in tensor memory (S: 2 x 128 columns, O: 2 x head_dim): while
// one tile's softmax runs, the tensor cores work on the other tile.  An item of at most 128 rows is
// a twin: both tiles hold the same rows and take the key tiles in turn, and as a row's two outputs lie in the same
// lane of tensor memory, the first tile's warps join them.  (16 requests x 8,000 tokens, 17 to 128 rows of 8
// heads of 128: 91 us, 121 with the second tile left empty; fetching codes two tiles ahead changes nothing: 91.)
//
// K and V are dequantized once per item and key by four warps each into bf16 tiles
// (exact: e2m1 times an E4M3 or E8M0 scale has at most six significant bits): the codes
// become f16 pairs by the hardware's converter, their exponents move to bf16's place with a
// shift and two masks, and one multiply by the block scale (two for E8M0, whose range
// needs it) restores the value.  256 rows an item halve that work a row.
//
// Softmax: a thread owns a row.  P is bf16 and so has fp32's range: the reference m_r is the
// first tile's maximum and moves only when 32 probabilities sum to more than 2^24, so that
// after the first tile the scores are read once, no maximum is taken of them and the output
// is almost never rescaled.  p is rounded to bf16 (2^-8), once; scores, sums and output are fp32.
// MXFP4's V reaches fp32's largest numbers, whose sums do not fit although their quotient does: an item whose output
// is not finite is done again with p 2^60 smaller.  (Found at its end: watching the sum beside V's scales tile by tile took
// the chunks below from 423 to 440 us, this to 430.)
//
// Work: up to 608 items are dealt out: their key tiles, with a fixed cost an item, form one
// sequence, of which each CTA takes an equal share; a cut near an item's end moves to
// it, and an item's pieces meet in the workspace, where the last warp to arrive joins its 32 rows'
// in the pieces' order (the same bits each time).  More items are handed out whole by an atomic
// counter, near the end of the one before; up to 64 requests the longest come first.
//   32 query heads on 8, NVFP4: a chunk of 512 tokens over 16,000 takes 130 us dealt out (1050 TFLOP/s) and 196 in
//   equal pieces handed out by the counter; 576 items of similar lengths (64 heads of 64 on 8, 4 chunks over 0..16k) take
//   as long either way.  Handed out whole, one long context among many short ones is its CTA's alone: 80 tokens of
//   which one has 131k keys, beside one chunk of 512, are 648 items and take 1.4 ms.
//
// What bounds it: for heads of 128 the tensor cores.  Two tiles' four products take 2300 cycles
// beside the other warps' traffic and a step about 3300, the rest being the ends of items and waits for a softmax
// (2000 cycles a tile, of which the exponentials 512).  For heads of 64 the softmax: the products take 1750 of 2900.
//   4096-token prompt, 40 heads of 128, NVFP4:      0.159 ms, 1082 TFLOP/s
//   4 chunks over 0..16k, 64 heads of 64, MXFP4:    0.430 ms,  717 TFLOP/s
// Tried and slower on the prompt: 64-key steps with two score buffers (200 us), scores fetched ahead (201), two warps a
// row (162, and 406 on the chunks), more registers for the softmax by setmaxnreg (186).
//
//   warps 0-7    softmax and output of tile warp / 4 (lane quadrant warp % 4)
//   warps 8-11   K: codes loaded a tile ahead into registers, dequantized into a
//                double-buffered tile; thread t owns key t
//   warps 12-15  V likewise
//   warp 16      MMA issue
//   warps 17-18  items, query tiles
#include <algorithm>
#include <cuda.h>

#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "kv_common.cuh"
#include "kv_split.h"
#include "launch.h"

namespace fp4 {
namespace {

constexpr int kRows = 256;      // query rows of an item
constexpr int kKeys = 128;      // keys of a tile
constexpr int kSorted = 64;     // requests of a call that are put in order
constexpr int kThreads = 608;
constexpr int kDealt = kThreads;  // calls of up to this many items are dealt out in equal shares (a thread computes an item's length)
constexpr float kFar = 0x1p24f;  // a row's reference moves when probabilities sum to more than this
constexpr float kNone = -1e30f;
// MXFP4's V may be so large that a sum of p V passes fp32 where the quotient does not.  A warp that finds it so has the item
// done again with p at most 2^-60, and moving at 2^-32: no context has the keys to pass it then.
constexpr float kLow = 60.f, kLowFar = 0x1p-32f;

template <int D>
struct Pre {
  static constexpr uint32_t kQ = 128 * D * 2;      // one query tile
  static constexpr uint32_t kKV = kKeys * D * 2;   // one K or V tile
  static constexpr uint32_t kHalf = 128 * 128;     // 64 elements of 128 rows
  static constexpr uint32_t offK = 2 * kQ, offV = offK + 2 * kKV, offBar = offV + 2 * kKV;
  static constexpr uint32_t offPre = offBar + 1024, offTiles = offPre + 8 * (kThreads + 1), offX = (offTiles + 8 * (kThreads + 1) + 15) / 16 * 16, kSmem = offX + 1024;
  static constexpr uint32_t kO = 256;              // output columns of tile 0; tile 1 follows
};

struct Item {
  int b, h, q0, qlen, total;  // total: keys
  int row0, rows;             // first row of the item in the request's (token, head) rows; rows of the request
  int j0;                     // first key tile
  int n[2];                   // key tiles of the two row tiles
  int tiles, twin;            // key tiles in all; both row tiles hold the same rows and take them in turn
  int stop;
  int again;                  // done again with small p, for the softmax warps of these bits
  int piece, pieces, first;   // this piece of the item's keys, of how many; CTA of the first one
};

// In the workspace an arrival word for each warp's 32 rows of a split item, and two pieces' results a CTA: outputs
// [tile][channel / 4][row][4], references and sums [tile][2][row].
template <int D>
constexpr size_t kSlotFloats = 256 * (D + 2);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// MN-major operand tile (keys as rows of 64 swizzled elements): 8-key atoms 1024 bytes apart, the next 64
// elements `lbo` bytes further
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
#define R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : R8(v, 0), R8(v, 8), R8(v, 16), R8(v, 24) : "r"(a));
}
#undef R8
#define R8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "r"(a), R8(v, 0) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      :: "r"(a), R8(v, 0), R8(v, 8) : "memory");
}
#undef R8
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return pack2(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes of a scale group -> eight bf16 (16 bytes).  `sc`: the scale (MXFP4), or the scale times 2^112 (NVFP4), as a
// bf16 pair.
template <int MODE>
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t sc) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // f16 bits moved to bf16's exponent place: the value times 2^-112
    uint32_t v = (h[i] & 0x80008000u) | ((h[i] >> 3) & 0x0FFF0FFFu);
    if (MODE == 1) v = mul_bf16x2(v, 0x77807780u);  // 2^112
    h[i] = mul_bf16x2(v, sc);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}
template <int MODE>
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
  if (MODE == 1) {  // 2^(byte - 127), 2^-127 as a subnormal number
    const uint32_t s = max(byte << 7, 0x40u);
    return __byte_perm(s, s, 0x1010);
  }
  const float s = e4m3_to_f32(byte) * 0x1p112f;
  return pack_bf16x2_rn(s, s);
}

template <int MODE, int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(const KvAttentionArgs a, int group,
                                                                  uint8_t* __restrict__ ws, int inject_timeout) {
  using C = Pre<D>;
  int* counters = reinterpret_cast<int*>(ws);
  int* arrivals = reinterpret_cast<int*>(ws + kKvArrivals);
  float* results = reinterpret_cast<float*>(ws + kKvResults);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  uint64_t* sfull = reinterpret_cast<uint64_t*>(smem + C::offBar);  // [2] scores of a row tile
  uint64_t* pfull = sfull + 2;                                      // [2] its probabilities
  uint64_t* ofull = pfull + 2;                                      // [2] its output complete
  uint64_t* kfull = ofull + 2;                                      // [2] K tile dequantized
  uint64_t* kempty = kfull + 2;                                     // [2] and read
  uint64_t* vfull = kempty + 2;                                     // [2]
  uint64_t* vempty = vfull + 2;                                     // [2]
  uint64_t* qfull = vempty + 2;                                     // [2] query tile landed
  uint64_t* qempty = qfull + 2;                                     // [2] and read
  uint64_t* ifull = qempty + 2;                                     // [2] item known
  uint64_t* iempty = ifull + 2;                                     // [2] and done with
  uint64_t* inear = iempty + 2;                                     // the item in work nears its end
  uint64_t* xgive = inear + 1;                                      // [4] twins: a quadrant's second output complete
  uint64_t* xtake = xgive + 4;                                      // [4] and read
  uint64_t* never = xtake + 4;                                     // fault injection: nothing arrives here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  Item* items = reinterpret_cast<Item*>(smem + C::offBar + 512);   // [2]
  int* again = reinterpret_cast<int*>(smem + C::offBar + 912);     // [2] warps whose output passed fp32
  static_assert(512 + 2 * sizeof(Item) <= 656 && 656 + 4 * kSorted <= 912, "the small areas");
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + C::offPre);  // [kThreads + 1] items before a thread's requests
  int64_t* cost_before = reinterpret_cast<int64_t*>(smem + C::offTiles);  // [kThreads + 1] cost of the items before an item

  float* xch = reinterpret_cast<float*>(smem + C::offX);  // [4][2][32] references and sums of the second outputs

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], 4);
      mbar_init(&ofull[s], 1);
      mbar_init(&qfull[s], 64);
      mbar_init(&qempty[s], 1);
      mbar_init(&kfull[s], 128);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], 128);
      mbar_init(&vempty[s], 1);
      mbar_init(&ifull[s], 1);
      mbar_init(&iempty[s], kThreads / 32);
    }
    mbar_init(inear, 1);
    for (int w = 0; w < 4; ++w) {
      mbar_init(&xgive[w], 1);
      mbar_init(&xtake[w], 1);
    }
    mbar_init(never, 1);
    again[0] = again[1] = 0;
    fence_barrier_init();
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(tmem_slot)), "n"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Items before each thread's requests; requests outside the contract are reported by the first CTA.
  const int per = (a.batch + kThreads - 1) / kThreads;
  auto blocks_of = [&](int b) {
    const int q0 = __ldg(a.query_start + b), ql = __ldg(a.query_start + b + 1) - q0;
    if (ql <= 0 || ql > a.max_query_len || q0 < 0 || (int64_t)q0 + ql > a.tokens) return 0;
    return (ql * group + kRows - 1) / kRows;
  };
  // few requests: the longest first (what is left for the end is then short).  More: as they come.
  int* order = reinterpret_cast<int*>(smem + C::offBar + 656);  // [kSorted]
  const bool sorted = a.batch <= kSorted;
  if (sorted && (int)threadIdx.x < a.batch) {
    const int mine = __ldg(a.total_lens + threadIdx.x);
    int rank = 0;
    for (int b = 0; b < a.batch; ++b) {
      const int other = __ldg(a.total_lens + b);
      rank += other > mine || (other == mine && b < (int)threadIdx.x);
    }
    order[rank] = threadIdx.x;
  }
  __syncthreads();
  auto request = [&](int b) { return sorted ? order[b] : b; };
  __shared__ int64_t wsum[kThreads / 32];
  {
    int64_t sum = 0;
    for (int b = min(a.batch, (int)threadIdx.x * per); b < min(a.batch, ((int)threadIdx.x + 1) * per); ++b) {
      sum += blocks_of(request(b));
      if (blockIdx.x == 0) {
        const int ql = __ldg(a.query_start + b + 1) - __ldg(a.query_start + b);
        if (ql < 0 || (ql > 0 && blocks_of(b) == 0) || __ldg(a.total_lens + b) > (int64_t)a.max_pages * a.cache.page_size)
          record_error(a.err, kErrIndex);
      }
    }
    sum *= a.cache.kv_heads;
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    prefix[threadIdx.x + 1] = before + incl;
    if (threadIdx.x == 0) prefix[0] = 0;
  }
  const int page_size = a.cache.page_size, page_shift = 31 - __clz(page_size);
  __syncthreads();
  auto describe = [&](int64_t idx) {  // item idx, whole
    Item x = {};
    int lo = 0, hi = kThreads;  // the thread whose requests hold the item
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= idx) lo = mid; else hi = mid;
    }
    int64_t off = idx - prefix[lo];
    int r = lo * per, b = request(r), nb = blocks_of(b);
    while (off >= (int64_t)nb * a.cache.kv_heads) {
      off -= (int64_t)nb * a.cache.kv_heads;
      b = request(++r);
      nb = blocks_of(b);
    }
    const int rb = nb - 1 - (int)(off / a.cache.kv_heads);  // longest rows first
    x.b = b;
    x.h = (int)(off % a.cache.kv_heads);
    x.q0 = __ldg(a.query_start + b);
    x.qlen = __ldg(a.query_start + b + 1) - x.q0;
    x.total = max(min(__ldg(a.total_lens + b), a.max_pages * page_size), 0);  // (the differences below stay within 32 bits)
    x.row0 = rb * kRows;
    x.rows = x.qlen * group;
    const int pos0 = x.total - x.qlen + x.row0 / group;  // of the first row
    x.j0 = a.window > 0 ? max(pos0 + 1 - a.window, 0) / kKeys : 0;
    for (int i = 0; i < 2; ++i) {
      const int last = min(x.row0 + 128 * (i + 1), x.rows) - 1;  // the tile's last row
      const int end = last >= x.row0 + 128 * i ? x.total - x.qlen + last / group + 1 : 0;  // keys it sees
      x.n[i] = max((end + kKeys - 1) / kKeys - x.j0, 0);
    }
    x.pieces = 1;
    return x;
  };
  // Few items: their key tiles in one sequence, an equal share of it each CTA.  More: whole items, handed out in turn.
  const int64_t total_items = prefix[kThreads];
  const bool dealt = total_items <= kDealt;
  if (dealt) {
    int len = 0;
    if ((int)threadIdx.x < total_items) {
      const Item x = describe(threadIdx.x);
      len = PromptSplit::kCost + max(x.n[0], x.n[1]);
    }
    int64_t incl = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += wsum[w];
    cost_before[threadIdx.x + 1] = incl;
    if (threadIdx.x == 0) cost_before[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool failed = false;

  if (warp >= 17) {
    // ------------------------------------------------------ items, queries
    if (blockIdx.x == 0 && threadIdx.x == 17 * 32) report_expired(a);
    const int64_t cost = dealt ? cost_before[total_items] : 0;
    const int64_t shares = PromptSplit::shares(cost, total_items, (int)gridDim.x);
    auto item_at = [&](int64_t unit) {  // the item that holds a unit of cost
      int lo = 0, hi = (int)total_items;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cost_before[mid] <= unit) lo = mid; else hi = mid;
      }
      return lo;
    };
    auto start_of = [&](int64_t c) {  // of a CTA's share
      const int64_t cut = PromptSplit::cut(c, shares, cost);
      if (cut >= cost) return cost;
      const int i = item_at(cut);
      return PromptSplit::moved(cut, cost_before[i], cost_before[i + 1]);
    };
    int64_t pos = start_of(blockIdx.x);
    const int64_t end = start_of((int64_t)blockIdx.x + 1);
    bool over = false;  // no item left
    for (int k = 0;; ++k) {
      Item* it = &items[k & 1];
      if (warp == 17) {
        if (k >= 2) mbar_wait(&iempty[k & 1], ((k >> 1) - 1) & 1, a.err, failed);
        if (k >= 1) mbar_wait(inear, (k - 1) & 1, a.err, failed);
        Item x = {};
        int redo = 0;
        if (lane == 0) {
          if (MODE == 1 && k >= 2) redo = again[k & 1];  // item k - 2
          if (failed || over) {
            x.stop = 1;
          } else if (redo) {
          } else if (dealt) {
            x.stop = pos >= end;
            if (!x.stop) {
              const int i = item_at(pos);
              const int64_t at = cost_before[i], next = cost_before[i + 1], stop = min(next, end);
              x = describe(i);
              x.first = PromptSplit::first(at, next, shares, cost);
              x.piece = blockIdx.x - x.first;
              x.pieces = PromptSplit::last(at, next, shares, cost) - x.first + 1;
              const int skip = PromptSplit::skip(pos, at), len = PromptSplit::length(stop, at, skip);
              x.j0 += skip;
              for (int e = 0; e < 2; ++e) x.n[e] = min(max(x.n[e] - skip, 0), len);
              pos = stop;
            }
          } else {
            const int64_t idx = atomicAdd(counters, 1);
            if (idx < total_items) {
              x = describe(idx);
            } else {
              x.stop = 1;
              // the last CTA to find the work gone leaves the counters ready for the next call
              if (atomicAdd(counters + 1, 1) == (int)gridDim.x - 1) {
                counters[0] = 0;
                counters[1] = 0;
              }
            }
          }
          over = x.stop;
          x.tiles = max(x.n[0], x.n[1]);
          x.twin = x.row0 + 128 >= x.rows;  // no rows for the second tile: it takes every other key tile of the first's
          if (x.twin) {
            x.n[0] = (x.tiles + 1) / 2;
            x.n[1] = x.tiles / 2;
          }
        }
        if (MODE == 1) {
          int at = k & 1;
          if (k >= 1 && __shfl_sync(0xffffffffu, (int)(x.stop && !redo), 0)) {  // the last item may have to be done again
            mbar_wait(&iempty[(k - 1) & 1], ((k - 1) >> 1) & 1, a.err, failed);
            at = (k - 1) & 1;
            redo = again[at];
          }
          if (lane == 0 && redo && !failed) {
            x = items[at];
            x.again = redo;
            again[at] = 0;
          }
        }
        if (lane == 0) {
          *it = x;
          mbar_arrive(&ifull[k & 1]);
        }
        __syncwarp();
      }
      mbar_wait(&ifull[k & 1], (k >> 1) & 1, a.err, failed);
      const Item x = *it;
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[k & 1]);
      if (x.stop || failed) break;
      // 256 rows of D / 8 times 16 bytes, rows past the request's as zeros; a thread keeps its place in a row and steps
      // through the rows, so that the division by the group is done once.  Before the tiles are free: into L2.
      constexpr int kPer = 64 / (D / 8);
      const int t = threadIdx.x - 17 * 32, ch = t % (D / 8), r0 = t / (D / 8), head0 = (x.row0 + r0) % group;
      const uint16_t* src0 = a.q + (int64_t)(x.q0 + (x.row0 + r0) / group) * a.q_token + (int64_t)(x.h * group + head0) * a.q_head + ch * 8;
      const int64_t step = (int64_t)(kPer / group) * a.q_token + (int64_t)(kPer % group) * a.q_head, wrap = a.q_token - group * a.q_head;
      auto rows = [&](int to, int& r, int& head, const uint16_t*& src, auto each) {
#pragma unroll 4
        for (; r < to; r += kPer) {
          each(r, src, x.row0 + r < x.rows);
          src += step;
          head += kPer % group;
          if (head >= group) head -= group, src += wrap;
        }
      };
      int r = r0, head = head0;
      const uint16_t* src = src0;
      if (k > 0 && (ch & 7) == 0)
        rows(kRows, r, head, src, [&](int, const uint16_t* p, bool ok) {
          if (ok) asm volatile("prefetch.global.L2 [%0];" :: "l"(p));
        });
      r = r0, head = head0, src = src0;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        if (k > 0) mbar_wait(&qempty[i], (k - 1) & 1, a.err, failed);
        rows(128 * (i + 1), r, head, src, [&](int at, const uint16_t* p, bool ok) {
          const uint32_t dst = base + i * C::kQ + (ch >> 3) * C::kHalf + (at & 127) * 128 + (((ch & 7) ^ (at & 7)) << 4);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(ok ? p : a.q), "r"(ok ? 16 : 0) : "memory");
        });
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(&qfull[i])) : "memory");
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 16) {
    // ------------------------------------------------------------ MMA issue
    const uint32_t leader = elect_one_sync();
    if (leader && inject_timeout) {
      bool injected = false;  // separate flag: the injected expiry must not stop later waits
      mbar_wait(never, 0, a.err, injected, 2000000LL);
    }
    constexpr uint32_t idesc_s = (1u << 4) | (1u << 7) | (1u << 10) | ((kKeys >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t idesc_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
    int g = 0, u[2] = {0, 0};  // key tiles so far; probabilities consumed of each row tile
    for (int k = 0;; ++k) {
      mbar_wait(&ifull[k & 1], (k >> 1) & 1, a.err, failed);
      const Item x = items[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[k & 1]);
      if (x.stop || failed) break;
      const int n = x.tiles;
      auto scores = [&](int i, int kb) {
        const uint64_t qd = desc_k(base + (x.twin ? 0 : i) * C::kQ, 1024, 2), kd = desc_k(base + C::offK + kb * C::kKV, 1024, 2);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss(tmem + 128 * i, qd + (ks >> 2) * (C::kHalf >> 4) + 2 * (ks & 3), kd + (ks >> 2) * (C::kHalf >> 4) + 2 * (ks & 3),
                 idesc_s, ks > 0);
        tc_commit(&sfull[i]);
      };
      auto values = [&](int i, int vb, bool first) {
        const uint64_t vd = desc_mn(base + C::offV + vb * C::kKV, C::kHalf);
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_ts(tmem + C::kO + D * i, tmem + 128 * i + 8 * ks, vd + ks * (2048 >> 4), idesc_o, !first || ks > 0);
      };
      if (n == 0 && leader) mbar_arrive(inear);
      if (x.twin) {
        for (int i = 0; i < 2; ++i) {
          mbar_wait(&qfull[i], k & 1, a.err, failed);
          if (i < n) mbar_wait(&kfull[(g + i) & 1], ((g + i) >> 1) & 1, a.err, failed);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the copied queries, for the tensor core
          tc_fence_after();
          if (leader && i < n) {
            scores(i, (g + i) & 1);
            tc_commit(&kempty[(g + i) & 1]);
          }
        }
        if (leader && n <= 2) {
          tc_commit(&qempty[0]);
          tc_commit(&qempty[1]);
        }
        for (int j = 0; j < n; ++j, ++g) {
          const int i = j & 1;
          if (leader && j == max(n - 4, 0)) mbar_arrive(inear);
          mbar_wait(&vfull[g & 1], (g >> 1) & 1, a.err, failed);
          mbar_wait(&pfull[i], u[i] & 1, a.err, failed);
          ++u[i];
          tc_fence_after();
          if (leader) {
            values(i, g & 1, j < 2);
            if (j + 2 >= n) tc_commit(&ofull[i]);
            tc_commit(&vempty[g & 1]);
          }
          if (j + 2 < n) {
            mbar_wait(&kfull[g & 1], ((g + 2) >> 1) & 1, a.err, failed);
            tc_fence_after();
            if (leader) {
              scores(i, g & 1);
              tc_commit(&kempty[g & 1]);
              if (j + 3 == n) {
                tc_commit(&qempty[0]);
                tc_commit(&qempty[1]);
              }
            }
          }
          __syncwarp();
        }
        continue;
      }
      if (n > 0) mbar_wait(&kfull[g & 1], (g >> 1) & 1, a.err, failed);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mbar_wait(&qfull[i], k & 1, a.err, failed);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the copied queries, for the tensor core
        tc_fence_after();
        if (leader) {
          if (x.n[i] > 0) scores(i, g & 1);
          if (n <= 1) tc_commit(&qempty[i]);
        }
      }
      if (n > 0 && leader) tc_commit(&kempty[g & 1]);
      for (int j = 0; j < n; ++j, ++g) {
        if (leader && j == max(n - 4, 0)) mbar_arrive(inear);
        mbar_wait(&vfull[g & 1], (g >> 1) & 1, a.err, failed);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (j < x.n[i]) {
            mbar_wait(&pfull[i], u[i] & 1, a.err, failed);
            ++u[i];
            tc_fence_after();
            if (leader) {
              values(i, g & 1, j == 0);
              if (j == x.n[i] - 1) tc_commit(&ofull[i]);
            }
          }
          if (i == 1 && leader) tc_commit(&vempty[g & 1]);
          if (i == 0 && j + 1 < n) mbar_wait(&kfull[(g + 1) & 1], ((g + 1) >> 1) & 1, a.err, failed);
          tc_fence_after();
          if (j + 1 < x.n[i] && leader) scores(i, (g + 1) & 1);
          if (j + 2 == n && leader) tc_commit(&qempty[i]);
        }
        if (j + 1 < n && leader) tc_commit(&kempty[(g + 1) & 1]);
        __syncwarp();
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------- K and V
    const int t = threadIdx.x & 127;
    const bool is_v = warp >= 12;
    const uint32_t* codes = is_v ? a.cache.v_codes : a.cache.k_codes;
    const uint8_t* scales = is_v ? a.cache.v_scales : a.cache.k_scales;
    uint64_t* full = is_v ? vfull : kfull;
    uint64_t* empty = is_v ? vempty : kempty;
    const uint32_t tiles = base + (is_v ? C::offV : C::offK);
    constexpr int GR = MODE == 2 ? 16 : 32, SB = D / GR, W = D / 8;  // scale bytes, code words of a row
    int g = 0;
    for (int k = 0;; ++k) {
      mbar_wait(&ifull[k & 1], (k >> 1) & 1, a.err, failed);
      const Item x = items[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[k & 1]);
      if (x.stop || failed) break;
      const int n = x.tiles;
      const int32_t* table = a.block_table + (int64_t)x.b * a.table_stride;
      const int lo = a.window > 0 ? max(x.total - x.qlen + x.row0 / group + 1 - a.window, 0) : 0;
      const int hi = min(x.total, (x.j0 + n) * kKeys);
      auto row_of = [&](int j) -> int {  // cache row of this thread's key of tile j, or -1
        const int key = (x.j0 + j) * kKeys + t;
        if (j >= n || key < lo || key >= hi) return -1;
        int page = __ldg(table + (key >> page_shift));
        if (page < 0 || page >= a.cache.num_pages) {
          record_error(a.err, kErrIndex);
          page = 0;
        }
        return ((page * a.cache.kv_heads + x.h) << page_shift) + (key & (page_size - 1));
      };
      uint4 q[W / 4];
      uint32_t sc[(SB + 3) / 4];
      auto load = [&](int row) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
          q[i] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)row * W) + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < (SB + 3) / 4; ++i)  // (a key no row sees: a scale of zero, or 2^-127, whatever is stored)
          sc[i] = row < 0 ? 0u
                  : SB >= 4 ? __ldg(reinterpret_cast<const uint32_t*>(scales + (int64_t)row * SB) + i)
                            : (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(scales + (int64_t)row * SB));
      };
      int next = row_of(1);
      load(row_of(0));
      for (int j = 0; j < n; ++j, ++g) {
        if (g >= 2) mbar_wait(&empty[g & 1], ((g >> 1) - 1) & 1, a.err, failed);
        const uint32_t r = tiles + (g & 1) * C::kKV + t * 128;
#pragma unroll
        for (int i = 0; i < W; ++i) {  // word i: channels 8 i .. 8 i + 7
          const int sb = i * 8 / GR;
          const uint4 v = q[i / 4];
          const uint32_t w = (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
          const uint4 o = dequant8<MODE>(w, scale_pair<MODE>((sc[sb / 4] >> (8 * (sb & 3))) & 0xFFu));
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                       :: "r"(r + (i >> 3) * C::kHalf + (((i & 7) ^ (t & 7)) << 4)), "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w)
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(&full[g & 1]);
        load(next);
        next = row_of(j + 2);
      }
    }
  } else {
    // ------------------------------------------------------ softmax, output
    const int i = warp >> 2, row = threadIdx.x & 127;
    const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * i;
    const uint32_t to = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C::kO + D * i;
    const float gsk = (MODE == 2 && a.cache.gs_k) ? __ldg(a.cache.gs_k) : 1.0f;
    const float gsv = (MODE == 2 && a.cache.gs_v) ? __ldg(a.cache.gs_v) : 1.0f;
    const float cs = a.scale * 1.4426950408889634f * gsk;
    int use = 0, outs = 0, twins = 0;
    for (int k = 0;; ++k) {
      mbar_wait(&ifull[k & 1], (k >> 1) & 1, a.err, failed);
      const Item& x = items[k & 1];  // (read again at the item's end, which gives it back)
      if (x.stop || failed) break;
      int hi = INT32_MAX, lo = 0;  // keys lo .. hi - 1, counted from the piece's first (rows past the request's are not used)
      {
        const int rr = x.row0 + (x.twin ? 0 : 128 * i) + row, pos = x.total - x.qlen + rr / group;
        if (rr < x.rows) {
          hi = max(pos + 1, 0) - x.j0 * kKeys;
          lo = (a.window > 0 ? max(pos + 1 - a.window, 0) : 0) - x.j0 * kKeys;
        }
      }
      float m = kNone;
      uint64_t l2 = 0;  // the sum, in two halves
      const int n = x.n[i], first = x.twin ? i * kKeys : 0, step = x.twin ? 2 * kKeys : kKeys;
      const float low = MODE == 1 && x.again ? kLow : 0.f, far = MODE == 1 && x.again ? kLowFar : kFar;
      for (int j = 0; j < n; ++j, ++use) {
        const int key0 = first + j * step;
        const bool mask = __any_sync(0xffffffffu, key0 < lo || key0 + kKeys > hi);
        mbar_wait(&sfull[i], use & 1, a.err, failed);
        tc_fence_after();
        auto hide = [&](int c, uint32_t (&s)[32]) {  // scores of keys the row does not see
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int key = key0 + 32 * c + e;
            if (key >= hi || key < lo) s[e] = 0xFF800000u;
          }
        };
        auto top = [&](const uint32_t (&s)[32]) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = fmaxf(fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 8])), fmaxf(__uint_as_float(s[e + 16]), __uint_as_float(s[e + 24])));
          return fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
        };
        if (j == 0) {
          float t = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            uint32_t sa[32], sb[32];
            tmem_ld32(ts + 32 * c, sa);
            tmem_ld32(ts + 32 * c + 32, sb);
            ld_wait();
            if (mask) hide(c, sa), hide(c + 1, sb);
            t = fmaxf(t, fmaxf(top(sa), top(sb)));
          }
          m = fmaxf(t * cs, kNone) + low;
        }
        auto exps = [&](uint32_t (&v)[32], uint32_t (&p)[16]) -> uint64_t {
          const uint64_t c2 = pack2(cs, cs), m2 = pack2(-m, -m);
          uint64_t s0 = 0, s1 = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float p0, p1;
            unpack2(fma2(pack2(v[2 * e], v[2 * e + 1]), c2, m2), p0, p1);
            p0 = exp2_approx(p0);
            p1 = exp2_approx(p1);
            if (e & 1) s1 = add2(s1, pack2(p0, p1));
            else s0 = add2(s0, pack2(p0, p1));
            p[e] = pack_bf16x2_rn(p0, p1);
          }
          return add2(s0, s1);
        };
        auto chunk = [&](int c, uint32_t (&v)[32]) {  // thirty-two scores to probabilities
          if (mask) hide(c, v);
          uint32_t p[16];
          uint64_t sum = exps(v, p);
          float a0, a1;
          unpack2(sum, a0, a1);
          if (__any_sync(0xffffffffu, !(a0 + a1 <= far))) {
            // a score is far above the row's reference: move it; what the row has so far is scaled down,
            // these probabilities start over
            tmem_ld32(ts + 32 * c, v);
            ld_wait();
            if (mask) hide(c, v);
            float t = a0 + a1 <= far ? m : fmaxf(top(v) * cs + low, m);
            if (m != kNone) t = m + ceilf(t - m);  // by a power of two, so that no p is rounded a second time
            const float f = exp2f(m - t);
            m = t;
            l2 = mul2(l2, pack2(f, f));
            st_wait();  // (the earlier ones are in place before they are read back)
            for (int cc = 0; cc < 2 * c; ++cc) {  // earlier ones of this tile
              uint32_t o[8];
              tmem_ld8(ts + 8 * cc, o);
              ld_wait();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = pack_bf16x2_rn(bf16_lo(o[e]) * f, bf16_hi(o[e]) * f);
              tmem_st8(ts + 8 * cc, o);
            }
            if (j > 0)  // the output: no MMA is adding to it (this tile's scores were issued after the last that did)
              for (int cc = 0; cc < D / 8; ++cc) {
                uint32_t o[8];
                tmem_ld8(to + 8 * cc, o);
                ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st8(to + 8 * cc, o);
              }
            st_wait();
            sum = exps(v, p);
          }
          l2 = add2(l2, sum);
          tmem_st16(ts + 16 * c, p);
        };
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(ts + 32 * c, v);
          ld_wait();
          chunk(c, v);
        }
        st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[i]);
      }
      // ---- output
      float l, lh;
      unpack2(l2, l, lh);
      l += lh;
      const int rr = x.row0 + (x.twin ? 0 : 128 * i) + row, tok = rr / group;
      const bool real = rr < x.rows;
      const int64_t at = (int64_t)(x.q0 + tok) * a.q_heads + x.h * group + (rr - tok * group);
      if (n > 0) {
        mbar_wait(&ofull[i], outs & 1, a.err, failed);
        ++outs;
        tc_fence_after();
      }
      float w0 = 1.f, w1 = 0.f;
      if (x.twin) {  // both outputs of a row lie in the same lane: the first tile's warp joins them
        float* xc = xch + 64 * (warp & 3) + lane;
        if (i == 1) {
          xc[0] = m;
          xc[32] = l;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&xgive[warp & 3]);
          mbar_wait(&xtake[warp & 3], twins & 1, a.err, failed);
          tc_fence_after();
        } else {
          mbar_wait(&xgive[warp & 3], twins & 1, a.err, failed);
          tc_fence_after();
          const float top1 = xc[0], l1 = xc[32], t = fmaxf(m, top1);
          w0 = exp2f(m - t);
          w1 = exp2f(top1 - t);
          m = t;
          l = l * w0 + l1 * w1;
        }
        ++twins;
      }
      if (!x.twin || i == 0) {
      auto sums = [&](int p) { return results + (size_t)(2 * (x.first + p) + (p == 0)) * kSlotFloats<D> + 256 * D + 256 * i + row; };
      auto outputs = [&](int p, int c) {
        return reinterpret_cast<float4*>(results + (size_t)(2 * (x.first + p) + (p == 0)) * kSlotFloats<D>) + (i * (D / 4) + 8 * c) * 128 + row;
      };
      // Outputs are divided by the sum before anything is added to them.
      const bool whole = x.pieces == 1;
      const float inv = l == 0.f ? 0.f : (whole ? gsv : 1.0f) / l;
      w0 *= inv;
      w1 *= inv;
      uint64_t seen = 0;  // 0 times every output: NaN where one is not a number or passed fp32
      const bool mine = MODE != 1 || !x.again || (x.again >> warp & 1);  // (done again for another warp's rows)
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(to + 32 * c, o);
          ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * w0);
          if (x.twin && x.n[1] > 0)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t p[8];
              tmem_ld8(to + D + 32 * c + 8 * h, p);
              ld_wait();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[8 * h + e] = __float_as_uint(fmaf(__uint_as_float(p[e]), w1, __uint_as_float(o[8 * h + e])));
            }
          if (MODE == 1)
#pragma unroll
            for (int e = 0; e < 32; e += 2) seen = fma2(pack2(o[e], o[e + 1]), 0ull, seen);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (!mine) {
        } else if (!whole) {
          uint4* dst = reinterpret_cast<uint4*>(outputs(x.piece, c));
#pragma unroll
          for (int e = 0; e < 8; ++e) __stcg(dst + 128 * e, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
        } else if (real) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + at * D + 32 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t v[4];
#pragma unroll
            for (int h = 0; h < 4; ++h)
              v[h] = pack_bf16x2_rn(__uint_as_float(o[8 * e + 2 * h]), __uint_as_float(o[8 * e + 2 * h + 1]));
            dst[e] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
      if (x.twin) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&xtake[warp & 3]);
      }
      bool done = mine;
      if (MODE == 1 && !x.again) {
        float s0, s1;
        unpack2(seen, s0, s1);
        done = !__any_sync(0xffffffffu, real && l < INFINITY && !(s0 + s1 == 0.f));
        if (!done && lane == 0) atomicOr(&again[k & 1], 1 << warp);
      }
      bool last = whole && done;
      if (!whole && done) {  // the warp whose piece comes last joins the item's pieces of its rows, in their order
        __stcg(sums(x.piece), m);
        __stcg(sums(x.piece) + 128, l);
        __threadfence();
        __syncwarp();
        int* arrived = arrivals + 8 * x.first + warp;
        int before = 0;
        if (lane == 0) before = atomicAdd(arrived, 1);
        last = __shfl_sync(0xffffffffu, before, 0) == x.pieces - 1;
        if (last) {
          __threadfence();
          if (lane == 0) *arrived = 0;
          const int np = x.pieces;
          m = kNone;
#pragma unroll 4
          for (int p = 0; p < np; ++p) m = fmaxf(m, __ldcg(sums(p)));
          l = 0.f;
#pragma unroll 4
          for (int p = 0; p < np; ++p) l += __ldcg(sums(p) + 128) * exp2f(__ldcg(sums(p)) - m);
          const float join = l == 0.f ? 0.f : gsv / l;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float o[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0.f;
#pragma unroll 2
            for (int p = 0; p < np; ++p) {
              const float4* src = outputs(p, 0) + 512 * c;
              const float w = __ldcg(sums(p) + 128) * exp2f(__ldcg(sums(p)) - m) * join;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 v = __ldcg(src + 128 * e);
                o[4 * e] += w * v.x;
                o[4 * e + 1] += w * v.y;
                o[4 * e + 2] += w * v.z;
                o[4 * e + 3] += w * v.w;
              }
            }
            if (real) {
              uint4* dst = reinterpret_cast<uint4*>(a.out + at * D + 16 * c);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t v[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) v[h] = pack_bf16x2_rn(o[8 * e + 2 * h], o[8 * e + 2 * h + 1]);
                dst[e] = make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
          }
        }
      }
      if (last && real && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[k & 1]);
      tc_fence_before();
    }
  }
  if (failed) mark_expired(a);
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(512) : "memory");
  }
}

template <int MODE, int D>
cudaError_t launch(const DevInfo& d, const KvAttentionArgs& a, cudaStream_t s) {
  const int smem = (int)Pre<D>::kSmem + 1024;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(d, kv_prefill_kernel<MODE, D>, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(d.sm_count, kKvCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_prefill_kernel<MODE, D>, a, a.q_heads / a.cache.kv_heads,
                            static_cast<uint8_t*>(a.ws), a.inject_timeout);
}

}  // namespace

size_t kv_prefill_ws_bytes(int64_t head_dim) { return kKvResults + (size_t)(2 * kKvCtas * 256 * (head_dim + 2) * 4); }

bool kv_prefill_supported(int head_dim) { return head_dim == 64 || head_dim == 128; }

cudaError_t launch_kv_prefill(const DevInfo& d, const KvAttentionArgs& a, cudaStream_t s) {
  if (a.cache.mode == FP4_MODE_NVFP4)
    return a.cache.head_dim == 64 ? launch<2, 64>(d, a, s) : launch<2, 128>(d, a, s);
  return a.cache.head_dim == 64 ? launch<1, 64>(d, a, s) : launch<1, 128>(d, a, s);
}

}  // namespace fp4
