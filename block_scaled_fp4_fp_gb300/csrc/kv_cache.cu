// kv_cache.cu -- the paged 4-bit KV cache: the step's plan (block tables, slots
// and positions from request lengths) and the append (new K and V rows
// quantized into their slots).
//
// A cache layer is four matrices of the library's own formats: K codes and
// scales, V codes and scales, each with one row of head_dim elements per (page,
// kv head, slot) in that order and linear block scales.  Whatever reads such a
// matrix (fp4_dequantize among them) reads the cache.
#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "launch.h"

namespace fp4 {
namespace {

// ----------------------------------------------------------------- kv_plan --
//   old_b  = ceil(cached_b / P),  need_b = ceil((cached_b + new_b) / P), both at most the entries of a table row
//   page j of request b, old_b <= j < need_b, is free[first_b + j - old_b],
//   first_b = sum over b' < b of (need - old);  query_start = exclusive sum of new
//   token t of request r sits at position p = cached_r + t - query_start[r], slot
//   table[r, p / P] P + p mod P.
// Both sums are over the batch, so every CTA forms them itself (a block scan of
// a few thousand lengths costs about as much as one more launch would, and the
// CTAs then need no word from each other); it then writes its share of the tokens
// and of the fresh pages, finding the owner of each by binary search in shared
// memory.  A token's page is taken from the free list directly when it is
// fresh, never read back from the table another CTA may be writing.
// Bound by latency: one launch, two dependent global reads, one scan.  2.4 us for 64 requests of one token, 4.6 us for
// 1,000 requests of 64,000 tokens together (in a graph).
constexpr int kPlanThreads = 512;

__device__ __forceinline__ int64_t warp_scan_incl(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// the last index i in [0, n) with a[i] <= key (a non-decreasing, a[0] = 0, key >= 0): entries
// of empty requests repeat, so the last one is the owner
__device__ __forceinline__ int owner_of(const int* a, int n, int key) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= key) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(
    const int32_t* __restrict__ cached, const int32_t* __restrict__ fresh, int B, int page_shift,
    const int32_t* __restrict__ free_pages, int num_free, int32_t* table, int64_t table_stride, int max_pages,
    int32_t* __restrict__ total_lens, int32_t* __restrict__ query_start, int64_t* __restrict__ slot_map,
    int32_t* __restrict__ positions, int64_t T, int32_t* __restrict__ pages_taken, unsigned* __restrict__ err) {
  extern __shared__ int plan_smem[];
  int* start = plan_smem;      // [B]: first token of request b
  int* first = plan_smem + B;  // [B]: first fresh page of request b, as an index into the free list
  __shared__ int64_t warp_sum[2][kPlanThreads / 32];
  __shared__ int64_t carry[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the lengths may come from the previous kernel
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int pmask = (1 << page_shift) - 1;
  const bool lead = blockIdx.x == 0;
  bool bad = false;
  if (t < 2) carry[t] = 0;
  __syncthreads();
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + t;
    int64_t c = 0, n = 0;
    if (b < B) {
      c = __ldg(cached + b);
      n = __ldg(fresh + b);
      bad |= c < 0 || n < 0 || c + n > INT32_MAX;
      c = c < 0 ? 0 : c;
      n = n < 0 ? 0 : n;
      if (c + n > INT32_MAX) n = 0;
    }
    const int64_t old = (c + pmask) >> page_shift, need = (c + n + pmask) >> page_shift;
    bad |= need > max_pages;
    int64_t v[2] = {n, min(need, (int64_t)max_pages) - min(old, (int64_t)max_pages)}, incl[2];  // (no page without an entry)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      incl[k] = warp_scan_incl(v[k], lane);
      if (lane == 31) warp_sum[k][warp] = incl[k];
    }
    __syncthreads();
    if (warp < 2) {  // warp k scans the warps' sums of quantity k
      const int64_t w = lane < kPlanThreads / 32 ? warp_sum[warp][lane] : 0;
      const int64_t i = warp_scan_incl(w, lane);
      if (lane < kPlanThreads / 32) warp_sum[warp][lane] = carry[warp] + i - w;  // exclusive
      __syncwarp();
      if (lane == kPlanThreads / 32 - 1) carry[warp] += i;
    }
    __syncthreads();
    if (b < B) {
      const int64_t s = warp_sum[0][warp] + incl[0] - v[0], f = warp_sum[1][warp] + incl[1] - v[1];
      start[b] = (int)min(s, (int64_t)INT32_MAX);
      first[b] = (int)min(f, (int64_t)INT32_MAX);
      if (lead) {
        total_lens[b] = (int)(c + n);
        query_start[b] = start[b];
      }
    }
    __syncthreads();
  }
  const int64_t tokens = carry[0], taken = carry[1];
  bad |= tokens > T || taken > num_free;
  if (lead) {
    if (t == 0) {
      query_start[B] = (int)min(tokens, (int64_t)INT32_MAX);
      *pages_taken = (int)min(taken, (int64_t)num_free);
    }
    if (__syncthreads_or(bad) && t == 0) record_error(err, kErrIndex);
  }
  const int64_t step = (int64_t)gridDim.x * kPlanThreads, g0 = (int64_t)blockIdx.x * kPlanThreads + t;
  for (int64_t i = g0; i < T; i += step) {
    int64_t slot = -1;
    int pos = -1;
    if (i < tokens) {
      const int r = owner_of(start, B, (int)i);
      const int c = max(__ldg(cached + r), 0);
      pos = c + (int)i - start[r];
      const int j = pos >> page_shift, old = (int)(((int64_t)c + pmask) >> page_shift);
      if (j < max_pages) {
        const int f = first[r] + j - old;
        int page = -1;
        if (j < old)
          page = table[r * table_stride + j];
        else if (f < num_free)
          page = __ldg(free_pages + f);
        if (page >= 0) slot = ((int64_t)page << page_shift) + (pos & pmask);
      }
    }
    slot_map[i] = slot;
    positions[i] = pos;
  }
  const int64_t npages = min(taken, (int64_t)num_free);
  for (int64_t f = g0; f < npages; f += step) {
    const int r = owner_of(first, B, (int)f);
    const int c = max(__ldg(cached + r), 0);
    const int64_t j = (((int64_t)c + pmask) >> page_shift) + f - first[r];
    table[r * table_stride + j] = __ldg(free_pages + f);
  }
}

// --------------------------------------------------------------- kv_append --
// One thread per scale group: it reads the group's 16 (NVFP4) or 32 (MXFP4)
// bf16 values as 16-byte pieces, applies the quantizer's block rule
// (block_scale_rule) and writes the packed codes and the scale byte to the row
// of the token's slot.  Neighbouring threads hold neighbouring groups of one
// head, so a head's codes leave as one contiguous run.  Bound by HBM: 2 B read
// and 0.5 + 1/g B written per element.
// 17,500 tokens of 8 heads of 128, MXFP4: 13.5 us, 6.7 TB/s, the copy rate; one token of 40 heads: 1.8 us.
constexpr int kAppendThreads = 256;

template <int MODE>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(
    const uint16_t* __restrict__ k, int64_t k_token, int64_t k_head, const uint16_t* __restrict__ v, int64_t v_token,
    int64_t v_head, const int64_t* __restrict__ slot_map, int64_t T, KvCacheDesc c, unsigned* __restrict__ err) {
  constexpr int kGroup = MODE == 2 ? 16 : 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // k and v may come from the previous kernel
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const unsigned groups = (unsigned)(c.head_dim / kGroup), per_token = groups * (unsigned)c.kv_heads * 2u;
  const int64_t idx = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
  const int64_t t = idx / per_token;
  if (t >= T) return;
  unsigned rem = (unsigned)(idx - t * per_token);
  const unsigned g = rem % groups;
  rem /= groups;
  const unsigned h = rem % (unsigned)c.kv_heads;
  const bool is_v = rem >= (unsigned)c.kv_heads;
  const int64_t slot = __ldg(slot_map + t);
  if (slot < 0) return;  // a padding token
  const int64_t page = slot / c.page_size;
  if (page >= c.num_pages) {
    if (rem == 0 && g == 0) record_error(err, kErrIndex);
    return;
  }
  const uint16_t* src = (is_v ? v + t * v_token + h * v_head : k + t * k_token + h * k_head) + (int64_t)g * kGroup;
  uint4 x[kGroup / 8];
  uint32_t mb = 0;
#pragma unroll
  for (int i = 0; i < kGroup / 8; ++i) {
    x[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
    mb = max(mb, max_mag8(x[i]));
  }
  const float* gsp = is_v ? c.gs_v : c.gs_k;
  const float gs = (MODE == 2 && gsp) ? __ldg(gsp) : 1.0f;
  float mul, sval;
  uint32_t sbyte;
  block_scale_rule<MODE>(mb, gs, mul, sbyte, sval);
  uint32_t words[kGroup / 8];
#pragma unroll
  for (int i = 0; i < kGroup / 8; ++i) {
    const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __fmul_rn(bf16_lo(in[j]), mul);
      f[2 * j + 1] = __fmul_rn(bf16_hi(in[j]), mul);
    }
    words[i] = e2m1x8_rn(f);
  }
  const int64_t row = (page * c.kv_heads + h) * c.page_size + (slot - page * c.page_size);
  uint32_t* codes = (is_v ? c.v_codes : c.k_codes) + row * (c.head_dim / 8) + g * (kGroup / 8);
  if (MODE == 2)
    *reinterpret_cast<uint2*>(codes) = make_uint2(words[0], words[1]);
  else
    *reinterpret_cast<uint4*>(codes) = make_uint4(words[0], words[1], words[kGroup / 8 - 2], words[kGroup / 8 - 1]);
  (is_v ? c.v_scales : c.k_scales)[row * groups + g] = (uint8_t)sbyte;
}

}  // namespace

cudaError_t launch_kv_plan(const DevInfo& d, const int32_t* cached, const int32_t* fresh, int64_t B, int page_size,
                           const int32_t* free_pages, int64_t num_free, int32_t* table, int64_t table_stride,
                           int64_t max_pages, int32_t* total_lens, int32_t* query_start, int64_t* slot_map,
                           int32_t* positions, int64_t T, int32_t* pages_taken, cudaStream_t s) {
  const size_t smem = (size_t)B * 2 * sizeof(int);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(d, kv_plan_kernel, 2 * 4 * 16384, done);
  if (e != cudaSuccess) return e;
  int64_t grid = (T + kPlanThreads - 1) / kPlanThreads;
  if (grid > d.sm_count) grid = d.sm_count;
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(grid < 1 ? 1 : grid));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_plan_kernel, cached, fresh, (int)B, shift, free_pages, (int)num_free, table,
                            table_stride, (int)max_pages, total_lens, query_start, slot_map, positions, T, pages_taken,
                            d.err);
}

cudaError_t launch_kv_append(const DevInfo& d, const KvCacheDesc& c, const uint16_t* k, int64_t k_token, int64_t k_head,
                             const uint16_t* v, int64_t v_token, int64_t v_head, const int64_t* slot_map, int64_t T,
                             cudaStream_t s) {
  const int group = c.mode == FP4_MODE_NVFP4 ? 16 : 32;
  const int64_t items = T * (int64_t)(c.head_dim / group) * c.kv_heads * 2;
  const int64_t grid = (items + kAppendThreads - 1) / kAppendThreads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (c.mode == FP4_MODE_NVFP4)
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<2>, k, k_token, k_head, v, v_token, v_head, slot_map, T, c, d.err);
  return cudaLaunchKernelEx(&cfg, kv_append_kernel<1>, k, k_token, k_head, v, v_token, v_head, slot_map, T, c, d.err);
}

}  // namespace fp4
