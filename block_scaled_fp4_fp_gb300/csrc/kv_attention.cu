// kv_attention.cu -- attention over the paged 4-bit cache, any head size: the
// kernel for head sizes without a tensor-core form.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j - m_i),
//   over the keys j <= pos_i (causal), j > pos_i - window, j < total_len.
// A block owns one (query token, query head); its warps take the visible keys
// in turn, each with its own running maximum m, sum l and output in registers
// (lane e owns head_dim / 32 neighbouring channels), and the block joins the
// warps' (m, l, o) at the end.  All sums in fp32.  One key costs a warp a
// five-step shuffle reduction: bound by instruction latency, not by memory.
#include <cuda.h>

#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "launch.h"

namespace fp4 {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxPer = 8;  // channels per lane at most (head_dim <= 256)

// code `ch` of a row of packed e2m1 codes
__device__ __forceinline__ float e2m1_at(const uint32_t* row, int ch) {
  const uint32_t c = __ldg(row + (ch >> 3)) >> (4 * (ch & 7));
  return f16_lo_to_f32(e2m1x2_to_f16x2(c & 15u));
}

template <int MODE>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return MODE == 2 ? e4m3_to_f32(byte) : e8m0_to_f32(byte);
}

template <int MODE>
__global__ void __launch_bounds__(kWarps * 32) kv_attention_any_kernel(KvAttentionArgs a) {
  constexpr int kGroup = MODE == 2 ? 16 : 32;
  __shared__ float sm[kWarps], sl[kWarps];
  __shared__ float so[kWarps][32 * kMaxPer];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int head = blockIdx.y;
  const KvCacheDesc& c = a.cache;
  // the request that owns token t: the last b with query_start[b] <= t
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.query_start + mid) <= t) lo = mid; else hi = mid;
  }
  const int b = lo;
  const int q0 = __ldg(a.query_start + b), q1 = __ldg(a.query_start + b + 1);
  if (t < q0 || t >= q1) return;  // a padding token of the query buffer
  if (q1 - q0 > a.max_query_len) {
    if (threadIdx.x == 0) record_error(a.err, kErrIndex);
    return;
  }
  const int total = __ldg(a.total_lens + b);
  const int64_t pos = (int64_t)total - (q1 - q0) + (t - q0);
  int64_t end = pos + 1;
  if (end > (int64_t)a.max_pages * c.page_size) {
    if (threadIdx.x == 0) record_error(a.err, kErrIndex);
    end = (int64_t)a.max_pages * c.page_size;
  }
  const int64_t begin = a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
  const int kvh = head / (a.q_heads / c.kv_heads);
  const int per = c.head_dim / 32, groups = c.head_dim / kGroup;
  const float gsk = (MODE == 2 && c.gs_k) ? __ldg(c.gs_k) : 1.0f, gsv = (MODE == 2 && c.gs_v) ? __ldg(c.gs_v) : 1.0f;
  const float mult = a.scale * 1.4426950408889634f * gsk;  // scores in units of log 2
  const uint16_t* qrow = a.q + t * a.q_token + head * a.q_head;
  float q[kMaxPer], o[kMaxPer];
#pragma unroll
  for (int e = 0; e < kMaxPer; ++e) {
    q[e] = e < per ? __uint_as_float((uint32_t)__ldg(qrow + lane * per + e) << 16) : 0.f;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j = begin + warp; j < end; j += kWarps) {
    int page = __ldg(a.block_table + (int64_t)b * a.table_stride + j / c.page_size);
    if (page < 0 || page >= c.num_pages) {
      if (lane == 0) record_error(a.err, kErrIndex);
      page = 0;
    }
    const int64_t row = ((int64_t)page * c.kv_heads + kvh) * c.page_size + j % c.page_size;
    const uint32_t* kc = c.k_codes + row * (c.head_dim / 8);
    const uint8_t* ks = c.k_scales + row * groups;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kMaxPer; ++e)
      if (e < per) {
        const int ch = lane * per + e;
        s = fmaf(q[e], e2m1_at(kc, ch) * scale_value<MODE>(__ldg(ks + ch / kGroup)), s);
      }
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= mult;
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - ref), p = exp2f(s - ref);
    m = mn;
    l = l * alpha + p;
    const uint32_t* vc = c.v_codes + row * (c.head_dim / 8);
    const uint8_t* vs = c.v_scales + row * groups;
#pragma unroll
    for (int e = 0; e < kMaxPer; ++e)
      if (e < per) {
        const int ch = lane * per + e;
        o[e] = o[e] * alpha + p * (e2m1_at(vc, ch) * scale_value<MODE>(__ldg(vs + ch / kGroup)));
      }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kMaxPer; ++e)
    if (e < per) so[warp][lane * per + e] = o[e];
  __syncthreads();
  float mm = -INFINITY;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w]);
  const float ref = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
  for (int w = 0; w < kWarps; ++w) ll += sl[w] * exp2f(sm[w] - ref);
  for (int ch = threadIdx.x; ch < c.head_dim; ch += kWarps * 32) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += so[w][ch] * exp2f(sm[w] - ref);
    v = ll == 0.f ? 0.f : v / ll * gsv;
    a.out[(t * a.q_heads + head) * c.head_dim + ch] = (uint16_t)f32_to_bf16_rn(v);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[t * a.q_heads + head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
}

cudaError_t launch_any(const KvAttentionArgs& args, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)args.tokens, (unsigned)args.q_heads);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (args.cache.mode == FP4_MODE_NVFP4) return cudaLaunchKernelEx(&cfg, kv_attention_any_kernel<2>, args);
  return cudaLaunchKernelEx(&cfg, kv_attention_any_kernel<1>, args);
}

}  // namespace

// Query rows of a kv head, up to which the few-row kernel runs: it passes over the cache once for every sixteen, the
// many-row kernel fills a tile of 256 whatever they are.  8 kv heads of 128, 8,000 tokens a request, NVFP4, few-row and
// many-row in us:  rows     4 requests   16 requests   64 requests
//                  17..32     36    61    102   121     351   406
//                  33..48     47    61    143   121     517   408
//                  64         57    61    184   122     681   408
constexpr int64_t kFewRows = 32;

bool few_rows(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_query_len) {
  return kv_decode_supported((int)head_dim) &&
         (max_query_len * (q_heads / kv_heads) <= kFewRows || !kv_prefill_supported((int)head_dim));
}

size_t kv_attention_ws_bytes(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                             int64_t max_query_len) {
  if (few_rows(q_heads, kv_heads, head_dim, max_query_len))
    return kv_decode_ws_bytes(batch, q_heads, kv_heads, head_dim, max_query_len);
  if (kv_prefill_supported((int)head_dim))
    return kv_prefill_ws_bytes(head_dim);
  return 16;
}

cudaError_t launch_kv_attention(const DevInfo& d, const KvAttentionArgs& args, cudaStream_t s) {
  const KvCacheDesc& c = args.cache;
  if (few_rows(args.q_heads, c.kv_heads, c.head_dim, args.max_query_len)) return launch_kv_decode(d, args, s);
  if (kv_prefill_supported(c.head_dim)) return launch_kv_prefill(d, args, s);
  return launch_any(args, s);
}

}  // namespace fp4
