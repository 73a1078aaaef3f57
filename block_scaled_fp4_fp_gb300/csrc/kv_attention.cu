// kv_attention.cu -- attention over the paged 4-bit cache, any head size: the
// kernel for head sizes without a tensor-core form.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j - m_i),
//   over the keys j <= pos_i (causal), j > pos_i - window, j < total_len.
// A block owns one (query token, query head); its warps take the visible keys 32 at a
// time, each with its own running maximum m, sum l and mean output.  Scores: a lane owns a key
// and reads its whole row (q is broadcast from shared memory), so that no score
// crosses a lane.  Outputs: a lane owns eight channels (one word of codes) of every
// KP-th of those keys, KP = 32 / (head_dim / 8), whose probabilities and rows come
// by shuffle.  The block joins the warps' (m, l, o) at the end.  All sums in fp32.
// Bound by instructions: about 5 an element of K and V for every query head (no group shares them).
// 8 requests of 4,000 tokens, 64 query heads on 8, NVFP4: heads of 96 129 us, of 32 50 us (a whole warp a key, with a
// five-step reduction of its score: 803 and 609); a 512-token prompt, 32 heads of 96 on 8: 245 us (1220).
#include <cuda.h>

#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "launch.h"

namespace fp4 {
namespace {

constexpr int kWarps = 8;

// eight codes -> eight values (exact)
__device__ __forceinline__ void e2m1x8(uint32_t w, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t h = e2m1x2_to_f16x2((w >> (8 * e)) & 0xFFu);
    v[2 * e] = f16_lo_to_f32(h);
    v[2 * e + 1] = f16_lo_to_f32(h >> 16);
  }
}

template <int MODE>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return MODE == 2 ? e4m3_to_f32(byte) : e8m0_to_f32(byte);
}

template <int MODE, int D>
__global__ void __launch_bounds__(kWarps * 32) kv_attention_any_kernel(KvAttentionArgs a) {
  constexpr int kGroup = MODE == 2 ? 16 : 32, kSB = D / kGroup;  // scale bytes of a row
  constexpr int W = D / 8, KP = 32 / W;                           // code words of a row; keys a warp adds up at a time
  __shared__ float sm[kWarps], sl[kWarps];
  __shared__ float so[kWarps][KP * D];
  __shared__ __align__(16) float sq[D];
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
  const float gsk = (MODE == 2 && c.gs_k) ? __ldg(c.gs_k) : 1.0f, gsv = (MODE == 2 && c.gs_v) ? __ldg(c.gs_v) : 1.0f;
  const float mult = a.scale * 1.4426950408889634f * gsk;  // scores in units of log 2
  const uint16_t* qrow = a.q + t * a.q_token + head * a.q_head;
  if (threadIdx.x < D) sq[threadIdx.x] = __uint_as_float((uint32_t)__ldg(qrow + threadIdx.x) << 16);
  __syncthreads();
  const int word = lane % W, sub = lane / W;  // (lanes from KP W on add nothing up)
  float o[8] = {};
  float m = -INFINITY, l = 0.f;
  for (int64_t j0 = begin + 32 * warp; j0 < end; j0 += 32 * kWarps) {
    const int n = (int)min((int64_t)32, end - j0);
    int row = 0;
    float s = -INFINITY;
    if (lane < n) {
      const int j = (int)(j0 + lane);
      int page = __ldg(a.block_table + (int64_t)b * a.table_stride + j / c.page_size);
      if (page < 0 || page >= c.num_pages) {
        record_error(a.err, kErrIndex);
        page = 0;
      }
      row = (page * c.kv_heads + kvh) * c.page_size + j % c.page_size;
      const uint4* kc = reinterpret_cast<const uint4*>(c.k_codes + (int64_t)row * W);
      const uint8_t* ks = c.k_scales + (int64_t)row * kSB;
      s = 0.f;
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint4 k4 = __ldg(kc + i);
        const uint32_t w4[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int g = 0; g < 32 / kGroup; ++g) {
          float x = 0.f;
#pragma unroll
          for (int e = 0; e < kGroup / 8; ++e) {
            const int at = g * (kGroup / 8) + e;
            float v[8];
            e2m1x8(w4[at], v);
            const float4 q0 = *reinterpret_cast<const float4*>(&sq[32 * i + 8 * at]);
            const float4 q1 = *reinterpret_cast<const float4*>(&sq[32 * i + 8 * at + 4]);
            x += v[0] * q0.x + v[1] * q0.y + v[2] * q0.z + v[3] * q0.w + v[4] * q1.x + v[5] * q1.y + v[6] * q1.z + v[7] * q1.w;
          }
          s = fmaf(x, scale_value<MODE>(__ldg(ks + i * (32 / kGroup) + g)), s);
        }
      }
      s *= mult;
    }
    float mn = fmaxf(m, s);
#pragma unroll
    for (int x = 16; x; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
    const float ref = mn == -INFINITY ? 0.f : mn;
    float p = exp2f(s - ref), sum = p;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    const float old = l * exp2f(m - ref);
    m = mn;
    l = old + sum;
    // o is the mean of the values so far, never their sum: V may be near fp32's largest numbers
    const float inv = l == 0.f ? 0.f : 1.0f / l, keep = old * inv;
    p *= inv;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= keep;
#pragma unroll 4
    for (int k = 0; k < n; k += KP) {
      const int key = k + sub;
      const float pk = __shfl_sync(0xffffffffu, p, key & 31);
      const int rk = __shfl_sync(0xffffffffu, row, key & 31);
      if (sub < KP && key < n) {
        float v[8];
        e2m1x8(__ldg(c.v_codes + (int64_t)rk * W + word), v);
        const float ps = pk * scale_value<MODE>(__ldg(c.v_scales + (int64_t)rk * kSB + word * 8 / kGroup));
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(ps, v[e], o[e]);
      }
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  if (sub < KP) {
#pragma unroll
    for (int e = 0; e < 8; ++e) so[warp][sub * D + word * 8 + e] = o[e];
  }
  __syncthreads();
  float mm = -INFINITY;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w]);
  const float ref = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
  for (int w = 0; w < kWarps; ++w) ll += sl[w] * exp2f(sm[w] - ref);
  const float inv = ll == 0.f ? 0.f : 1.0f / ll;
  if (threadIdx.x < D) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      float u = 0.f;
#pragma unroll
      for (int k = 0; k < KP; ++k) u += so[w][k * D + threadIdx.x];
      v += u * (sl[w] * exp2f(sm[w] - ref) * inv);
    }
    a.out[(t * a.q_heads + head) * D + threadIdx.x] = (uint16_t)f32_to_bf16_rn(v * gsv);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[t * a.q_heads + head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
}

template <int MODE, int D>
cudaError_t launch(const KvAttentionArgs& args, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)args.tokens, (unsigned)args.q_heads);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_attention_any_kernel<MODE, D>, args);
}

template <int MODE>
cudaError_t launch_any(const KvAttentionArgs& args, cudaStream_t s) {
  switch (args.cache.head_dim) {
    case 32: return launch<MODE, 32>(args, s);
    case 96: return launch<MODE, 96>(args, s);
    case 160: return launch<MODE, 160>(args, s);
    case 192: return launch<MODE, 192>(args, s);
    default: return launch<MODE, 224>(args, s);
  }
}

}  // namespace

// Query rows of a kv head, up to which the few-row kernel runs: it passes over the cache once for every sixteen, the
// many-row kernel fills two tiles of 128 whatever they are.  8 kv heads of 128, 8,000 tokens a request, NVFP4, few-row
// and many-row in us:  rows     4 requests   16 requests   64 requests
//                      9..16      26    48     61    90     192   296
//                      17..32     37    48    105    90     366   296
//                      33..48     48    48    148    91     543   297
//                      64         59    48    199    90     719   297
// The rule asks for the rows only: at 17..32 it is right for few requests and 17 to 24 % slow for many.
constexpr int64_t kFewRows = 32;

bool few_rows(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_query_len) {
  return kv_decode_supported((int)head_dim) &&
         (max_query_len * (q_heads / kv_heads) <= kFewRows || !kv_prefill_supported((int)head_dim));
}

size_t kv_attention_ws_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_query_len) {
  if (few_rows(q_heads, kv_heads, head_dim, max_query_len))
    return kv_decode_ws_bytes(q_heads, kv_heads, head_dim, max_query_len);
  if (kv_prefill_supported((int)head_dim))
    return kv_prefill_ws_bytes(head_dim);
  return 16;
}

cudaError_t launch_kv_attention(const DevInfo& d, const KvAttentionArgs& args, cudaStream_t s) {
  const KvCacheDesc& c = args.cache;
  if (few_rows(args.q_heads, c.kv_heads, c.head_dim, args.max_query_len)) return launch_kv_decode(d, args, s);
  if (kv_prefill_supported(c.head_dim)) return launch_kv_prefill(d, args, s);
  return c.mode == FP4_MODE_NVFP4 ? launch_any<2>(args, s) : launch_any<1>(args, s);
}

}  // namespace fp4
