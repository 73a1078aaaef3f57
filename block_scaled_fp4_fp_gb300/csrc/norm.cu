// norm.cu -- root-mean-square norm with the residual's addition, out in bf16 and in the block-scaled 4-bit formats.
//   h = x + residual,  rstd = (mean h^2 + eps)^-1/2,  y = (h rstd) w;  sum_out = bf16(h), out = bf16(y),
//   xq and scales = the quantizer's block rule on the fp32 y.
#include <algorithm>

#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "launch.h"

namespace fp4 {
namespace {

// a + b = s + e exactly, whatever their order of size
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

// sum over the `width` lanes of an aligned group (a power of two), as a pair hi + lo
__device__ __forceinline__ void group_sum(float& hi, float& lo, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) {
    const float h2 = __shfl_xor_sync(0xffffffffu, hi, o), l2 = __shfl_xor_sync(0xffffffffu, lo, o);
    float e;
    two_sum(hi, h2, hi, e);
    lo = __fadd_rn(__fadd_rn(lo, l2), e);
  }
}

// 1 / sqrt((hi + lo) / n + eps): the hardware's approximation and one Newton step whose residual 1 - m r^2 is formed
// in two parts, which leaves little but the rounding of the result
__device__ __forceinline__ float inv_rms(float hi, float lo, float n, float eps) {
  const float q = __fdiv_rn(hi, n);
  const float rest = __fdividef(__fadd_rn(__fmaf_rn(-q, n, hi), lo), n);
  float m, e;
  two_sum(q, eps, m, e);
  e = __fadd_rn(e, rest);
  const float r = rsqrtf(m);
  const float p = __fmul_rn(m, r), pe = __fmaf_rn(m, r, -p);
  float d = __fmaf_rn(-p, r, 1.0f);
  d = __fmaf_rn(-pe, r, d);
  d = __fmaf_rn(-__fmul_rn(e, r), r, d);
  return __fmaf_rn(__fmul_rn(0.5f, r), d, r);
}

// A row belongs to `tpr` threads: a power of two of a warp's lanes (then a warp holds several rows), or a whole CTA.
// A thread's 16-byte pieces of the row are tpr pieces apart, so neighbouring lanes hold neighbouring pieces, and a
// scale group is 2 (NVFP4) or 4 (MXFP4) neighbouring lanes.  The row stays in registers from its one reading to its
// last writing; between them the sum of squares goes through the CTA.
//
// Precision: a thread's up to 32 squares are added in fp32, the threads' sums in pairs hi + lo, so that rstd is the
// rounding of its exact value but for a few rows in a hundred.  Elements next to a border of the 4-bit formats move
// by a whole step with rstd's last bit; the pairs cost six additions a step of the reduction.
// Squares outside fp32's range (|h| near 2^63 and above, or sums below 2^-80 beside an eps that does not hide them):
// the row is summed and scaled in fp64.
template <int V, int MODE>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const RmsNormArgs a, int tpr, int padded_rows, int padded_cols,
                                                        int word_scales) {
  constexpr int G = MODE == 2 ? 2 : 4;  // pieces of a scale group
  __shared__ float2 part[32];
  __shared__ double part64[32];
  __shared__ double rstd64;
  __shared__ float rstd_sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rpb = tpr > 32 ? 1 : (int)blockDim.x / tpr;
  const int sub = tpr > 32 ? 0 : (int)threadIdx.x / tpr;
  const int l = (int)threadIdx.x - sub * tpr;
  const int64_t row = (int64_t)blockIdx.x * rpb + sub;
  const int pieces = a.cols >> 3;
  const bool live = row < a.rows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  float h[V][8];
  uint4 xv[V], rv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = v * tpr + l;
    const bool in = live && p < pieces;
    xv[v] = in ? *reinterpret_cast<const uint4*>(a.x + row * a.x_stride + 8 * p) : make_uint4(0, 0, 0, 0);
    if (a.residual)
      rv[v] = in ? *reinterpret_cast<const uint4*>(a.residual + row * a.residual_stride + 8 * p) : make_uint4(0, 0, 0, 0);
  }
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t xw[4] = {xv[v].x, xv[v].y, xv[v].z, xv[v].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[v][2 * j] = bf16_lo(xw[j]);
      h[v][2 * j + 1] = bf16_hi(xw[j]);
    }
    if (a.residual) {
      const uint32_t rw[4] = {rv[v].x, rv[v].y, rv[v].z, rv[v].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[v][2 * j] = __fadd_rn(h[v][2 * j], bf16_lo(rw[j]));
        h[v][2 * j + 1] = __fadd_rn(h[v][2 * j + 1], bf16_hi(rw[j]));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s0 = __fmaf_rn(h[v][2 * j], h[v][2 * j], s0);
      s1 = __fmaf_rn(h[v][2 * j + 1], h[v][2 * j + 1], s1);
    }
  }
  if (a.sum_out) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = v * tpr + l;
      if (live && p < pieces)
        *reinterpret_cast<uint4*>(a.sum_out + row * a.sum_stride + 8 * p) =
            make_uint4(pack_bf16x2_rn(h[v][0], h[v][1]), pack_bf16x2_rn(h[v][2], h[v][3]),
                       pack_bf16x2_rn(h[v][4], h[v][5]), pack_bf16x2_rn(h[v][6], h[v][7]));
    }
  }
  // the row's sum of squares and 1 / rms
  float hi, lo;
  two_sum(s0, s1, hi, lo);
  group_sum(hi, lo, min(tpr, 32));
  float rstd;
  if (tpr > 32) {
    const int nw = (int)blockDim.x >> 5;
    if (lane == 0) part[warp] = make_float2(hi, lo);
    __syncthreads();
    if (warp == 0) {
      const float2 t = lane < nw ? part[lane] : make_float2(0.f, 0.f);
      hi = t.x;
      lo = t.y;
      group_sum(hi, lo, 32);
      if (lane == 0) {
        const bool wide = !(hi <= 0x1p120f) || (hi < 0x1p-80f && a.eps < 0x1p-50f);
        rstd_sh = wide ? -1.0f : inv_rms(hi, lo, (float)a.cols, a.eps);
      }
    }
    __syncthreads();
    rstd = rstd_sh;
  } else {
    const bool wide = !(hi <= 0x1p120f) || (hi < 0x1p-80f && a.eps < 0x1p-50f);
    rstd = wide ? -1.0f : inv_rms(hi, lo, (float)a.cols, a.eps);
  }
  // (a CTA's threads agree on their row's rstd; of rows in one warp, any wide one takes the warp along)
  const bool wide = rstd < 0.0f;
  if (tpr > 32 ? wide : __any_sync(0xffffffffu, wide)) {
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (double)h[v][j] * (double)h[v][j];
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tpr > 32) {
      if (lane == 0) part64[warp] = s;
      __syncthreads();
      if (threadIdx.x == 0) {
        s = 0.0;
        for (int w = 0; w < (int)blockDim.x >> 5; ++w) s += part64[w];
        rstd64 = s;
      }
      __syncthreads();
      s = rstd64;
    }
    const double m = s / a.cols + (double)a.eps;
    const double r = m == 0.0 ? 0.0 : 1.0 / sqrt(m);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = wide ? (float)((double)h[v][j] * r) : __fmul_rn(h[v][j], rstd);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = __fmul_rn(h[v][j], rstd);
  }
  const float gs = (MODE == 2 && a.gs) ? __ldg(a.gs) : 1.0f;
  const float div = __fmul_rn(6.0f, gs);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = v * tpr + l;
    const bool in = live && p < pieces;
    if (a.weight && p < pieces) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.weight) + p);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[v][2 * j] = __fmul_rn(h[v][2 * j], bf16_lo(ww[j]));
        h[v][2 * j + 1] = __fmul_rn(h[v][2 * j + 1], bf16_hi(ww[j]));
      }
    }
    if (a.out && in)
      *reinterpret_cast<uint4*>(a.out + row * a.cols + 8 * p) =
          make_uint4(pack_bf16x2_rn(h[v][0], h[v][1]), pack_bf16x2_rn(h[v][2], h[v][3]), pack_bf16x2_rn(h[v][4], h[v][5]),
                     pack_bf16x2_rn(h[v][6], h[v][7]));
    if (MODE != 0) {
      float b = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) b = fmaxf(b, fabsf(h[v][j]));
#pragma unroll
      for (int o = 1; o < G; o <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
      float mul;
      uint32_t sbyte;
      block_scale_rule_f32<MODE>(b, div, gs, mul, sbyte);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(h[v][j], mul);
      if (in) a.xq[row * pieces + p] = e2m1x8_rn(f);
      // scale bytes: four groups' in one word by their first lane, where the buffer allows words
      const int c = p / G;  // scale column
      if (!in) sbyte = 0;   // (the padding's bytes are 0)
      if (word_scales) {
        uint32_t w = sbyte | __shfl_down_sync(0xffffffffu, sbyte, G) << 8;
        w |= __shfl_down_sync(0xffffffffu, w, 2 * G) << 16;
        if ((l & (4 * G - 1)) == 0 && c < padded_cols && row < padded_rows) {
          const int64_t at = a.tiled ? tiled_scale_offset(row, c, padded_cols) : row * padded_cols + c;
          *reinterpret_cast<uint32_t*>(a.scales + at) = w;
        }
      } else if ((l & (G - 1)) == 0 && c < padded_cols && row < padded_rows) {
        a.scales[a.tiled ? tiled_scale_offset(row, c, padded_cols) : row * padded_cols + c] = (uint8_t)sbyte;
      }
    }
  }
}

template <int V>
cudaError_t launch_v(const cudaLaunchConfig_t& cfg, const RmsNormArgs& a, int tpr, int prows, int pcols, int words) {
  if (!a.xq) return cudaLaunchKernelEx(&cfg, rms_norm_kernel<V, 0>, a, tpr, prows, pcols, words);
  if (a.mode == FP4_MODE_NVFP4) return cudaLaunchKernelEx(&cfg, rms_norm_kernel<V, 2>, a, tpr, prows, pcols, words);
  return cudaLaunchKernelEx(&cfg, rms_norm_kernel<V, 1>, a, tpr, prows, pcols, words);
}

}  // namespace

cudaError_t launch_rms_norm(const DevInfo& d, const RmsNormArgs& a, cudaStream_t s) {
  (void)d;
  const int group = a.mode == FP4_MODE_NVFP4 ? 16 : 32;
  int pieces = a.cols / 8, prows = a.rows, pcols = 0, words = 0, least = 4;
  if (a.xq) {
    const int scols = a.cols / group;
    pcols = a.tiled ? (scols + 3) / 4 * 4 : scols;
    prows = a.tiled ? (a.rows + 127) / 128 * 128 : a.rows;
    words = pcols % 4 == 0 && (reinterpret_cast<uintptr_t>(a.scales) & 3) == 0;
    least = group / 8 * 4;                            // the lanes of four scales
    pieces = (pieces + least - 1) / least * least;    // (whole words of scales, and the padding's)
  }
  int V = 1;
  while (V < 4 && pieces > 1024 * V) V *= 2;
  const int need = (pieces + V - 1) / V;
  int tpr = (need + 31) / 32 * 32;
  if (need <= 32)
    for (tpr = least; tpr < need;) tpr *= 2;
  cudaLaunchConfig_t cfg = {};
  const int block = tpr > 32 ? tpr : 128, rpb = tpr > 32 ? 1 : block / tpr;
  cfg.gridDim = dim3((unsigned)(((int64_t)prows + rpb - 1) / rpb));
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (V == 1) return launch_v<1>(cfg, a, tpr, prows, pcols, words);
  if (V == 2) return launch_v<2>(cfg, a, tpr, prows, pcols, words);
  return launch_v<4>(cfg, a, tpr, prows, pcols, words);
}

}  // namespace fp4
