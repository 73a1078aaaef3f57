// norm.cu -- root-mean-square norm with the residual's addition, out in bf16 and in the block-scaled 4-bit formats.
//   h = x + residual,  rstd = (mean h^2 + eps)^-1/2,  y = (h rstd) w;  sum_out = bf16(h), out = bf16(y),
//   xq and scales = the quantizer's block rule on the fp32 y.
#include <algorithm>

#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "launch.h"
#include "packed.cuh"

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

// The same over a whole warp in two reductions instead of five steps of eleven instructions: the lanes' sums (>= 0, without
// a second part) as whole numbers of 2^-26 of the largest's power of two, added as integers.  Each is off by half a unit, as
// much as 2^-27 of the largest one; the sum of 32 of about the same size by some 2^-30.
__device__ __forceinline__ void warp_sum(float s, float& hi, float& lo) {
  const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(s));
  if (most >= 0x7f800000u) {  // overflown, or NaN
    hi = __uint_as_float(most);
    lo = 0.0f;
    return;
  }
  const int e = max((int)(most >> 23) - 127, -90);  // sums of this size say nothing (out_of_range, or a large eps)
  const uint32_t t = __reduce_add_sync(0xffffffffu, __float2uint_rn(__fmul_rn(s, exp2i_f32(26 - e))));
  hi = __uint2float_rz(t);
  lo = (float)(int)(t - __float2uint_rz(hi));
  const float unit = exp2i_f32(e - 26);
  hi *= unit;
  lo *= unit;
}

// The lanes' sums in two parts (the second at most 2^-16 of the first), exactly enough: the first as whole numbers of 2^-26
// of the largest's power of two, what is left and the second parts as whole numbers of 2^-14 of those.  Off by no more than
// 2^-36 of the largest.
__device__ __forceinline__ void warp_sum_exactly(float& hi, float& lo) {
  const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(hi));
  if (most >= 0x7f800000u) {  // overflown, or NaN
    hi = __uint_as_float(most);
    lo = 0.0f;
    return;
  }
  const int e = max((int)(most >> 23) - 127, -90);
  const float up = exp2i_f32(26 - e), v = __fmul_rn(hi, up);
  const uint32_t n = __float2uint_rz(v);
  const float rest = __fmaf_rn(lo, up, __fsub_rn(v, __uint2float_rz(n)));  // (n: 24 bits, so the difference is exact)
  const uint32_t t = __reduce_add_sync(0xffffffffu, n);
  const int r = __reduce_add_sync(0xffffffffu, __float2int_rn(__fmul_rn(rest, 0x1p14f)));
  hi = __uint2float_rz(t);
  lo = __fmaf_rn((float)r, 0x1p-14f, (float)(int)(t - __float2uint_rz(hi)));
  const float unit = exp2i_f32(e - 26);
  hi *= unit;
  lo *= unit;
}

// 1 / sqrt(m + e), e small beside m: the hardware's approximation and one Newton step whose residual 1 - (m + e) r^2 is
// formed in two parts, which leaves little but the rounding of the result
__device__ __forceinline__ float inv_sqrt(float m, float e) {
  const float r = rsqrtf(m);
  const float p = __fmul_rn(m, r), pe = __fmaf_rn(m, r, -p);
  float d = __fmaf_rn(-p, r, 1.0f);
  d = __fmaf_rn(-pe, r, d);
  d = __fmaf_rn(-__fmul_rn(e, r), r, d);
  return __fmaf_rn(__fmul_rn(0.5f, r), d, r);
}

// 1 / sqrt((hi + lo) / n + eps) (inv_n: 1 / n, whose rounding the remainder makes good)
__device__ __forceinline__ float inv_rms(float hi, float lo, float n, float inv_n, float eps) {
  const float q = __fmul_rn(hi, inv_n);
  const float rest = __fmul_rn(__fadd_rn(__fmaf_rn(-q, n, hi), lo), inv_n);
  float m, e;
  two_sum(q, eps, m, e);
  return inv_sqrt(m, __fadd_rn(e, rest));
}

// 1 / sqrt(m) = r 2^k of any m >= 0 in fp64 (0 for m = 0): r in [1/2, 1], k in two halves that fp32 holds as powers
__device__ __forceinline__ void inv_sqrt_wide(double m, float& r, float& p0, float& p1) {
  p0 = p1 = 1.0f;
  r = 0.0f;  // (an infinite m too)
  if (m != m) r = __int_as_float(0x7fffffff);
  if (!(m > 0.0) || m > 1.0e300) return;
  const int e = ((__double2hiint(m) >> 20) - 1023) & ~1;  // even; m 2^-e is in [1, 4)
  const double f = m * __hiloint2double((1023 - e) << 20, 0);
  const float hi = (float)f;
  r = inv_sqrt(hi, (float)(f - hi));
  const int k = -(e / 2);
  p0 = exp2i_f32(k / 2);
  p1 = exp2i_f32(k - k / 2);
}

// Sums of squares that say nothing: overflown (or NaN), or made of squares that may have vanished, with no eps above them.
__device__ __forceinline__ bool out_of_range(float sum, float eps) {
  return !(sum <= 0x1p120f) || (sum < 0x1p-80f && eps < 0x1p-50f);
}

// ------------------------------------------------------------------ the row --
// A row belongs to `tpr` threads: a power of two of a warp's lanes (then a warp holds several rows), or a whole CTA.
// A thread holds U chunks of 16 elements, tpr chunks apart, so neighbouring lanes hold neighbouring chunks; a
// chunk is a scale group of NVFP4, two lanes' chunks are one of MXFP4.  The row stays in registers from its one reading
// to its last writing; between them the sum of squares goes through the CTA.
//
// Precision: a thread's up to 32 squares are added in two chains in fp32, the threads' sums as integers or in pairs hi + lo.
// What the chains round away averages out over a row's threads, but not where one thread holds most of the sum (a massive
// channel: what is added behind its square loses its low bits; 4e-7 of the sum, three units of 1/rms): a warp with a
// thread of more than a quarter of the warp's sum, or half of a row that is part of a warp, adds up again with nothing lost.
// The sum is then off by less than 2^-23 of itself (2^-22 in rows of up to 1024 columns several of which are massive), and 1/rms
// is the rounding of its exact value in nine rows of ten, else the number beside it.  (bf16 results do not feel that; elements
// next to a border of the 4-bit formats move by a whole step.)  4096 x 5120 to NVFP4 without a residual: 15.7 us, with a massive
// channel 16.1, and 18.1 where every warp adds up exactly, which makes 1/rms the rounding in every row.
// Squares outside fp32's range (|h| near 2^60 and above, or sums below 2^-80 beside an eps that does not hide them):
// the row is summed again in fp64.
struct Shared {
  float2 part[32];
  double part64[32];
  double sum64;
  float rstd;
};

template <int U>
struct Row {
  uint64_t h[U][8];

  __device__ __forceinline__ void set(int u, int i, uint4 v) {  // elements 8 i .. 8 i + 7 of chunk u
    h[u][4 * i] = widen(v.x);
    h[u][4 * i + 1] = widen(v.y);
    h[u][4 * i + 2] = widen(v.z);
    h[u][4 * i + 3] = widen(v.w);
  }
  __device__ __forceinline__ void add(int u, int i, uint4 v) {
    h[u][4 * i] = add2(h[u][4 * i], widen(v.x));
    h[u][4 * i + 1] = add2(h[u][4 * i + 1], widen(v.y));
    h[u][4 * i + 2] = add2(h[u][4 * i + 2], widen(v.z));
    h[u][4 * i + 3] = add2(h[u][4 * i + 3], widen(v.w));
  }
  // the thread's sum of squares
  __device__ __forceinline__ float squares() const {
    uint64_t s = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma2(h[u][j], h[u][j], s);
    return __fadd_rn(lo_of(s), hi_of(s));
  }
  // The same in two parts, with nothing lost: sums that start from a power of two no smaller than any of the squares never
  // meet a larger one, so what a step rounds away, h^2 + (s - t), comes out exactly, and so does the power's subtraction.
  // (Squares near fp32's end make it NaN: out_of_range then, as they are.)
  __device__ __forceinline__ void squares_exactly(float& hi, float& lo) const {
    float m = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max_abs3(m, lo_of(h[u][j]), hi_of(h[u][j]));
    const int e = 2 * (int)(__float_as_uint(m) >> 23) - 125;
    const uint64_t base = pair_of(__uint_as_float((uint32_t)min(max(e, 1), 255) << 23)), minus = pair_of(-1.0f);
    uint64_t s = base, err = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint64_t t = fma2(h[u][j], h[u][j], s);
        err = add2(err, fma2(h[u][j], h[u][j], fma2(t, minus, s)));
        s = t;
      }
    s = fma2(base, minus, s);
    two_sum(lo_of(s), hi_of(s), hi, lo);
    lo = __fadd_rn(lo, __fadd_rn(lo_of(err), hi_of(err)));
  }
  // rstd (or, in fp64, a row that fp32's squares do not hold: then scaled by its power of two) for this thread's row
  template <bool CTA>
  __device__ __forceinline__ float scale(float rstd, const RmsNormArgs& a, int tpr, double inv_n, Shared& sh) {
    // (a CTA's threads agree on their row's rstd; of rows in one warp, any wide one takes the warp along)
    const bool wide = rstd < 0.0f;
    if (!(CTA ? wide : __any_sync(0xffffffffu, wide))) return rstd;
    double s = 0.0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double p = lo_of(h[u][j]), q = hi_of(h[u][j]);
        s += p * p + q * q;
      }
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (CTA) {
      if ((threadIdx.x & 31) == 0) sh.part64[threadIdx.x >> 5] = s;
      __syncthreads();
      if (threadIdx.x == 0) {
        s = 0.0;
        for (int w = 0; w < (int)blockDim.x >> 5; ++w) s += sh.part64[w];
        sh.sum64 = s;
      }
      __syncthreads();
      s = sh.sum64;
    }
    if (!wide) return rstd;
    float r, p0, p1;
    inv_sqrt_wide(s * inv_n + (double)a.eps, r, p0, p1);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = mul2(mul2(h[u][j], pair_of(p0)), pair_of(p1));
    return r;
  }
  __device__ __forceinline__ void write_sum(const RmsNormArgs& a, int row, bool live, int l, int tpr, int pieces) const {
    uint4* sr = reinterpret_cast<uint4*>(a.sum_out + (int64_t)row * a.sum_stride);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = 2 * (u * tpr + l);
      if (live && p < pieces) sr[p] = narrow(h[u]);
      if (live && p + 1 < pieces) sr[p + 1] = narrow(h[u] + 4);
    }
  }
  // y, and what is wanted of it
  template <int MODE>
  __device__ __forceinline__ void write(const RmsNormArgs& a, float rstd, const BlockScale& rule, int row,
                                        bool live, int l, int tpr, int pieces, int padded_rows, int padded_cols,
                                        int word_scales) {
    constexpr int G = MODE == 1 ? 2 : 1;  // chunks of a scale group
    const uint64_t r2 = pair_of(rstd);
    uint4* out = reinterpret_cast<uint4*>(a.out + (int64_t)row * a.cols);
    uint32_t* codes = a.xq + (int64_t)row * pieces;
    uint8_t* scales = a.tiled ? a.scales + (int64_t)(row >> 7) * (padded_cols << 7) + ((row & 31) << 4) + ((row & 127) >> 5 << 2)
                              : a.scales + (int64_t)row * padded_cols;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ch = u * tpr + l, p = 2 * ch;
      const bool in = live && p < pieces;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[u][j] = mul2(h[u][j], r2);
      if (a.weight) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (p + i < pieces) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.weight) + p + i);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) h[u][4 * i + j] = mul2(h[u][4 * i + j], widen(ww[j]));
          }
      }
      if (a.out) {
        if (in) out[p] = narrow(h[u]);
        if (live && p + 1 < pieces) out[p + 1] = narrow(h[u] + 4);
      }
      if (MODE != 0) {
        float b = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) b = max_abs3(b, lo_of(h[u][j]), hi_of(h[u][j]));
        if (MODE == 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 1));
        float mul;
        uint32_t sbyte;
        block_scale_rule_f32<MODE>(b, rule, mul, sbyte);
        const uint64_t m2 = pair_of(mul);
        float f[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint64_t v = mul2(h[u][j], m2);
          f[j >> 2][2 * (j & 3)] = lo_of(v);
          f[j >> 2][2 * (j & 3) + 1] = hi_of(v);
        }
        if (in) *reinterpret_cast<uint2*>(codes + p) = make_uint2(e2m1x8_rn(f[0]), e2m1x8_rn(f[1]));  // (4-bit rows are whole chunks)
        // scale bytes: four groups' in one word by their first lane, where the buffer allows words
        const int c = ch / G;  // scale column
        if (!in) sbyte = 0;    // (the padding's bytes are 0)
        if (word_scales) {
          uint32_t w = sbyte | __shfl_down_sync(0xffffffffu, sbyte, G) << 8;
          w |= __shfl_down_sync(0xffffffffu, w, 2 * G) << 16;
          if ((l & (4 * G - 1)) == 0 && c < padded_cols && row < padded_rows)
            *reinterpret_cast<uint32_t*>(scales + (a.tiled ? c << 7 : c)) = w;
        } else if ((l & (G - 1)) == 0 && c < padded_cols && row < padded_rows) {
          scales[a.tiled ? ((c >> 2) << 9) + (c & 3) : c] = (uint8_t)sbyte;
        }
      }
    }
  }
};

// Bound by HBM in bf16 with a residual (4096 x 5120: 27.5 us, 6.1 TB/s).  Without one, and with 4-bit results, by latency:
// registers hold the warps to half of what an SM takes, each CTA loads, sums, computes and stores one after the other, and
// while it computes it has nothing in flight; loads are the first stall by a factor of three, half of the issue slots are used
// (4096 x 5120 with a residual to NVFP4: 24.8 us, 5.5 TB/s, without one 15.75; 8001 x 2880 to MXFP4: 16.7 us, 3.5 TB/s).
// One row by latency alone (1 x 5120: 2.2 us).
// Tried: CTAs that stay, the next row on its way into shared memory by bulk copy (31.8 us in bf16 with a residual, 28.3 to NVFP4;
// without one 17.7 against 18.2 then); four chunks a thread (31 and 34 us; without a residual, x kept as bf16 and widened twice,
// 24 against 16.4 in bf16: spills); loads past L1 (within 2 %).
template <int U, int MODE, bool CTA>
__global__ void __launch_bounds__(CTA ? 1024 : 128) rms_norm_kernel(const RmsNormArgs a, int tpr, int padded_rows,
                                                                     int padded_cols, int word_scales, double inv_n) {
  __shared__ Shared sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int sub = CTA ? 0 : (int)threadIdx.x / tpr, l = (int)threadIdx.x - sub * tpr;
  const int row = CTA ? (int)blockIdx.x : (int)blockIdx.x * ((int)blockDim.x / tpr) + sub;
  const int pieces = a.cols >> 3;  // of 16 bytes
  const bool live = row < a.rows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  Row<U> r;
  {
    const uint4* xr = reinterpret_cast<const uint4*>(a.x + (int64_t)row * a.x_stride);
    const uint4* rr = reinterpret_cast<const uint4*>(a.residual + (int64_t)row * a.residual_stride);
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 xv[U][2], rv[U][2];
    if (CTA && live && pieces == 2 * U * tpr) {  // (no select a load)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) xv[u][i] = xr[2 * (u * tpr + l) + i];
      if (a.residual) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) rv[u][i] = rr[2 * (u * tpr + l) + i];
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = 2 * (u * tpr + l) + i;
          const bool in = live && p < pieces;
          xv[u][i] = in ? xr[p] : none;
          rv[u][i] = a.residual && in ? rr[p] : none;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        r.set(u, i, xv[u][i]);
        if (a.residual) r.add(u, i, rv[u][i]);
      }
  }
  const float own = r.squares();
  float hi = own, lo = 0.0f;
  if (a.sum_out) r.write_sum(a, row, live, l, tpr, pieces);
  if (CTA || tpr == 32)
    warp_sum(own, hi, lo);
  else
    group_sum(hi, lo, tpr);
  if (const unsigned votes = __ballot_sync(0xffffffffu, own * (CTA || tpr == 32 ? 4.0f : 2.0f) > hi)) {
    float whole, rest;
    r.squares_exactly(whole, rest);
    if (CTA || tpr == 32)
      warp_sum_exactly(whole, rest);
    else
      group_sum(whole, rest, tpr);
    // (a row that shares its warp goes by its own vote: its bits do not depend on its neighbours)
    if (CTA || tpr == 32 || votes >> (lane & -tpr) & ((1u << tpr) - 1)) {
      hi = whole;
      lo = rest;
    }
  }
  // The warps' sums: added up by every warp for itself (each aligned group of lanes all of them), which saves a barrier, or
  // with 4-bit results, where each warp has more to do, by the first warp (4096 x 5120 to NVFP4: 15.7 us against 17.2 without a
  // residual, 24.9 against 25.2 with one; to bf16 16.6 against 16.4, and 28.0 against 27.6).
  constexpr bool kEvery = MODE == 0;
  if (CTA) {
    const int nw = (int)blockDim.x >> 5, width = nw <= 4 ? 4 : nw <= 8 ? 8 : nw <= 16 ? 16 : 32, w = lane & (width - 1);
    if (lane == 0) sh.part[warp] = make_float2(hi, lo);
    __syncthreads();
    if (kEvery || warp == 0) {
      const float2 t = w < nw ? sh.part[w] : make_float2(0.f, 0.f);
      hi = t.x;
      lo = t.y;
      group_sum(hi, lo, width);
    }
  }
  float rstd = 0.0f;
  if (!CTA || kEvery || warp == 0)
    rstd = out_of_range(hi, a.eps) ? -1.0f : inv_rms(hi, lo, (float)a.cols, (float)inv_n, a.eps);
  if (CTA && !kEvery) {
    if (threadIdx.x == 0) sh.rstd = rstd;
    __syncthreads();
    rstd = sh.rstd;
  }
  rstd = r.template scale<CTA>(rstd, a, tpr, inv_n, sh);
  r.template write<MODE>(a, rstd, block_scale<MODE>(a.gs), row, live, l, tpr, pieces, padded_rows, padded_cols, word_scales);
}

template <int U, bool CTA>
cudaError_t launch_u(const cudaLaunchConfig_t& cfg, const RmsNormArgs& a, int tpr, int prows, int pcols, int words) {
  const double inv_n = 1.0 / a.cols;
  if (!a.xq) return cudaLaunchKernelEx(&cfg, rms_norm_kernel<U, 0, CTA>, a, tpr, prows, pcols, words, inv_n);
  if (a.mode == FP4_MODE_NVFP4) return cudaLaunchKernelEx(&cfg, rms_norm_kernel<U, 2, CTA>, a, tpr, prows, pcols, words, inv_n);
  return cudaLaunchKernelEx(&cfg, rms_norm_kernel<U, 1, CTA>, a, tpr, prows, pcols, words, inv_n);
}

}  // namespace

cudaError_t launch_rms_norm(const DevInfo& d, const RmsNormArgs& a, cudaStream_t s) {
  int chunks = (a.cols + 15) / 16, prows = a.rows, pcols = 0, words = 0, least = 1;
  if (a.xq) {
    const int scols = a.cols / (a.mode == FP4_MODE_NVFP4 ? 16 : 32);
    pcols = a.tiled ? (scols + 3) / 4 * 4 : scols;
    prows = a.tiled ? (a.rows + 127) / 128 * 128 : a.rows;
    words = pcols % 4 == 0 && (reinterpret_cast<uintptr_t>(a.scales) & 3) == 0;
    least = a.mode == FP4_MODE_NVFP4 ? 4 : 8;       // the lanes of four scales
    chunks = (chunks + least - 1) / least * least;  // (whole words of scales, and the padding's)
  }
  // Two chunks a thread where the rows fill the GPU anyway (4096 x 5120: 27.6 us against 28.9 in bf16, 26.5 against 31.8 to
  // NVFP4, when both were measured), one where latency counts (1 x 5120: 2.4 us against 2.7, 2.8 against 3.3); more than 1024
  // chunks need two.
  const int U = chunks > 1024 || (int64_t)chunks * prows >= (int64_t)d.sm_count * 1024 ? 2 : 1;
  const int need = (chunks + U - 1) / U;
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
  if (tpr > 32)
    return U == 1 ? launch_u<1, true>(cfg, a, tpr, prows, pcols, words) : launch_u<2, true>(cfg, a, tpr, prows, pcols, words);
  return U == 1 ? launch_u<1, false>(cfg, a, tpr, prows, pcols, words) : launch_u<2, false>(cfg, a, tpr, prows, pcols, words);
}

}  // namespace fp4
