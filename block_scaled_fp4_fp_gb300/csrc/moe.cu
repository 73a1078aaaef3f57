// moe.cu -- routed rows in order of their experts (what gather_rows and gather_qmm take), the experts' rows back to
// their tokens with weights applied, and the gradients of that.
#include <algorithm>

#include "../../include/fp4_gb300.h"
#include "common.cuh"
#include "launch.h"

namespace fp4 {
namespace {

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// an int of the same shared-memory place in CTA `rank` of the cluster
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// ---------------------------------------------------------------- moe_sort --
// A stable counting sort.  Every warp owns a run of routed rows, in order of the CTA's rank in its cluster and the
// warp's in its CTA, and counts its run's rows by expert: lanes with the same expert find one another
// (match) and the first of them adds their number, so nothing is atomic and the order is fixed.  Sums of the counts
// over the warps before (shared memory), the CTAs before (distributed shared memory) and the experts before give every
// (warp, expert) its first place; the second pass over the run hands the places out.
// Bound by latency.  One CTA up to kSortOne rows, above a cluster of eight: its counts need no workspace and no second launch.
constexpr int kSortBatch = 4;  // loads in flight a lane

__global__ void __launch_bounds__(1024) moe_sort_kernel(const int32_t* __restrict__ ids, int R, int k, int E, int run,
                                                        int32_t* __restrict__ lhs, int32_t* __restrict__ rhs,
                                                        int32_t* __restrict__ slot, int32_t* __restrict__ offsets,
                                                        unsigned* __restrict__ err) {
  extern __shared__ int sort_smem[];
  const int W = (int)blockDim.x >> 5, pitch = E + 1;  // (odd pitch of counts for even E: a column's words lie in different banks)
  int* count = sort_smem;             // [W][pitch]: rows of the warp, then of the warps before it
  int* total = sort_smem + W * pitch; // [E] of this CTA
  int* first = total + E;             // [E]: place of this CTA's first row of the expert
  __shared__ int warp_sum[32];
  __shared__ int kept_sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int ctas = (int)gridDim.x;  // one cluster
  const uint32_t rank = cluster_rank();
  for (int i = t; i < W * pitch; i += (int)blockDim.x) count[i] = 0;
  __syncthreads();
  // R <= 2^30 and at most 8 * 32 runs of R / 256 + 31 rows: no overflow
  const int lo = ((int)rank * W + warp) * run, hi = min(lo + run, R);
  int* mine = count + warp * pitch;
  bool bad = false;
  for (int i0 = lo; i0 < hi; i0 += 32 * kSortBatch) {
    int e[kSortBatch];
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      const int i = i0 + 32 * u + lane;
      e[u] = i < hi ? __ldg(ids + i) : -1;
      bad |= e[u] >= E;
      if ((unsigned)e[u] >= (unsigned)E) e[u] = E;  // dropped
    }
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      const unsigned peers = __match_any_sync(0xffffffffu, e[u]);
      if (e[u] < E && lane == __ffs((int)peers) - 1) mine[e[u]] += __popc(peers);
      __syncwarp();
    }
  }
  if (bad) record_error(err, kErrIndex);
  __syncthreads();
  // over the CTA's warps: a warp an expert, a lane a warp
  for (int e = warp; e < E; e += W) {
    const int c = lane < W ? count[lane * pitch + e] : 0;
    int s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane < W) count[lane * pitch + e] = s - c;
    if (lane == 31) total[e] = s;
  }
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // over the CTAs, then over the experts (a thread an expert: the block has at least E threads)
  int before = 0, all = 0;
  if (t < E) {
    if (ctas == 1) {
      all = total[t];
    } else {
      for (int c = 0; c < ctas; ++c) {
        const int v = ld_cluster(total + t, (uint32_t)c);
        all += v;
        if (c < (int)rank) before += v;
      }
    }
  }
  if (ctas > 1) cluster_arrive();  // this CTA has read the others' totals (waited for at the end)
  int s = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sum[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const int v = lane < W ? warp_sum[lane] : 0;
    int i = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, i, o);
      if (lane >= o) i += u;
    }
    if (lane < W) warp_sum[lane] = i - v;
    if (lane == 31) kept_sh = i;
  }
  __syncthreads();
  const int kept = kept_sh;
  if (t < E) {
    const int at = warp_sum[warp] + s - all;
    first[t] = at + before;
    if (rank == 0) offsets[t] = at;
  }
  if (rank == 0 && t == 0) offsets[E] = kept;
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += 32 * kSortBatch) {
    int e[kSortBatch];
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      const int i = i0 + 32 * u + lane;
      e[u] = i < hi ? __ldg(ids + i) : -1;
      if ((unsigned)e[u] >= (unsigned)E) e[u] = E;
    }
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
      const int i = i0 + 32 * u + lane;
      const unsigned peers = __match_any_sync(0xffffffffu, e[u]);
      const unsigned ahead = peers & ((1u << lane) - 1);
      int at = -1;
      if (e[u] < E) {
        at = first[e[u]] + mine[e[u]] + __popc(ahead);
        lhs[at] = (int)((unsigned)i / (unsigned)k);
        rhs[at] = e[u];
      }
      if (i < hi) slot[i] = at;
      __syncwarp();
      if (e[u] < E && ahead == 0) mine[e[u]] += __popc(peers);
      __syncwarp();
    }
  }
  for (int64_t i = (int64_t)kept + (int)rank * (int)blockDim.x + t; i < R; i += (int64_t)ctas * (int)blockDim.x) {
    lhs[i] = 0;
    rhs[i] = E - 1;
  }
  if (ctas > 1) cluster_wait();  // no CTA's shared memory goes away while another may read its totals
}

// ------------------------------------------------------------- moe_combine --
// A thread a 16-byte piece of a token's row: its k rows are read with up to eight loads in flight, added in fp32 in
// order of j, rounded once.  Bound by HBM.
constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(
    const uint16_t* __restrict__ y, int rows, const int32_t* __restrict__ slot, const float* __restrict__ weights,
    const uint16_t* residual, int64_t T, int k, int pieces, uint16_t* out, unsigned* __restrict__ err) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t base = (int64_t)blockIdx.x * kCombineThreads;
  const int64_t t0 = base <= UINT32_MAX ? (int64_t)((unsigned)base / (unsigned)pieces) : base / pieces;
  const unsigned rem = (unsigned)(base - t0 * pieces) + threadIdx.x;
  const int64_t t = t0 + rem / (unsigned)pieces;
  const int p = (int)(rem % (unsigned)pieces);
  if (t >= T) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (residual) {
    const uint4 r = *(reinterpret_cast<const uint4*>(residual) + t * pieces + p);
    const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] = bf16_lo(rw[i]);
      acc[2 * i + 1] = bf16_hi(rw[i]);
    }
  }
  const int32_t* sl = slot + t * k;
  for (int j0 = 0; j0 < k; j0 += 8) {
    uint4 v[8];
    int at[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      at[j] = j0 + j < k ? __ldg(sl + j0 + j) : -1;
      if (at[j] >= rows) {
        if (p == 0) record_error(err, kErrIndex);
        at[j] = -1;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at[j] >= 0) v[j] = ld_stream_v4(reinterpret_cast<const uint4*>(y) + (int64_t)at[j] * pieces + p);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (at[j] < 0) continue;
      const float w = weights ? __ldg(weights + t * k + j0 + j) : 1.0f;
      const uint32_t vw[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = __fmaf_rn(w, bf16_lo(vw[i]), acc[2 * i]);
        acc[2 * i + 1] = __fmaf_rn(w, bf16_hi(vw[i]), acc[2 * i + 1]);
      }
    }
  }
  *(reinterpret_cast<uint4*>(out) + t * pieces + p) =
      make_uint4(pack_bf16x2_rn(acc[0], acc[1]), pack_bf16x2_rn(acc[2], acc[3]), pack_bf16x2_rn(acc[4], acc[5]),
                 pack_bf16x2_rn(acc[6], acc[7]));
}

// ---------------------------------------------------- moe_combine_backward --
// A CTA a token: dout's row is read once (again from L1 for each further eight of the k rows), a row of dy written and a
// row of y multiplied with it for each j.  The dot products of eight rows are reduced together: each step of the
// butterfly halves the number of sums a lane holds, nine shuffles instead of forty.  The CTAs from T on clear the rows that no slot names.
// Bound by HBM.
constexpr int kTailCtas = 64, kBackwardThreads = 512;

__global__ void __launch_bounds__(kBackwardThreads) moe_combine_backward_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y, const int32_t* __restrict__ slot,
    const float* __restrict__ weights, int64_t T, int k, int pieces, int64_t rows, const int32_t* __restrict__ rows_used,
    uint16_t* __restrict__ dy, float* __restrict__ dweights, unsigned* __restrict__ err) {
  __shared__ float part[kBackwardThreads / 32][8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t = blockIdx.x;
  if (t >= T) {
    const int64_t tail = (int64_t)gridDim.x - T;
    for (int64_t r = max(0, __ldg(rows_used)) + (t - T); r < rows; r += tail)
      for (int p = threadIdx.x; p < pieces; p += (int)blockDim.x)
        *(reinterpret_cast<uint4*>(dy) + r * pieces + p) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint4* g4 = reinterpret_cast<const uint4*>(dout) + t * pieces;
  for (int j0 = 0; j0 < k; j0 += 8) {
    int at[8];
    float w[8], dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      at[j] = j0 + j < k ? __ldg(slot + t * k + j0 + j) : -1;
      if (at[j] >= rows) {
        if (threadIdx.x == 0) record_error(err, kErrIndex);
        at[j] = -1;
      }
      w[j] = at[j] >= 0 && weights ? __ldg(weights + t * k + j0 + j) : 1.0f;
      dot[j] = 0.f;
    }
    for (int p = threadIdx.x; p < pieces; p += (int)blockDim.x) {
      const uint4 gv = __ldg(g4 + p);
      const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
      uint4 v[8];
      if (dweights) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at[j] >= 0) v[j] = ld_stream_v4(reinterpret_cast<const uint4*>(y) + (int64_t)at[j] * pieces + p);
      }
      float g[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[2 * i] = bf16_lo(gw[i]);
        g[2 * i + 1] = bf16_hi(gw[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (at[j] < 0) continue;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2_rn(__fmul_rn(w[j], g[2 * i]), __fmul_rn(w[j], g[2 * i + 1]));
        *(reinterpret_cast<uint4*>(dy) + (int64_t)at[j] * pieces + p) = make_uint4(o[0], o[1], o[2], o[3]);
        if (dweights) {
          const uint32_t vw[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dot[j] = __fmaf_rn(g[2 * i], bf16_lo(vw[i]), dot[j]);
            dot[j] = __fmaf_rn(g[2 * i + 1], bf16_hi(vw[i]), dot[j]);
          }
        }
      }
    }
    if (!dweights) continue;
    // lane bits 4, 3, 2 pick the half of the sums that the lane keeps
#pragma unroll
    for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = upper ? dot[i] : dot[i + n], keep = upper ? dot[i + n] : dot[i];
        dot[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
    }
    float d = dot[0];
    d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, 2));
    d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, 1));
    if ((lane & 3) == 0) part[warp][lane >> 2] = d;  // lane >> 2 is j: its bits picked the halves
    __syncthreads();
    if (threadIdx.x < 8 && j0 + (int)threadIdx.x < k) {
      float sum = 0.f;
      for (int i = 0; i < (int)blockDim.x >> 5; ++i) sum = __fadd_rn(sum, part[i][threadIdx.x]);
      const int s = __ldg(slot + t * k + j0 + threadIdx.x);
      dweights[t * k + j0 + threadIdx.x] = s >= 0 && s < rows ? sum : 0.0f;
    }
    __syncthreads();
  }
}

void pdl(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int64_t grid, int block, size_t smem, cudaStream_t s) {
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

}  // namespace

constexpr int kSortOne = 4096;  // rows that one CTA sorts

cudaError_t launch_moe_sort(const DevInfo& d, const int32_t* ids, int64_t T, int k, int E, int32_t* lhs, int32_t* rhs,
                            int32_t* slot, int32_t* offsets, cudaStream_t s) {
  const int64_t R = T * k;
  const int ctas = R > kSortOne ? 8 : 1;
  int64_t threads = std::max<int64_t>((E + 31) / 32 * 32, std::min<int64_t>((R + 31) / 32 * 32, 1024));
  if (ctas > 1) threads = 1024;
  const int warps = (int)threads / 32;
  const int64_t per = (R + (int64_t)ctas * warps - 1) / ((int64_t)ctas * warps);
  const int run = (int)((per + 31) / 32 * 32);
  const int smem = (warps * (E + 1) + 2 * E) * 4;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(d, moe_sort_kernel, (32 * 1025 + 2 * 1024) * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  pdl(cfg, attr, ctas, (int)threads, (size_t)smem, s);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, moe_sort_kernel, ids, (int)R, k, E, run, lhs, rhs, slot, offsets, d.err);
}

cudaError_t launch_moe_combine(const DevInfo& d, const uint16_t* y, int64_t rows, const int32_t* slot,
                               const float* weights, const uint16_t* residual, int64_t T, int k, int cols,
                               uint16_t* out, cudaStream_t s) {
  const int pieces = cols / 8;
  const int64_t grid = (T * pieces + kCombineThreads - 1) / kCombineThreads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, grid, kCombineThreads, 0, s);
  return cudaLaunchKernelEx(&cfg, moe_combine_kernel, y, (int)rows, slot, weights, residual, T, k, pieces, out, d.err);
}

cudaError_t launch_moe_combine_backward(const DevInfo& d, const uint16_t* dout, const uint16_t* y, const int32_t* slot,
                                        const float* weights, int64_t T, int k, int cols, int64_t rows,
                                        const int32_t* rows_used, uint16_t* dy, float* dweights, cudaStream_t s) {
  const int pieces = cols / 8;
  const int64_t grid = T + (rows_used ? std::min<int64_t>(rows, kTailCtas) : 0);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, grid, std::min(kBackwardThreads, (pieces + 31) / 32 * 32), 0, s);
  return cudaLaunchKernelEx(&cfg, moe_combine_backward_kernel, dout, y, slot, weights, T, k, pieces, rows, rows_used, dy,
                            dweights, d.err);
}

}  // namespace fp4
