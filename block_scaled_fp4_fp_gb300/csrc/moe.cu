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
// A stable counting sort in one launch: one CTA, or a cluster whose CTAs hold the routed rows in order of their ranks.
//   1. Each CTA counts its rows by expert; the counts of the CTAs before (distributed shared memory) and the experts
//      before give the place of its first row of each expert.
//   2. Tile by tile of up to kTileRows rows, a run of them a warp: lanes with the same expert find one another by a
//      vote on each bit of its number (nothing is atomic, so the order is fixed), which with the counts of the warps
//      before gives each row its place in the tile's own order.  The tile is put into that order in shared memory and
//      written from there, neighbouring places by neighbouring lanes.
// A CTA of one tile takes its counts from 2.  No workspace, no second launch.  Bound by latency (384 rows of 32 experts:
// 2.1 us, of which a launch is 1.7), and with many rows by what 16 SMs issue (131,072 rows of 256 experts: 12.5 us).
// Tried, for 131,072 rows of 256 experts on eight CTAs: the match instruction in place of the votes (41 us against 31),
// rows written straight to their places (31 against 22: a sector a lane; a tile of one row a lane still does).
constexpr int kRunRows = 8;                        // a lane's rows of a tile
constexpr int kTileRows = 32 * 32 * kRunRows;      // of a CTA of 32 warps: 13 bits
constexpr int kExpertBits = 10;

// exclusive sum over the block of one value a thread (all threads; `part`: 33 ints)
__device__ __forceinline__ int block_scan(int v, int* part, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = (int)blockDim.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < W ? part[lane] : 0;
    int i = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, i, o);
      if (lane >= o) i += u;
    }
    if (lane < W) part[lane] = i - w;
    if (lane == 31) part[32] = i;
  }
  __syncthreads();
  all = part[32];
  return part[warp] + s - v;
}

__global__ void __launch_bounds__(1024) moe_sort_kernel(const int32_t* __restrict__ ids, int R, int k, int E, int bits,
                                                        int rows_cta, int run, int32_t* __restrict__ lhs,
                                                        int32_t* __restrict__ rhs, int32_t* __restrict__ slot,
                                                        int32_t* __restrict__ offsets, unsigned* __restrict__ err) {
  extern __shared__ int sort_smem[];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, W = (int)blockDim.x >> 5;
  int* count = sort_smem;                                // [W][E]: rows of the warp, then of the warps before it
  int* total = count + W * E;                            // [E] rows of this CTA
  int* delta = total + E;                                // [E] from a place in the tile's order to one in the list
  int* start = delta + E;                                // [E] the expert's first place in the tile's order
  uint32_t* stage = reinterpret_cast<uint32_t*>(start + E);  // [tile]: row of the tile and expert
  __shared__ int part[33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ctas = (int)gridDim.x;  // one cluster
  const uint32_t rank = cluster_rank();
  const int tile = run * W;
  // rows [begin, end) of this CTA (R <= 2^30: no overflow)
  const int begin = min((int)rank * rows_cta, R), end = min(begin + rows_cta, R);
  const bool one_tile = rows_cta <= tile;
  int e[kRunRows], at[kRunRows];
  bool bad = false;

  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kRunRows; ++u) {
      const int i = i0 + warp * run + 32 * u + lane;
      e[u] = 32 * u < run && i < end ? __ldg(ids + i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kRunRows; ++u) {
      bad |= e[u] >= E;
      if (e[u] >= E) e[u] = -1;  // dropped
    }
  };
  // at: a row's place among its warp's of the same expert; count: the warps' numbers of rows, then of those before
  auto places = [&]() -> int {  // returns (thread t) the tile's rows of expert t
    for (int i = t; i < W * E; i += (int)blockDim.x) count[i] = 0;
    __syncthreads();
    int* mine = count + warp * E;
#pragma unroll
    for (int u = 0; u < kRunRows; ++u) {
      if (32 * u >= run) break;
      const bool kept = e[u] >= 0;
      unsigned peers = __ballot_sync(0xffffffffu, kept);
#pragma unroll
      for (int b = 0; b < kExpertBits; ++b) {
        if (b >= bits) break;
        const bool one = (e[u] >> b) & 1;
        const unsigned v = __ballot_sync(0xffffffffu, one);
        peers &= one ? v : ~v;
      }
      const unsigned ahead = peers & ((1u << lane) - 1);
      const int base = kept ? mine[e[u]] : 0;
      at[u] = base + __popc(ahead);
      __syncwarp();
      if (kept && ahead == 0) mine[e[u]] = base + __popc(peers);
      __syncwarp();
    }
    __syncthreads();
    int s = 0;
    if (t < E) {  // a thread an expert (the block has at least E)
      for (int w0 = 0; w0 < W; w0 += 8) {
        int c[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = w0 + w < W ? count[(w0 + w) * E + t] : 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          if (w0 + w < W) count[(w0 + w) * E + t] = s;
          s += c[w];
        }
      }
    }
    return s;
  };

  int in_tile = 0;  // (thread t < E) the tile's rows of expert t
  load(begin);
  if (one_tile) {
    in_tile = places();
    if (t < E) total[t] = in_tile;
  } else {
    if (t < E) total[t] = 0;
    __syncthreads();
    for (int i0 = begin;;) {
#pragma unroll
      for (int u = 0; u < kRunRows; ++u)
        if (e[u] >= 0) atomicAdd(total + e[u], 1);
      i0 += tile;
      if (i0 >= end) break;
      load(i0);
    }
  }
  int before = 0, all = 0;
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
    if (t < E)
      for (int c = 0; c < ctas; ++c) {
        const int v = ld_cluster(total + t, (uint32_t)c);
        all += v;
        if (c < (int)rank) before += v;
      }
    cluster_arrive();  // this CTA has read the others' totals (waited for at the end)
  } else {
    __syncthreads();
    if (t < E) all = total[t];
  }
  int kept;
  int first = block_scan(all, part, kept);  // (thread t < E) place of the expert's first row, then of this CTA's next
  if (rank == 0) {
    if (t < E) offsets[t] = first;
    if (t == 0) offsets[E] = kept;
  }
  first += before;
  if (one_tile && run == 32) {  // a row a lane: straight to its place
    if (t < E) start[t] = first;
    __syncthreads();
    const int i = begin + warp * 32 + lane;
    if (i < end) {
      int to = -1;
      if (e[0] >= 0) {
        to = start[e[0]] + count[warp * E + e[0]] + at[0];
        lhs[to] = (int)((unsigned)i / (unsigned)k);
        rhs[to] = e[0];
      }
      slot[i] = to;
    }
  } else for (int i0 = begin; i0 < end; i0 += tile) {
    if (!one_tile) {
      load(i0);
      in_tile = places();
    }
    __syncthreads();  // (part is free again)
    int staged;
    const int s = block_scan(t < E ? in_tile : 0, part, staged);
    if (t < E) {
      start[t] = s;
      delta[t] = first - s;
      first += in_tile;
    }
    __syncthreads();
    const int* mine = count + warp * E;
#pragma unroll
    for (int u = 0; u < kRunRows; ++u) {
      const int j = warp * run + 32 * u + lane, i = i0 + j;
      if (32 * u >= run || i >= end) break;
      int to = -1;
      if (e[u] >= 0) {
        to = start[e[u]] + mine[e[u]] + at[u];
        stage[to] = (uint32_t)j << kExpertBits | (uint32_t)e[u];
        to += delta[e[u]];
      }
      slot[i] = to;
    }
    __syncthreads();
    for (int j = t; j < staged; j += (int)blockDim.x) {
      const uint32_t v = stage[j];
      const int x = (int)(v & ((1u << kExpertBits) - 1)), to = j + delta[x];
      lhs[to] = (int)(((unsigned)i0 + (v >> kExpertBits)) / (unsigned)k);
      rhs[to] = x;
    }
    if (!one_tile) __syncthreads();  // count, delta and stage have been read
  }
  if (bad) record_error(err, kErrIndex);
  for (int64_t i = (int64_t)kept + (int)rank * (int)blockDim.x + t; i < R; i += (int64_t)ctas * (int)blockDim.x) {
    lhs[i] = 0;
    rhs[i] = E - 1;
  }
  if (ctas > 1) cluster_wait();  // no CTA's shared memory goes away while another may read its totals
}

// ------------------------------------------------------------- moe_combine --
// A thread has P 16-byte pieces of tokens' rows, K rows of each in flight: eight loads whatever k is (bytes in flight are
// what the rate goes by: 2048 x 4 of 2880 took 17.9 us with four).  Added in fp32 in order of j, rounded once.
// Bound by HBM: 8192 x 8 of 2880 66 us, 6.4 TB/s; 2048 x 4 of 2880 12.5 us, 4.7 TB/s (seven CTAs of 128 an SM, 2.7 waves:
// the loads behind a slot wait for it).  Tried: CTAs that stay and fetch the next slots while rows are on their way (13.1 and
// 69.0 us).
constexpr int kCombineThreads = 128;

template <int K, int P>
__global__ void __launch_bounds__(kCombineThreads, P == 4 ? 4 : 7) moe_combine_kernel(
    const uint16_t* __restrict__ y, int rows, const int32_t* __restrict__ slot, const float* __restrict__ weights,
    const uint16_t* residual, int64_t T, int k, int pieces, uint16_t* out, unsigned* __restrict__ err) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t base = (int64_t)blockIdx.x * (kCombineThreads * P);
  const int64_t t0 = base <= UINT32_MAX ? (int64_t)((unsigned)base / (unsigned)pieces) : base / pieces;
  const unsigned rem = (unsigned)(base - t0 * pieces) + threadIdx.x;
  int64_t t[P];
  int p[P];
  float acc[P][8];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const unsigned r = rem + (unsigned)(q * kCombineThreads), n = r / (unsigned)pieces;
    t[q] = t0 + n;
    p[q] = (int)(r - n * (unsigned)pieces);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[q][i] = 0.f;
  }
  if (residual) {
    uint4 r[P];
#pragma unroll
    for (int q = 0; q < P; ++q)
      if (t[q] < T) r[q] = *(reinterpret_cast<const uint4*>(residual) + t[q] * pieces + p[q]);
#pragma unroll
    for (int q = 0; q < P; ++q)
      if (t[q] < T) unpack8(r[q], acc[q]);
  }
  for (int j0 = 0; j0 < k; j0 += K) {
    uint4 v[P][K];
    int at[P][K];
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int j = 0; j < K; ++j) at[q][j] = t[q] < T && j0 + j < k ? __ldg(slot + t[q] * k + j0 + j) : -1;
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (at[q][j] >= rows) {
          if (p[q] == 0) record_error(err, kErrIndex);
          at[q][j] = -1;
        }
        if (at[q][j] >= 0) v[q][j] = ld_stream_v4(reinterpret_cast<const uint4*>(y) + (int64_t)at[q][j] * pieces + p[q]);
      }
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int j = 0; j < K; ++j) {
        if (at[q][j] < 0) continue;
        const float w = weights ? __ldg(weights + t[q] * k + j0 + j) : 1.0f;
        float f[8];
        unpack8(v[q][j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[q][i] = __fmaf_rn(w, f[i], acc[q][i]);
      }
  }
#pragma unroll
  for (int q = 0; q < P; ++q)
    if (t[q] < T) *(reinterpret_cast<uint4*>(out) + t[q] * pieces + p[q]) = pack8(acc[q]);
}

// ---------------------------------------------------- moe_combine_backward --
// A CTA a token, or a warp a token where rows are short and tokens many: dout's row is read (again from L1 for each
// further K of the k rows), a row of dy written and a row of y multiplied with it for each j; two pieces of K rows are in
// flight a thread.  The dot products of the K rows are reduced together: each step of the butterfly halves the number of
// sums a lane holds, nine shuffles instead of forty for eight.
// The CTAs behind the tokens' clear the rows that no slot names.  Bound by HBM: 4096 x 8 of 5120 110 us, 6.5 TB/s; 2048 x 4
// of 2880 21 us, 5.0 TB/s.  Tried: packed fp32 for the products (no change, here as in moe_combine: loads are what is waited
// for).
constexpr int kTailCtas = 64, kBackwardThreads = 512;

enum TokenOf { kCta512, kCta128, kWarp };  // what a token belongs to
template <int K, int OF>
__global__ void __launch_bounds__(OF == kCta512 ? kBackwardThreads : 128, OF == kCta512 ? 1 : K == 8 ? 4 : K == 4 ? 5 : 6) moe_combine_backward_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y, const int32_t* __restrict__ slot,
    const float* __restrict__ weights, int64_t T, int k, int pieces, int64_t rows, const int32_t* __restrict__ rows_used,
    uint16_t* __restrict__ dy, float* __restrict__ dweights, unsigned* __restrict__ err) {
  constexpr int P = 2;
  constexpr bool WARP = OF == kWarp;
  __shared__ float part[kBackwardThreads / 32][K];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token_ctas = WARP ? (T + 3) / 4 : T;
  if (blockIdx.x >= token_ctas) {
    const int64_t tail = (int64_t)gridDim.x - token_ctas;
    for (int64_t r = max(0, __ldg(rows_used)) + (blockIdx.x - token_ctas); r < rows; r += tail)
      for (int p = threadIdx.x; p < pieces; p += (int)blockDim.x)
        *(reinterpret_cast<uint4*>(dy) + r * pieces + p) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t t = WARP ? (int64_t)blockIdx.x * 4 + warp : blockIdx.x;
  if (WARP && t >= T) return;
  const int thread = WARP ? lane : (int)threadIdx.x, step = WARP ? 32 : (int)blockDim.x;  // of the token's
  const uint4* g4 = reinterpret_cast<const uint4*>(dout) + t * pieces;
  for (int j0 = 0; j0 < k; j0 += K) {
    int at[K];
    float w[K], dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) at[j] = j0 + j < k ? __ldg(slot + t * k + j0 + j) : -1;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (at[j] >= rows) {
        if (thread == 0) record_error(err, kErrIndex);
        at[j] = -1;
      }
      w[j] = at[j] >= 0 && weights ? __ldg(weights + t * k + j0 + j) : 1.0f;
      dot[j] = 0.f;
    }
    for (int p0 = thread; p0 < pieces; p0 += P * step) {
      uint4 gv[P], v[P][K];
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const int p = p0 + q * step;
        if (p >= pieces) continue;
        gv[q] = __ldg(g4 + p);
        if (dweights) {
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (at[j] >= 0) v[q][j] = ld_stream_v4(reinterpret_cast<const uint4*>(y) + (int64_t)at[j] * pieces + p);
        }
      }
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const int p = p0 + q * step;
        if (p >= pieces) continue;
        float g[8];
        unpack8(gv[q], g);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          if (at[j] < 0) continue;
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(w[j], g[i]);
          *(reinterpret_cast<uint4*>(dy) + (int64_t)at[j] * pieces + p) = pack8(f);
          if (dweights) {
            unpack8(v[q][j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[j] = __fmaf_rn(g[i], f[i], dot[j]);
          }
        }
      }
    }
    if (!dweights) continue;
    // the lane's top bits pick the half of the sums that it keeps: lane / (32 / K) is then j
#pragma unroll
    for (int n = K / 2, o = 16; n > 0; n >>= 1, o >>= 1) {
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = upper ? dot[i] : dot[i + n], keep = upper ? dot[i + n] : dot[i];
        dot[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
    }
    float d = dot[0];
#pragma unroll
    for (int o = 16 / K; o > 0; o >>= 1) d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, o));
    if (WARP) {
      const int j = lane / (32 / K);
      if (lane % (32 / K) == 0 && j0 + j < k) {
        const int s = __ldg(slot + t * k + j0 + j);
        dweights[t * k + j0 + j] = s >= 0 && s < rows ? d : 0.0f;
      }
      continue;
    }
    if (lane % (32 / K) == 0) part[warp][lane / (32 / K)] = d;
    __syncthreads();
    if (threadIdx.x < K && j0 + (int)threadIdx.x < k) {
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

// Rows that one CTA sorts (2048 of 32 experts: 4.5 us, with a cluster 4.4; 4096: 5.7 against 4.4), and the CTAs of a
// cluster above: 16, the most there is (131,072 rows of 256 experts: 12.5 us, with eight 22).  A CTA takes an SM whole, and a
// part of a GPU may hold no 16 of them side by side: then eight, or one.
constexpr int kSortOne = 2048, kSortCtas[] = {16, 8, 1};

namespace {
constexpr int kSortSmem = (35 * 1024 + kTileRows) * 4;  // the most that a CTA wants

void sort_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int ctas, int threads, int smem, cudaStream_t s) {
  pdl(cfg, attr, ctas, threads, (size_t)smem, s);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
}

// The largest of kSortCtas that the device has room for, asked once a device (where the kernel's attributes are set too).
cudaError_t sort_ctas(const DevInfo& d, int& most) {
  static std::atomic<int> known[64];
  std::atomic<int>& mine = known[d.device & 63];
  if ((most = mine.load(std::memory_order_acquire)) != 0) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  for (int ctas : kSortCtas) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    sort_config(cfg, attr, ctas, 1024, kSortSmem, nullptr);
    int clusters = 0;
    most = ctas;
    if (ctas == 1 || (cudaOccupancyMaxActiveClusters(&clusters, moe_sort_kernel, &cfg) == cudaSuccess && clusters > 0)) break;
    (void)cudaGetLastError();
  }
  mine.store(most, std::memory_order_release);
  return cudaSuccess;
}
}  // namespace

cudaError_t launch_moe_sort(const DevInfo& d, const int32_t* ids, int64_t T, int k, int E, int32_t* lhs, int32_t* rhs,
                            int32_t* slot, int32_t* offsets, int most_ctas, cudaStream_t s) {
  const int64_t R = T * k;
  int most = 1, ctas = 1;
  const cudaError_t e = sort_ctas(d, most);
  if (e != cudaSuccess) return e;
  if (most_ctas > 0) most = std::min(most, most_ctas);
  if (R > kSortOne)
    for (int n : kSortCtas) ctas = std::max(ctas, n <= most ? n : 1);
  const int64_t whole = std::max<int64_t>((E + 31) / 32 * 32, std::min<int64_t>((R + 31) / 32 * 32, 1024));
  const int threads = ctas > 1 ? 1024 : (int)whole, warps = threads / 32;
  const int64_t rows_cta = (R + ctas - 1) / ctas;
  const int run = (int)std::min<int64_t>((rows_cta + threads - 1) / threads, kRunRows) * 32;
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  sort_config(cfg, attr, ctas, threads, ((warps + 3) * E + run * warps) * 4, s);
  return cudaLaunchKernelEx(&cfg, moe_sort_kernel, ids, (int)R, k, E, bits, (int)rows_cta, run, lhs, rhs, slot, offsets,
                            d.err);
}

namespace {
template <int K, int P>
cudaError_t combine(const DevInfo& d, const uint16_t* y, int64_t rows, const int32_t* slot, const float* weights,
                    const uint16_t* residual, int64_t T, int k, int pieces, uint16_t* out, cudaStream_t s) {
  const int64_t grid = (T * pieces + kCombineThreads * P - 1) / (kCombineThreads * P);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, grid, kCombineThreads, 0, s);
  return cudaLaunchKernelEx(&cfg, moe_combine_kernel<K, P>, y, (int)rows, slot, weights, residual, T, k, pieces, out, d.err);
}
}  // namespace

cudaError_t launch_moe_combine(const DevInfo& d, const uint16_t* y, int64_t rows, const int32_t* slot,
                               const float* weights, const uint16_t* residual, int64_t T, int k, int cols,
                               uint16_t* out, cudaStream_t s) {
  const int pieces = cols / 8;
  // several pieces a thread only where there are threads enough for the GPU (2048 x 4 of 2880: 12.5 us against 13.5 with one;
  // 96 x 4 of 5120: 3.1 against 2.7)
  const bool many = T * pieces >= (int64_t)d.sm_count * 2048;
  if (!many || k > 4) return combine<8, 1>(d, y, rows, slot, weights, residual, T, k, pieces, out, s);
  if (k > 2) return combine<4, 2>(d, y, rows, slot, weights, residual, T, k, pieces, out, s);
  return combine<2, 4>(d, y, rows, slot, weights, residual, T, k, pieces, out, s);
}

cudaError_t launch_moe_combine_backward(const DevInfo& d, const uint16_t* dout, const uint16_t* y, const int32_t* slot,
                                        const float* weights, int64_t T, int k, int cols, int64_t rows,
                                        const int32_t* rows_used, uint16_t* dy, float* dweights, cudaStream_t s) {
  const int pieces = cols / 8;
  // (20,000 x 2 of 512: 20 us a warp a token, 29 a CTA; 5000 x 4 of 1024: 18 and 25; 20,000 x 8 of 256: 39 and 36)
  const bool warps = pieces > 32 && pieces <= 128 && T >= 32 * (int64_t)d.sm_count;
  const int64_t grid = (warps ? (T + 3) / 4 : T) + (rows_used ? std::min<int64_t>(rows, kTailCtas) : 0);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  // many tokens share an SM, few take it whole
  const int most = warps || T >= 4 * d.sm_count ? 128 : kBackwardThreads;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl(cfg, attr, grid, warps ? 128 : std::min(most, (pieces + 31) / 32 * 32), 0, s);
  auto go = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, dout, y, slot, weights, T, k, pieces, rows, rows_used, dy, dweights, d.err);
  };
  if (warps)
    return k > 4   ? go(moe_combine_backward_kernel<8, kWarp>)
           : k > 2 ? go(moe_combine_backward_kernel<4, kWarp>)
                   : go(moe_combine_backward_kernel<2, kWarp>);
  if (most == 128)
    return k > 4   ? go(moe_combine_backward_kernel<8, kCta128>)
           : k > 2 ? go(moe_combine_backward_kernel<4, kCta128>)
                   : go(moe_combine_backward_kernel<2, kCta128>);
  return k > 4   ? go(moe_combine_backward_kernel<8, kCta512>)
         : k > 2 ? go(moe_combine_backward_kernel<4, kCta512>)
                 : go(moe_combine_backward_kernel<2, kCta512>);
}

}  // namespace fp4
