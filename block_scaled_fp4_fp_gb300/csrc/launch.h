// launch.h -- host-side launchers shared between the C ABI (api.cu) and the
// kernel translation units.  Arguments reaching these functions have already
// been validated by api.cu; each returns the cudaError_t of its launch(es).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace fp4 {

struct DevInfo {
  int device = -1;
  int sm_count = 0;
  size_t smem_optin = 0;   // max dynamic shared memory per block (opt-in)
  unsigned* err = nullptr; // device address of the error word on this device
};

// api.cu: the current device's cached properties (initialized on first use);
// returns an fp4_status value
int current_device_info(const DevInfo** out);

// Lets a kernel use `bytes` of dynamic shared memory, once per device and kernel: the attribute stays set,
// and setting it costs a driver call.  `done`: a bit per device, the caller's static.
template <typename Kernel>
cudaError_t allow_smem(const DevInfo& d, Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  const uint64_t bit = 1ull << (d.device & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// quant.cu
size_t amax_workspace_bytes(int64_t n);
cudaError_t launch_amax(const DevInfo& d, const uint16_t* x, int64_t n, float* gs_out,
                        float* amax_out, uint32_t* partials, int max_partials, cudaStream_t s);
// sr != 0: stochastic rounding of the elements (Philox4x32-10 words from seed and offset)
cudaError_t launch_quantize(const DevInfo& d, const uint16_t* x, int64_t rows, int64_t cols,
                            int mode, int group, const float* gs, uint32_t* xq, uint8_t* scales,
                            int tiled, int sr, uint64_t seed, uint64_t offset, cudaStream_t s);
cudaError_t launch_dequantize(const DevInfo& d, const uint32_t* wq, const void* scales,
                              const uint16_t* biases, int64_t rows, int64_t cols, int mode,
                              int group, const float* gs, int tiled, uint16_t* out,
                              cudaStream_t s);

// qmv.cu (qx != 0: the quantized-activation route -- x is replaced by
// fp_dequantize(fp_quantize(x, gs_x)) before the GEMV; NVFP4 and MXFP4 only)
cudaError_t launch_qmv(const DevInfo& d, const uint16_t* x, const float* gs_x, int qx, const uint32_t* w,
                       const void* scales, const uint16_t* biases, const float* gs_w, int64_t N, int64_t K,
                       int mode, int group, uint16_t* y, int inject_timeout, cudaStream_t s);

// qmv_tc.cu (NVFP4 = mode 2 and MXFP4 = mode 1 on tcgen05; launch_qmv dispatches to it when supported)
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // driver's tensor-map encoder (nullptr if unavailable)
// the NVFP4 plan: CTAs per cluster (K slices), row blocks, rows per CTA, weight ring slots
bool qmv_tc_geometry(const DevInfo& d, int64_t N, int64_t K, int* split, int* nblk, int* R, int* nslots);
bool qmv_tc_supported(const DevInfo& d, int mode, int64_t N, int64_t K);
bool qmv_tc_group_supported(const DevInfo& d, int mode, int count, const int64_t* N, int64_t K);
// the weights of a GEMV launch (a group of up to 4 matrices of one K)
struct GemvGroupDesc {
  int count = 0;
  const uint32_t* w[4] = {};
  const uint8_t* scales[4] = {};   // FP4: E4M3/E8M0 bytes; affine: bf16 scales
  const uint16_t* biases[4] = {};  // affine only
  int64_t N[4] = {};
  int64_t K = 0;
};
cudaError_t launch_qmv_tc_group(const DevInfo& d, int mode, const uint16_t* x, const float* gs_x, int qx, int count,
                                const uint32_t* const* w, const uint8_t* const* scales, const float* const* gs_w,
                                const int64_t* N, int64_t K, uint16_t* const* y, const GemvGroupDesc* next,
                                int inject_timeout, cudaStream_t s);
cudaError_t launch_qmv_tc(const DevInfo& d, int mode, const uint16_t* x, const float* gs_x, int qx,
                          const uint32_t* w, const uint8_t* scales, const float* gs_w, int64_t N, int64_t K,
                          uint16_t* y, int inject_timeout, cudaStream_t s);

// qmv_affine.cu (affine-4 GEMV on a TMA ring; launch_qmv dispatches to it when the plan fits:
// K a multiple of max(512, 8 group) and at most 32768, 16-byte aligned scales and biases)
bool qmv_affine_supported(const DevInfo& d, int64_t N, int64_t K, int group);
cudaError_t launch_qmv_affine(const DevInfo& d, const uint16_t* x, const uint32_t* w, const uint16_t* scales,
                              const uint16_t* biases, int64_t N, int64_t K, int group, uint16_t* y,
                              cudaStream_t s);
bool qmv_affine_group_supported(const DevInfo& d, int count, const int64_t* N, int64_t K, int group);
cudaError_t launch_qmv_affine_group(const DevInfo& d, const uint16_t* x, int count, const uint32_t* const* w,
                                    const uint16_t* const* scales, const uint16_t* const* biases, const int64_t* N,
                                    int64_t K, int group, uint16_t* const* y, const GemvGroupDesc* next,
                                    cudaStream_t s);

// qqmm.cu: batch b reads xq + b stride_xq (uint32 words), sx + b stride_sx (bytes),
// wq + b stride_wq (0: one W for every batch), sw + b stride_sw, gs_x[b], gs_w[b],
// and writes out + b stride_out (elements); a plain call is batch 1.
struct BatchArgs {
  int64_t batch = 1;
  int64_t stride_xq = 0, stride_sx = 0, stride_wq = 0, stride_sw = 0, stride_out = 0;
};
cudaError_t launch_qqmm(const DevInfo& d, const uint32_t* xq, const uint8_t* sx, const uint32_t* wq,
                        const uint8_t* sw, const float* gs_x, const float* gs_w, int64_t M,
                        int64_t N, int64_t K, const BatchArgs& ba, int mode, uint16_t* out, int inject_timeout,
                        cudaStream_t s);

// qqmm.cu: the fused call -- bf16 x quantized by the same (cooperative) launch
// into the workspace, then the GEMM (gs_in: the NVFP4 activation global scale,
// or nullptr to take amax(x) / 2688; gs_out: where the scale used goes, nullable)
size_t qqmm_fused_workspace_bytes(int64_t M, int64_t K, int mode);
cudaError_t launch_qqmm_fused(const DevInfo& d, const uint16_t* x, const float* gs_in, float* gs_out,
                              const uint32_t* wq, const uint8_t* sw, const float* gs_w, int64_t M, int64_t N,
                              int64_t K, int mode, void* ws, uint16_t* out, int inject_timeout, cudaStream_t s);

// weight_stream.cu (measurement aid: the GEMV's weight stream without the GEMV)
cudaError_t launch_weight_stream(const DevInfo& d, const uint32_t* w, const uint8_t* scales, int64_t N,
                                 int64_t K, cudaStream_t s);

// gather_qmm.cu: W4A16 GEMMs (MXFP4 = 1, NVFP4 = 2, affine = 0 weights) -- the MoE
// gather_qmm (rows sorted by expert) and the dense qmm (gs_w: NVFP4 weight global
// scale or nullptr; biases: affine only)
cudaError_t launch_gather_rows(const DevInfo& d, const uint16_t* x, int64_t x_rows, const int32_t* idx, int64_t R,
                               int64_t K, uint16_t* out, cudaStream_t s);
cudaError_t launch_gather_qmm(const DevInfo& d, const uint16_t* x, const int32_t* lhs, const int32_t* rhs, int64_t R,
                              const uint32_t* w, const void* scales, const uint16_t* biases, const float* gs_w,
                              int64_t E, int64_t N, int64_t K, int mode, int group, uint16_t* out, int inject_timeout,
                              cudaStream_t s);
cudaError_t launch_qmm(const DevInfo& d, const uint16_t* x, int64_t M, const uint32_t* w, const void* scales,
                       const uint16_t* biases, const float* gs_w, int64_t N, int64_t K, int mode, int group,
                       uint16_t* out, int inject_timeout, cudaStream_t s);

// kv_cache.cu, kv_attention.cu: the paged 4-bit KV cache (fp4_kv_cache of the C ABI) and
// what works on it
struct KvCacheDesc {
  uint32_t* k_codes = nullptr;
  uint8_t* k_scales = nullptr;
  uint32_t* v_codes = nullptr;
  uint8_t* v_scales = nullptr;
  const float* gs_k = nullptr;
  const float* gs_v = nullptr;
  int64_t num_pages = 0;
  int page_size = 0, kv_heads = 0, head_dim = 0, mode = 0;
};
cudaError_t launch_kv_plan(const DevInfo& d, const int32_t* cached, const int32_t* fresh, int64_t B, int page_size,
                           const int32_t* free_pages, int64_t num_free, int32_t* table, int64_t table_stride,
                           int64_t max_pages, int32_t* total_lens, int32_t* query_start, int64_t* slot_map,
                           int32_t* positions, int64_t T, int32_t* pages_taken, cudaStream_t s);
cudaError_t launch_kv_append(const DevInfo& d, const KvCacheDesc& c, const uint16_t* k, int64_t k_token, int64_t k_head,
                             const uint16_t* v, int64_t v_token, int64_t v_head, const int64_t* slot_map, int64_t T,
                             cudaStream_t s);
struct KvAttentionArgs {
  KvCacheDesc cache;
  const uint16_t* q = nullptr;  // [tokens, q_heads, head_dim]; strides in elements
  int64_t q_token = 0, q_head = 0, tokens = 0;
  int q_heads = 0, batch = 0, max_query_len = 0, max_pages = 0, window = 0;  // window 0: none
  const int32_t* query_start = nullptr;
  const int32_t* total_lens = nullptr;
  const int32_t* block_table = nullptr;
  int64_t table_stride = 0;
  float scale = 0.f;
  uint16_t* out = nullptr;  // [tokens, q_heads, head_dim]
  float* lse = nullptr;     // [tokens, q_heads] or nullptr
  void* ws = nullptr;
  unsigned* err = nullptr;
  int inject_timeout = 0;
};
// norm.cu: the root-mean-square norm (mode 0: no 4-bit output)
struct RmsNormArgs {
  const uint16_t* x = nullptr;  // row strides in elements
  int x_stride = 0;
  const uint16_t* residual = nullptr;  // nullptr: none
  int residual_stride = 0;
  const uint16_t* weight = nullptr;  // nullptr: 1
  float eps = 0.f;
  int rows = 0, cols = 0;
  uint16_t* sum_out = nullptr;  // nullptr: not wanted, as out and xq
  int sum_stride = 0;
  uint16_t* out = nullptr;
  int mode = 0;
  const float* gs = nullptr;
  uint32_t* xq = nullptr;
  uint8_t* scales = nullptr;
  int tiled = 0;
};
cudaError_t launch_rms_norm(const DevInfo& d, const RmsNormArgs& a, cudaStream_t s);

// rope.cu: rotary positions, on their own and on the way into the cache
struct RopeDesc {
  const float2* table = nullptr;  // [positions, rotary_dim / 2]: cos, sin
  int positions = 0, rotary_dim = 0, interleaved = 0;
};
struct HeadsView {  // bf16 [tokens, heads, head_dim]; strides in elements
  const uint16_t* in = nullptr;
  int64_t in_token = 0, in_head = 0;
  uint16_t* out = nullptr;
  int64_t out_token = 0, out_head = 0;
  int heads = 0, dim = 0;
};
cudaError_t launch_rope_table(const DevInfo& d, const double* frequencies, int rotary_dim, double scale,
                              int64_t positions, float* table, cudaStream_t s);
cudaError_t launch_rope(const DevInfo& d, const RopeDesc& r, const HeadsView& x, const int32_t* positions, int64_t T,
                        int backward, cudaStream_t s);
cudaError_t launch_kv_append_rope(const DevInfo& d, const KvCacheDesc& c, const RopeDesc& r, const uint16_t* k,
                                  int64_t k_token, int64_t k_head, const uint16_t* v, int64_t v_token, int64_t v_head,
                                  const int64_t* slot_map, const int32_t* positions, int64_t T, const HeadsView& q,
                                  cudaStream_t s);

// moe.cu: routed rows by expert and back
// (most_ctas: 0, or a limit on the cluster's CTAs)
cudaError_t launch_moe_sort(const DevInfo& d, const int32_t* ids, int64_t T, int k, int E, int32_t* lhs, int32_t* rhs,
                            int32_t* slot, int32_t* offsets, int most_ctas, cudaStream_t s);
cudaError_t launch_moe_combine(const DevInfo& d, const uint16_t* y, int64_t rows, const int32_t* slot,
                               const float* weights, const uint16_t* residual, int64_t T, int k, int cols,
                               uint16_t* out, cudaStream_t s);
cudaError_t launch_moe_combine_backward(const DevInfo& d, const uint16_t* dout, const uint16_t* y, const int32_t* slot,
                                        const float* weights, int64_t T, int k, int cols, int64_t rows,
                                        const int32_t* rows_used, uint16_t* dy, float* dweights, cudaStream_t s);

// the attention's dispatch (kv_attention.cu) and its workspace
size_t kv_attention_ws_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_query_len);
cudaError_t launch_kv_attention(const DevInfo& d, const KvAttentionArgs& args, cudaStream_t s);
// The workspace, the same for both tensor-core kernels and whatever the call's sizes, so that calls of different kinds may
// take turns on one: the two counters of the prompt kernel's hand-out, and a word that is set when a wait expired (what
// is counted here may then be left short, so later calls report it); the arrivals of split items' pieces, eight words for
// the CTA that holds an item's first piece (a CTA begins at most one item that it does not end) -- zero between calls --
// and then results of the pieces, which mean nothing between calls.
constexpr int kKvCtas = 160;  // CTAs of a launch at most (one an SM)
constexpr int kKvExpired = 2;  // that word
constexpr size_t kKvArrivals = 64, kKvResults = kKvArrivals + (size_t)kKvCtas * 8 * 4;
// kv_decode.cu: a few query rows a request, head_dim 64, 128 or 256
bool kv_decode_supported(int head_dim);
size_t kv_decode_ws_bytes(int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_query_len);
cudaError_t launch_kv_decode(const DevInfo& d, const KvAttentionArgs& args, cudaStream_t s);
// kv_prefill.cu: many query rows a request, head_dim 64 or 128
bool kv_prefill_supported(int head_dim);
size_t kv_prefill_ws_bytes(int64_t head_dim);
cudaError_t launch_kv_prefill(const DevInfo& d, const KvAttentionArgs& args, cudaStream_t s);

}  // namespace fp4
