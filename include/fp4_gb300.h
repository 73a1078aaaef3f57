/*
 * fp4_gb300.h -- C ABI of libfp4gb300: block-scaled 4-bit quantization and
 * quantized matmul on one NVIDIA GB300 (sm_103a).
 *
 * Sources (pages cited by title and section):
 *   [P1] "perf(cuda): enable hardware NVFP4/MXFP4 conversion on Blackwell
 *        builds" -- fp_quantize: MXFP4 and NVFP4 share one template; e2m1 by
 *        cvt.rn.satfinite.e2m1x2.f32 on sm_100a-class targets.
 *   [P2] "epic: NVIDIA Volta (sm_70) inference acceleration program #1536" --
 *        Baseline and Diagnosis 3: qmv over affine 4-bit group-64 weights, the
 *        decode-step weight stream; Diagnosis 1 and 5: gather_gemm / grouped
 *        GEMM for MoE.
 *   [P3] "mlx 0.30.7.3 -> 0.30.7.6" -- qqmm.cpp (QQMatmul::eval_gpu,
 *        quantize_input: packed codes [.., K*bits/32] uint32, scales uint8,
 *        W always transposed [N, K]), qqmm_utils.h (128x4 scale tiles, zero
 *        padding, 16-byte aligned start), qqmm_utils.cu (alpha =
 *        amax_x*amax_w/(448*6)^2, beta = 0), quantized.cpp
 *        (fast::Quantize::eval_gpu: optional NVFP4 global scale).
 *   [P4] "mlx: opt-in dense GEMM for nvfp4 prefill ... - #287" -- global scale
 *        representations (multiplier m versus m*2688).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library
 *     keeps none of them after the call returns and allocates nothing.
 *   - bf16 tensors are raw bfloat16 bit patterns (fp4_bf16), row-major and
 *     contiguous.  Packed 4-bit codes are uint32 words: element k of a row is
 *     word k/8, nibble k%8, low nibble first (8 codes per word).
 *   - Work is enqueued on `stream` (stream-ordered, asynchronous).  Arguments
 *     are validated on the host before anything is launched; an invalid call
 *     launches nothing and returns a non-OK status.  No C++ exception crosses
 *     the ABI.  Launch failures return FP4_ERR_CUDA.  A device-side wait that
 *     gives up (bounded spin) records FP4_ERR_TIMEOUT, which
 *     fp4_check_device_error() reports.
 *   - Every size (n, rows, cols, N, K, M, R, E) must be at least 1: an empty
 *     problem returns FP4_ERR_INVALID_ARG and launches nothing.
 *   - NVFP4: e2m1 codes, groups of 16, E4M3 block scales, optional fp32 global
 *     scale gs in the multiplier form gs = amax/2688 (2688 = 448*6).
 *     MXFP4: e2m1 codes, groups of 32, E8M0 block scales.
 *     Affine: unsigned 4-bit q, groups of 32/64/128, bf16 scale and bias,
 *     w = q*scale + bias.
 */
#ifndef FP4_GB300_H
#define FP4_GB300_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t fp4_bf16; /* raw bfloat16 bits */

typedef enum {
  FP4_OK = 0,
  FP4_ERR_INVALID_ARG = 1,  /* null pointer, negative or inconsistent size */
  FP4_ERR_UNSUPPORTED = 2,  /* mode/bits/group combination or device not supported */
  FP4_ERR_ALIGNMENT = 3,    /* a pointer or a row pitch breaks the alignment rule */
  FP4_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
  FP4_ERR_TIMEOUT = 5       /* a bounded device wait expired (see fp4_check_device_error) */
} fp4_status;

typedef enum { FP4_MODE_AFFINE = 0, FP4_MODE_MXFP4 = 1, FP4_MODE_NVFP4 = 2 } fp4_mode;

/* Scale layouts.  LINEAR: row-major [rows, cols/group].
 * TILED_128x4 [P3 qqmm_utils.h]: rows padded to a multiple of 128 and scale
 * columns to a multiple of 4; byte (r, c) sits at
 *   ((r/128)*(Cp/4) + c/4)*512 + (r%32)*16 + ((r%128)/32)*4 + c%4
 * (Cp = padded scale columns), every padding byte is zero, total Rp*Cp bytes. */
typedef enum { FP4_SCALES_LINEAR = 0, FP4_SCALES_TILED_128x4 = 1 } fp4_scale_layout;

/* Checks that `device` is compute capability 10.3 (GB300) and caches its
 * properties.  Every other entry point initializes the current device lazily,
 * so calling this is optional; it is the place to learn FP4_ERR_UNSUPPORTED. */
fp4_status fp4_init(int device);

/* Static string for a status code; never NULL. */
const char* fp4_status_string(fp4_status status);

/* Synchronizes `stream`, then reports and clears the device error word of the
 * current device: FP4_ERR_TIMEOUT if any bounded wait of an earlier launch
 * expired since the last check, FP4_ERR_INVALID_ARG if a kernel found an index
 * argument outside its contract (gather_qmm's expert ids), FP4_ERR_CUDA if the
 * stream reports an error, else FP4_OK. */
fp4_status fp4_check_device_error(cudaStream_t stream);

/* Padded scale-tile dimensions for `rows` x `scale_cols` scales
 * [P3 qqmm_utils.h get_padded_scale_dims]: rows up to a multiple of 128,
 * columns up to a multiple of 4. */
void fp4_padded_scale_dims(int64_t rows, int64_t scale_cols, int64_t* padded_rows,
                           int64_t* padded_cols);

/* Bytes of device workspace fp4_amax_global_scale needs for n elements. */
size_t fp4_amax_workspace_bytes(int64_t n);

/* a1: tensor amax and NVFP4 global scale [P3 quantize_input / compute_qqmm_pointers,
 * P4 global-scale representation].
 *   x        bf16[n], 16-byte aligned, n >= 1
 *   gs_out   device fp32 scalar: fl(amax/2688), the multiplier form m
 *   amax_out device fp32 scalar or NULL: max |x| (MLX's m*2688 form)
 *   ws       device scratch of ws_bytes >= fp4_amax_workspace_bytes(n) bytes;
 *            no initial contents needed; not read after the call completes.
 * NaN inputs give an unspecified result. */
fp4_status fp4_amax_global_scale(const fp4_bf16* x, int64_t n, float* gs_out, float* amax_out,
                                 void* ws, size_t ws_bytes, cudaStream_t stream);

/* a2-a4: fp_quantize [P1; P3 qqmm.cpp quantize_input, quantized.cpp].
 *   x            bf16[rows, cols], 16-byte aligned
 *   mode, bits, group_size: (NVFP4, 4, 16) or (MXFP4, 4, 32); affine quantize is
 *                not provided (FP4_ERR_UNSUPPORTED)
 *   global_scale device fp32 scalar gs (NVFP4 only) or NULL (gs = 1)
 *   xq           uint32[rows, cols/8] packed codes, 8-byte (NVFP4) / 16-byte (MXFP4) aligned
 *   scales       uint8 E4M3/E8M0 block scales in `layout`; for TILED_128x4 the
 *                whole padded buffer (Rp*Cp bytes) is written, padding with 0
 * Per NVFP4 group: b = max|x|, s8 = E4M3_rn_sat(b/(6*gs)) (0 when b = 0),
 *   q = e2m1_rn_sat(x * (1/(s8*gs))) (0 codes with their sign when s8*gs = 0).
 * Per MXFP4 group: se = clamp(floor(log2 b) - 2, -127, 127) (-127 when b = 0),
 *   byte = se + 127, q = e2m1_rn_sat(x * 2^-se).
 * Requires cols % group_size == 0 and rows >= 1. */
fp4_status fp4_quantize(const fp4_bf16* x, int64_t rows, int64_t cols, fp4_mode mode, int bits,
                        int group_size, const float* global_scale, uint32_t* xq, uint8_t* scales,
                        fp4_scale_layout layout, cudaStream_t stream);

/* fp_quantize with stochastic rounding [P1: the NVFP4/MXFP4 quantizer's USE_SR
 * template parameter, which needs the Blackwell converters; the pages state
 * neither the rule nor the random numbers, so both are fixed here].
 * Arguments as fp4_quantize, plus seed and offset.  Block scales are exactly
 * fp4_quantize's.  Each element v = x * mul (mul as fp4_quantize) is rounded to
 * one of its two e2m1 neighbours lo <= |v| < hi: up when the top 24 bits of its
 * random word are below floor(2^24 (|v| - lo) / (hi - lo)), so the expected
 * value is v (to 2^-24 of the step); |v| >= 6 gives 6 and the sign is kept.
 * The random word of element e = r * cols + c is word e % 4 of Philox4x32-10
 * (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", SC 2011) at
 * the 128-bit counter offset + floor(e / 4) (32-bit words little-endian) under
 * the key (low 32 bits of seed, high 32 bits): independent of the launch
 * configuration, so a call is reproducible, and successive calls that advance
 * offset by ceil(rows * cols / 4) never reuse a word. */
fp4_status fp4_quantize_sr(const fp4_bf16* x, int64_t rows, int64_t cols, fp4_mode mode, int bits,
                           int group_size, const float* global_scale, uint64_t seed, uint64_t offset, uint32_t* xq,
                           uint8_t* scales, fp4_scale_layout layout, cudaStream_t stream);

/* a5: fp_dequantize / affine_dequantize [P3 quantized.cpp].
 *   wq      uint32[rows, cols/8]
 *   scales  NVFP4/MXFP4: uint8 block scales in `layout`; affine: bf16[rows, cols/group]
 *           (linear layout only)
 *   biases  affine: bf16[rows, cols/group]; must be NULL otherwise
 *   global_scale NVFP4 only, device fp32 or NULL
 *   out     bf16[rows, cols], 16-byte aligned
 * Each element is the fp32 value code*scale*gs (affine q*scale + bias) rounded
 * to nearest-even bf16. */
fp4_status fp4_dequantize(const uint32_t* wq, const void* scales, const fp4_bf16* biases,
                          int64_t rows, int64_t cols, fp4_mode mode, int bits, int group_size,
                          const float* global_scale, fp4_scale_layout layout, fp4_bf16* out,
                          cudaStream_t stream);

/* a6: qmv, the M = 1 decode GEMV [P2 Baseline, Diagnosis 3; P3 qqmm.cpp fp_qmv route].
 *   y[n] = sum_k x[k] * deq(W)[n, k]   (fp32 accumulation, bf16 output)
 *   x       bf16[K], 16-byte aligned
 *   w       uint32[N, K/8] (W stored [N, K]), 16-byte aligned
 *   scales  linear block scales: uint8[N, K/group] (NVFP4/MXFP4) or bf16 (affine)
 *   biases  affine: bf16[N, K/group]; NULL otherwise
 *   global_scale_w NVFP4 only: device fp32 gs of W, multiplied in the epilogue, or NULL
 *   y       bf16[N]
 * Requires K % 32 == 0 and K % group_size == 0.
 * Launch order: qmv uses programmatic dependent launch and may read w and its
 * scales before the kernel launched just before it on the stream has finished;
 * x, global_scale_w and y are touched only after that kernel completes.  What
 * fp4_quantize and fp4_quantize_sr write is complete before a kernel behind them
 * starts, so any sequence of those calls and qmv is ordered.  A kernel that writes
 * w or scales and triggers its dependents early must not directly precede qmv: a
 * caller's own, or rms_norm, whose codes are activations.
 * A NaN or infinity in x gives non-finite rows (tensor-core path, NVFP4 and MXFP4: NaN). */
fp4_status qmv(const fp4_bf16* x, const uint32_t* w, const void* scales, const fp4_bf16* biases,
               const float* global_scale_w, int64_t N, int64_t K, fp4_mode mode, int bits,
               int group_size, fp4_bf16* y, cudaStream_t stream);

/* The weights of one GEMV launch: up to 4 matrices of the same K, each given as
 * qmv takes it (biases: affine only; global_scale_w: NVFP4 only, may be NULL). */
typedef struct fp4_matrix_group {
  int count; /* 1 .. 4 */
  const uint32_t* w[4];
  const void* scales[4];
  const fp4_bf16* biases[4];
  const float* global_scale_w[4];
  int64_t N[4];
  int64_t K;
} fp4_matrix_group;

/* qmv_grouped: the decode GEMV of one x against the matrices of `mats` in one
 * launch -- the projections that multiply the same activation (q, k and v;
 * gate and up) stored as separate matrices [P2 Baseline: the decode step is the
 * qmv weight stream; grouping them pays the per-launch fixed cost once].
 *   y[i] = x . deq(W_i)^T  for i < mats->count (each y[i] as qmv computes it);
 *   y: a HOST array of mats->count device pointers.
 * prefetch_next (NULL: none): the weights of the GEMV the caller launches next
 * on this stream, same mode.  A hint: once this launch has issued its own
 * weight loads, it warms L2 with the first stages that launch will read, so
 * that its start does not wait on DRAM.  It is validated like `mats` (its
 * pointers must be device memory); nothing is written through it.
 * NVFP4 and MXFP4 run as one tensor-core launch, affine as one launch of the
 * affine GEMV, when the stacked rows have a plan and every scale (and bias)
 * row is 16-byte aligned; other cases run as mats->count qmv launches (and
 * ignore the hint).  Otherwise qmv's rules. */
fp4_status qmv_grouped(const fp4_bf16* x, const fp4_matrix_group* mats, fp4_mode mode, int bits, int group_size,
                       fp4_bf16* const* y, const fp4_matrix_group* prefetch_next, cudaStream_t stream);

/* qqmv: the one-row route of the quantized-activation matmul [P3 qqmm.cpp,
 * QQMatmul::eval_gpu: with quantized W and a single row of x, x goes through
 * fp_quantize_dequantize into an array of x's dtype and then through fp_qmv].
 *   y[n] = sum_k xhat[k] * deq(W)[n, k]   (fp32 accumulation, bf16 output)
 *   xhat = fp4_dequantize(fp4_quantize(x)): per block of 16 (NVFP4, global scale
 *          global_scale_x or 1) or 32 (MXFP4) the rule of fp4_quantize, then each
 *          value bf16_rn(fl(fl(e2m1(q) * scale) * gs_x)) -- x's own dtype, as the
 *          page's route stores it.  The quantization happens inside the GEMV
 *          kernel (no extra launch, no scratch).
 *   x, w, scales, global_scale_w, y, N, K: as for qmv (linear scales); mode is
 *          NVFP4 or MXFP4; global_scale_x (device fp32 or NULL) is NVFP4 only.
 * Requires K % 32 == 0 (hence whole blocks) and K <= 65536.  Launch order as qmv. */
fp4_status qqmv(const fp4_bf16* x, const float* global_scale_x, const uint32_t* w, const uint8_t* scales,
                const float* global_scale_w, int64_t N, int64_t K, fp4_mode mode, fp4_bf16* y,
                cudaStream_t stream);

/* a7-a9: qqmm, the FP4 x FP4 GEMM [P3 qqmm.cpp, qqmm_impl, qqmm_utils.cu].
 *   out[m, n] = bf16( alpha * sum_k deq(xq)[m, k] * deq(wq)[n, k] ),  beta = 0
 *   alpha = (*global_scale_x) * (*global_scale_w); a NULL pointer counts as 1.
 *   With multiplier-form global scales this is amax_x*amax_w/(448*6)^2.  To pass a
 *   precomputed alpha, give it as global_scale_x and NULL as global_scale_w.
 *   xq      uint32[M, K/8], 16-byte aligned (NVFP4 or MXFP4 codes)
 *   sx      uint8 block scales of xq, TILED_128x4 layout
 *   wq      uint32[N, K/8] (W stored [N, K]), 16-byte aligned
 *   sw      uint8 block scales of wq, TILED_128x4 layout
 *   out     bf16[M, N], 16-byte aligned
 * Requires K % 256 == 0 (hence K % 64 == 0 for the tensor-core K step), N % 8 == 0,
 * M >= 1.  mode is NVFP4 (E4M3 scales, group 16) or MXFP4 (E8M0, group 32). */
fp4_status qqmm(const uint32_t* xq, const uint8_t* sx, const uint32_t* wq, const uint8_t* sw,
                const float* global_scale_x, const float* global_scale_w, int64_t M, int64_t N,
                int64_t K, fp4_mode mode, fp4_bf16* out, cudaStream_t stream);

/* a10: gather_qmm, the MoE grouped GEMM with 4-bit weights and bf16 activations
 * [P2 Diagnosis 1 and 5: gather_gemm / grouped GEMM].
 *   out[r, n] = sum_k x[lhs_idx[r], k] * deq(w[rhs_idx[r]])[n, k]  (fp32 accumulation)
 *   x        bf16[T, K] activations (T = 1 + max lhs_idx), 16-byte aligned
 *   lhs_idx  int32[R] activation row of each routed row
 *   rhs_idx  int32[R] expert of each routed row, in [0, E)
 *   w        uint32[E, N, K/8], 16-byte aligned
 *   scales   MXFP4 uint8[E, N, K/32] E8M0, NVFP4 uint8[E, N, K/16] E4M3 (no global
 *            scale), affine bf16[E, N, K/group]; linear layout, 2-byte aligned
 *   biases   affine: bf16[E, N, K/group]; NULL otherwise
 *   out      bf16[R, N], 16-byte aligned
 * sorted != 0 promises rhs_idx is non-decreasing (rows grouped by expert), which
 * this version requires.  Requires K % 64 == 0 and N % 16 == 0.  The expert ids
 * live in device memory, so the kernel checks them: an id outside [0, E) or a
 * decrease leaves the affected output rows unwritten and makes the next
 * fp4_check_device_error return FP4_ERR_INVALID_ARG.  lhs_idx values must lie in
 * [0, T); they are not checked.  A tile whose routed rows are consecutive rows
 * of x (activations already in routed order, e.g. after gather_rows) loads
 * them by TMA; scattered rows are gathered 16 bytes at a time. */
fp4_status gather_qmm(const fp4_bf16* x, const int32_t* lhs_idx, const int32_t* rhs_idx, int64_t R,
                      const uint32_t* w, const void* scales, const fp4_bf16* biases, int64_t E,
                      int64_t N, int64_t K, fp4_mode mode, int bits, int group_size, int sorted,
                      fp4_bf16* out, cudaStream_t stream);

/* gather_rows: the routed activations in routing order [P2 Diagnosis 5: the
 * MoE grouped GEMM gathers each routed row's activations], so that a following
 * gather_qmm with lhs_idx = 0 .. R-1 reads them as whole tiles.
 *   out[i, :] = x[idx[i], :]   for i < R (pure data movement, bit-exact)
 *   x      bf16[x_rows, K], 16-byte aligned;  idx int32[R], 4-byte aligned
 *   out    bf16[R, K], 16-byte aligned, caller-owned (R K 2 bytes)
 * Requires K % 8 == 0.  An index outside [0, x_rows) leaves its output row
 * unwritten and makes the next fp4_check_device_error return
 * FP4_ERR_INVALID_ARG. */
fp4_status gather_rows(const fp4_bf16* x, int64_t x_rows, const int32_t* idx, int64_t R, int64_t K, fp4_bf16* out,
                       cudaStream_t stream);

/* qqmm_batched: batch_count independent FP4 x FP4 GEMMs in one launch [P3
 * qqmm_impl: the page's cuBLASLt call fixes the batch count at 1; this is the
 * strided-batch generalization].
 *   out_b = bf16( gs_x[b] * gs_w[b] * Xq_b . Wq_b^T ),  b = 0 .. batch - 1
 *   Xq_b = xq + b * stride_xq (uint32 words), its tiled scales sx + b * stride_sx (bytes);
 *   Wq_b = wq + b * stride_wq, scales sw + b * stride_sw; a stride of 0 shares one W
 *   (and its scales) across the batch; out_b = out + b * stride_out (elements).
 *   global_scale_x / global_scale_w: device fp32 arrays of `batch` values, or NULL (1).
 * Each batch follows qqmm's rules (M, N, K, layouts, alignment).  The strides
 * must keep the batches apart (stride_xq >= M K / 8, stride_sx >= the padded
 * scale bytes, stride_out >= M N, and likewise for W unless 0) and aligned
 * (16 bytes for codes and scales, 8 elements for out); batch <= 65535. */
fp4_status qqmm_batched(const uint32_t* xq, const uint8_t* sx, const uint32_t* wq, const uint8_t* sw,
                        const float* global_scale_x, const float* global_scale_w, int64_t batch, int64_t M,
                        int64_t N, int64_t K, int64_t stride_xq, int64_t stride_sx, int64_t stride_wq,
                        int64_t stride_sw, int64_t stride_out, fp4_mode mode, fp4_bf16* out, cudaStream_t stream);

/* Workspace bytes qqmm_quantize_x needs for an M x K activation. */
size_t qqmm_quantize_x_workspace_bytes(int64_t M, int64_t K, fp4_mode mode);

/* qqmm_quantize_x: the quantized-activation GEMM with the activation's
 * quantization fused into the same launch [P3 qqmm.cpp: QQMatmul::eval_gpu
 * quantizes x with quantize_input (fp_quantize, optional global scale) and then
 * calls the block-scaled GEMM -- separate launches there].
 *   out = bf16( gs_x * gs_w * fp4_quantize(x, gs_x) . Wq^T ), bit for bit what
 *   fp4_amax_global_scale (when global_scale_x is NULL) + fp4_quantize (tiled
 *   scales) + qqmm compute.
 *   x        bf16[M, K], 16-byte aligned
 *   global_scale_x  NVFP4: device fp32 activation global scale (a calibrated value),
 *            or NULL to take fl(amax(x) / 2688) from x; MXFP4: must be NULL
 *   global_scale_x_out  NVFP4 only, nullable: receives the activation scale used
 *   wq, sw, global_scale_w, M, N, K, mode, out: as for qqmm
 *   ws       device workspace of ws_bytes >= qqmm_quantize_x_workspace_bytes(M, K, mode)
 *            bytes, 128-byte aligned.  It must be zero-filled once when allocated;
 *            each call leaves its grid-barrier words ready for the next.  The
 *            quantized x (codes, then 128x4-tiled scales) sits at its start.
 *            Calls that overlap on the GPU must not share a workspace.
 * One persistent cooperative launch: every CTA quantizes a share of x (after a
 * grid-wide amax when NVFP4 has no activation scale), a grid barrier, then the
 * GEMM reads the quantized x from the workspace (still in L2).  The launch needs
 * every CTA resident (at most one per SM); a device that cannot co-schedule it
 * returns FP4_ERR_CUDA. */
fp4_status qqmm_quantize_x(const fp4_bf16* x, const float* global_scale_x, const uint32_t* wq, const uint8_t* sw,
                           const float* global_scale_w, int64_t M, int64_t N, int64_t K, fp4_mode mode, void* ws,
                           size_t ws_bytes, float* global_scale_x_out, fp4_bf16* out, cudaStream_t stream);

/* qmm: the dense prefill GEMM with 4-bit weights and bf16 activations (W4A16)
 * ["mlx: opt-in dense GEMM for nvfp4 prefill ... - #287": the mixed-input GEMM
 * of bf16 activations against NVFP4 weights at M > 1; "perf(cuda): enable
 * hardware NVFP4/MXFP4 conversion on Blackwell builds": qmm_sm80].
 *   out[m, n] = sum_k x[m, k] * deq(W)[n, k]   (fp32 accumulation, bf16 output)
 *   x        bf16[M, K], 16-byte aligned
 *   w        uint32[N, K/8] (W stored [N, K]), 16-byte aligned
 *   scales   linear block scales: NVFP4 uint8[N, K/16], MXFP4 uint8[N, K/32], affine
 *            bf16[N, K/group]; 2-byte aligned
 *   biases   affine: bf16[N, K/group]; NULL otherwise
 *   global_scale_w NVFP4 only: device fp32 gs of W (applied to the fp32 sums), or NULL
 *   out      bf16[M, N], 16-byte aligned
 * The weights are dequantized exactly (FP4: e2m1 * block scale is exact in bf16;
 * affine: q * scale + bias in fp32 carried as two bf16 terms).  Requires
 * K % 64 == 0 and N % 16 == 0. */
fp4_status qmm(const fp4_bf16* x, const uint32_t* w, const void* scales, const fp4_bf16* biases,
               const float* global_scale_w, int64_t M, int64_t N, int64_t K, fp4_mode mode, int bits, int group_size,
               fp4_bf16* out, cudaStream_t stream);

/* Maximum element count accepted by fp4_amax_global_scale_noalloc (2^36). */
#define FP4_AMAX_NOALLOC_MAX_ELEMS ((int64_t)1 << 36)

/* Allocation-free variant of fp4_amax_global_scale.  The pages have no
 * counterpart: this entry point exists for callers that cannot allocate device
 * memory where they need a global scale -- code recording into a CUDA stream
 * capture, engines that hand every kernel a pre-planned memory arena, hosts
 * that forbid allocation on a latency-critical path.  The per-block partial
 * maxima that fp4_amax_global_scale keeps in caller scratch live here in a
 * fixed 4 KiB file-scope device array (1024 partials) that every GPU loading
 * the library holds until the process exits.  The results are identical to
 * fp4_amax_global_scale's.
 *   x, n, gs_out, amax_out: as for fp4_amax_global_scale; n in [1, 2^36],
 *            larger n returns FP4_ERR_INVALID_ARG.
 * Nothing is allocated or freed, by this library or through any allocating
 * library routine.  The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress) and checks the compute capability; make that
 * first call before any stream capture.  All calls share the array and it keeps
 * the last call's contents (each call writes every slot it reads, so nothing
 * needs clearing); calls that overlap on the GPU -- unordered streams -- race
 * on it and give unspecified results. */
fp4_status fp4_amax_global_scale_noalloc(const fp4_bf16* x, int64_t n, float* gs_out, float* amax_out,
                                         cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Serving: a paged KV cache held in 4 bits, the plan that places a step's tokens
 * in it, the append that fills it and the attention that reads it.
 *
 * One layer's cache is four matrices of this header's formats (linear scales,
 * mode NVFP4 or MXFP4), each with one row of head_dim elements per (page, kv
 * head, slot):
 *   k_codes, v_codes    uint32[num_pages, kv_heads, page_size, head_dim/8]
 *   k_scales, v_scales  uint8[num_pages, kv_heads, page_size, head_dim/group]
 * so fp4_dequantize reads it as num_pages*kv_heads*page_size rows.  All four are
 * 16-byte aligned.  global_scale_k / global_scale_v: NVFP4 only, device fp32
 * multiplier-form global scales of K and V (or NULL: 1); fixed for the cache's
 * life, since every stored row was quantized with them.
 * page_size is 16, 32, 64 or 128; head_dim a multiple of 32, at most 256;
 * num_pages * kv_heads * page_size < 2^31.  Slot s of the cache is slot
 * s % page_size of page s / page_size. */
typedef struct fp4_kv_cache {
  uint32_t* k_codes;
  uint8_t* k_scales;
  uint32_t* v_codes;
  uint8_t* v_scales;
  const float* global_scale_k;
  const float* global_scale_v;
  int64_t num_pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  fp4_mode mode;
} fp4_kv_cache;

/* kv_plan: block tables, slots and positions of a step, from the requests'
 * lengths, in one launch (capturable: lengths stay on the device).
 *   cached_lens  int32[batch] tokens already in the cache;  new_lens int32[batch]
 *                tokens this step adds (0 allowed in both)
 *   free_pages   int32[num_free] page ids, taken from the front
 *   block_table  int32[batch, table_stride], the first max_pages entries of a row used,
 *                in/out: entries below ceil(cached/page_size) are read; request b's
 *                further entries up to ceil((cached+new)/page_size) are written with
 *                free pages, in request order
 *   total_lens   int32[batch] out: cached + new
 *   query_start  int32[batch+1] out: first token of each request, then their number
 *   slot_map     int64[tokens] out: cache slot of each token;  positions int32[tokens]
 *                out: its position.  Entries past the step's tokens are -1.
 *   pages_taken  int32 scalar out: free pages used
 * total_lens must not overlap cached_lens.  Negative lengths count as 0.  If the free list
 * runs out, a row of the table is full, or the step has more than `tokens`
 * tokens, the tokens concerned get slot -1 (or no entry), nothing outside the
 * arrays is touched, and the next fp4_check_device_error returns
 * FP4_ERR_INVALID_ARG.  batch <= 16384. */
fp4_status kv_plan(const int32_t* cached_lens, const int32_t* new_lens, int64_t batch, int page_size,
                   const int32_t* free_pages, int64_t num_free, int32_t* block_table, int64_t table_stride,
                   int64_t max_pages, int32_t* total_lens, int32_t* query_start, int64_t* slot_map,
                   int32_t* positions, int64_t tokens, int32_t* pages_taken, cudaStream_t stream);

/* kv_append: the step's new K and V rows, quantized by fp4_quantize's rule (bit
 * for bit its codes and scales), into their slots of the cache.
 *   k, v       bf16[tokens, kv_heads, head_dim], 16-byte aligned; strides in elements
 *              between tokens and between heads, multiples of 8 (views of a fused
 *              q|k|v row are read in place)
 *   slot_map   int64[tokens]; a negative slot skips the token, a slot past the cache
 *              skips it and makes the next fp4_check_device_error return
 *              FP4_ERR_INVALID_ARG; two tokens of one call must not share a slot. */
fp4_status kv_append(const fp4_kv_cache* cache, const fp4_bf16* k, int64_t k_token_stride, int64_t k_head_stride,
                     const fp4_bf16* v, int64_t v_token_stride, int64_t v_head_stride, const int64_t* slot_map,
                     int64_t tokens, cudaStream_t stream);

/* Workspace bytes kv_attention needs (any argument out of range: 0). */
size_t kv_attention_workspace_bytes(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                    int64_t max_query_len);

/* kv_attention: causal attention of the step's queries over the cache.
 *   out[t, h] = sum_j p_j V_j / sum_j p_j,  p_j = exp(softmax_scale * q[t, h] . K_j)
 * for token t of request b (query_start[b] <= t < query_start[b+1]) at position
 * pos = total_lens[b] - (query_start[b+1] - t), over the keys j with 0 <= j <= pos
 * and, when window > 0, j > pos - window, of kv head h / (q_heads / kv_heads).
 * A row that sees no key gives zeros (lse = -inf); a negative total counts as 0.
 * softmax_scale is positive and finite.
 *   q            bf16[tokens, q_heads, head_dim], 16-byte aligned; strides in elements,
 *                multiples of 8;  q_heads a multiple of kv_heads
 *   query_start  int32[batch+1], total_lens int32[batch] (kv_plan's outputs, after
 *                kv_append); tokens outside every request's range are not written
 *   block_table  int32[batch, table_stride], max_pages entries of a row valid; pages that
 *                no query of the request can see are not read (a sliding window's
 *                freed pages may be stale)
 *   max_query_len  the longest request's query count, at least 1: it picks the kernel
 *   ws           device workspace, 16-byte aligned, ws_bytes >=
 *                kv_attention_workspace_bytes(batch, q_heads, kv_heads, head_dim,
 *                max_query_len); zero-filled once when allocated, each call leaves it
 *                ready for the next, but for one whose wait expired (FP4_ERR_TIMEOUT):
 *                it sets the workspace's third 32-bit word, and later calls report
 *                FP4_ERR_TIMEOUT too until the workspace is zero-filled again.
 *                Calls that overlap on the GPU must not share one.
 *                Calls of any kind may take turns on one workspace that has the bytes each
 *                needs: one sized for the longest max_query_len serves shorter ones.
 *   out          bf16[tokens, q_heads, head_dim], 16-byte aligned
 *   lse          fp32[tokens, q_heads] or NULL: log of the sum of exp(score), with which
 *                results over disjoint keys can be merged
 * What is held in fewer bits than fp32: the probabilities, of which the product with
 * V takes bf16's 8 bits or, with few query rows, where its range allows f16's 8 to
 * 11; their sum takes them unrounded.
 * Scores, softmax statistics and sums are fp32, a score within fp32's rounding of
 * the sum of its products.  With few query rows (up to 32 a kv head, or head_dim
 * 256) what lies below 2^-23 of a query row's largest element is not seen by its
 * scores.  A score's size is to stay below 2^30 (fp32 rounds larger ones by whole
 * powers of e: rows may then be zeros or NaN), and with few rows the scales of an
 * MXFP4 K between 2^-100 and 2^110 (a row's products are formed with its largest
 * element brought to between 128 and 256).  With more rows, where a sum of p V
 * passes fp32 (MXFP4), the rows concerned are summed again with p 2^60 smaller, and
 * beside such channels those below about 2^-66 are lost.
 * Slots that no query of the call sees may hold anything; a value of V that is NaN
 * for one query of a request (a NaN scale) may make the request's other queries of
 * the same call NaN too, those before it among them (their probability of it is 0,
 * and 0 NaN is NaN).
 * A page id outside [0, num_pages),
 * a request with more than max_query_len queries or more tokens than its table
 * row holds makes the next fp4_check_device_error return FP4_ERR_INVALID_ARG
 * and leaves that request's rows unspecified; nothing outside the arrays is read. */
fp4_status kv_attention(const fp4_kv_cache* cache, const fp4_bf16* q, int64_t q_token_stride, int64_t q_head_stride,
                        int64_t tokens, int64_t q_heads, const int32_t* query_start, const int32_t* total_lens,
                        int64_t batch, const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                        int64_t max_query_len, float softmax_scale, int64_t window, void* ws, size_t ws_bytes,
                        fp4_bf16* out, float* lse, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Around a decoder layer's products: the norm in front of one, the positions'
 * rotation between the projection and the cache, the experts' rows and back. */

/* rms_norm: root-mean-square norm of the rows of x, after the residual's addition,
 * out in bf16, in 4 bits, or both.
 *   h[r, c] = x[r, c] + residual[r, c]        (residual NULL: h = x; fp32)
 *   rstd[r] = 1 / sqrt(mean over c of h[r, c]^2 + eps)
 *   y[r, c] = (h[r, c] * rstd[r]) * weight[c] (weight NULL: h * rstd; fp32)
 *   sum_out = bf16(h), out = bf16(y), xq and scales = fp4_quantize's rule on the fp32
 *   y: b is the block's largest |y| in fp32, nothing is rounded to bf16 on the way.
 *   x        bf16[rows, cols], 16-byte aligned; row strides in elements, multiples of 8
 *   residual bf16[rows, cols] or NULL, as x;  weight bf16[cols] or NULL, 16-byte aligned
 *   sum_out  bf16[rows, cols] or NULL, as x; may be residual or x itself (same stride)
 *   out      bf16[rows, cols] or NULL, contiguous, 16-byte aligned; may be x itself
 *   xq       uint32[rows, cols/8] or NULL (at least one of out and xq), 8-byte aligned;
 *            mode, global_scale, scales, layout: as for fp4_quantize, read only with xq
 * rstd is held in fp32 from a sum of squares that is off by less than 2^-23 of itself
 * (2^-22 in rows of up to 1024 columns several of which hold most of it), so within one
 * unit of fp32's last place (two); it holds over bf16's whole range (squares that fp32
 * cannot hold are summed in fp64).  A row
 * of zeros gives zeros also where eps is 0.  An infinity or a NaN in a row gives what the
 * formula gives in out (NaN), and unspecified codes.
 * Requires cols a multiple of 8 (with xq, of 16 or 32, the group), at most 32768;
 * eps in [0, 1]. */
fp4_status rms_norm(const fp4_bf16* x, int64_t x_stride, const fp4_bf16* residual, int64_t residual_stride,
                    const fp4_bf16* weight, float eps, int64_t rows, int64_t cols, fp4_bf16* sum_out,
                    int64_t sum_stride, fp4_bf16* out, fp4_mode mode, const float* global_scale, uint32_t* xq,
                    uint8_t* scales, fp4_scale_layout layout, cudaStream_t stream);

/* Rotary positions.  Pair i of a head (0 <= i < rotary_dim / 2) is turned by an angle
 * that grows with the position, and scaled:
 *   (a, b) -> (a cos - b sin, b cos + a sin),  cos and sin: table[position][i]
 * Pair i is channels (i, i + rotary_dim/2), or (2 i, 2 i + 1) when interleaved is not
 * 0; channels from rotary_dim on stay as they are.
 *   table      fp32[positions, rotary_dim/2, 2]: cos and sin, 8-byte aligned (rope_table
 *              fills one; a caller's own is as good)
 *   rotary_dim even, 2 .. 256 */
typedef struct fp4_rope {
  const float* table;
  int64_t positions;
  int32_t rotary_dim;
  int32_t interleaved;
} fp4_rope;

/* How the angles are scaled for contexts longer than the trained one.  f_i = base^(-2 i / rotary_dim)
 * radians a position, L = original_positions:
 *   NONE        f_i
 *   LINEAR      f_i / factor
 *   BASE        base * factor^(rotary_dim / (rotary_dim - 2)) in place of base (rotary_dim 2: base)
 *   WAVELENGTH  with t = L f_i / 2 pi, the pair's turns over L, and s = (t - low) / (high - low) held to
 *               [0, 1]:  (1 - s) f_i / factor + s f_i
 *   RAMP        the same blend over the pairs' numbers: with n(t) = rotary_dim ln(L / (2 pi t)) / (2 ln base),
 *               first = max(floor n(high), 0), last = min(ceil n(low), rotary_dim - 1),
 *               s = 1 - (i - first) / max(last - first, 0.001) held to [0, 1]; and cos and sin are multiplied
 *               by 0.1 ln(factor) + 1 */
typedef enum {
  FP4_ROPE_NONE = 0,
  FP4_ROPE_LINEAR = 1,
  FP4_ROPE_BASE = 2,
  FP4_ROPE_WAVELENGTH = 3,
  FP4_ROPE_RAMP = 4
} fp4_rope_scaling;

/* rope_frequencies (host only): frequencies[i], i < rotary_dim / 2, in radians a position, and what cos and sin
 * are multiplied by, in fp64.  base > 1; factor >= 1 (NONE: not read); low < high and original_positions >= 1
 * for WAVELENGTH and RAMP (else not read), low > 0 for RAMP.  frequencies and scale: HOST memory. */
fp4_status rope_frequencies(int rotary_dim, double base, fp4_rope_scaling scaling, double factor,
                            int64_t original_positions, double low, double high, double* frequencies, double* scale);

/* rope_table: cos and sin of positions 0 .. positions - 1, each scale * cos(position * frequency) and
 * scale * sin(...) rounded once from fp64.  The angle is formed as a 64-bit fraction of a turn, so it is exact
 * to 2^-33 of a turn at any position.
 *   frequencies  HOST array of rotary_dim / 2 finite values (copied before the call returns)
 *   table        device fp32[positions, rotary_dim/2, 2], 8-byte aligned
 * positions in [1, 2^31). */
fp4_status rope_table(const double* frequencies, int rotary_dim, double scale, int64_t positions, float* table,
                      cudaStream_t stream);

/* rope: the rotation of a [tokens, heads, head_dim] view, or (backward != 0) its transpose: the gradient by x of
 * the gradient by the result.  fp32 products, one rounding to bf16.
 *   x, out     bf16[tokens, heads, head_dim], 16-byte aligned; strides in elements, multiples of 8; out may be x
 *              itself (same strides), else they do not overlap
 *   positions  int32[tokens]; a token with a negative position (padding) is not written; one past the table is not
 *              written and makes the next fp4_check_device_error return FP4_ERR_INVALID_ARG
 * Requires head_dim a multiple of 8, at most 256, rotary_dim <= head_dim, at most 65535 heads, strides below 2^31 (that of
 * a single token or head: any from head_dim on). */
fp4_status rope(const fp4_rope* rope, const fp4_bf16* x, int64_t x_token_stride, int64_t x_head_stride,
                const int32_t* positions, int64_t tokens, int64_t heads, int64_t head_dim, int backward, fp4_bf16* out,
                int64_t out_token_stride, int64_t out_head_stride, cudaStream_t stream);

/* kv_append_rope: kv_append with K rotated on the way (fp32; not rounded to bf16 between rotation and
 * quantization), and the step's queries rotated by the same launch.
 *   cache, k, v, slot_map, tokens: as for kv_append;  rope, positions: as for rope
 *   q, q_out   bf16[tokens, q_heads, head_dim], as rope's x and out (q_out may be q), or both NULL (q_heads 0); q_out
 *              overlaps neither k nor v, which are read at the same time
 * A token with a negative position is skipped altogether; one with a negative slot has its q rotated only.  A
 * position past the table skips the token, a slot past the cache its K and V, and either makes the next
 * fp4_check_device_error return FP4_ERR_INVALID_ARG. */
fp4_status kv_append_rope(const fp4_kv_cache* cache, const fp4_rope* rope, const fp4_bf16* k, int64_t k_token_stride,
                          int64_t k_head_stride, const fp4_bf16* v, int64_t v_token_stride, int64_t v_head_stride,
                          const int64_t* slot_map, const int32_t* positions, int64_t tokens, const fp4_bf16* q,
                          int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads, fp4_bf16* q_out,
                          int64_t q_out_token_stride, int64_t q_out_head_stride, cudaStream_t stream);

/* moe_sort: the routed rows in order of their experts, as gather_rows and gather_qmm take them, in one launch
 * without workspace (capturable: the routing stays on the device).  R = tokens * k routed rows; entry (t, j) of ids
 * is routed row t * k + j.
 *   ids      int32[tokens, k] expert of each; a negative one is dropped, one that is num_experts or more is dropped
 *            and makes the next fp4_check_device_error return FP4_ERR_INVALID_ARG
 *   lhs_idx  int32[R] out: token of each sorted row, by expert and within an expert by routed row (stable)
 *   rhs_idx  int32[R] out: its expert
 *   slot     int32[tokens, k] out: where each routed row went, -1 if it was dropped
 *   offsets  int32[num_experts + 1] out: first sorted row of each expert, then the number of rows kept
 * The outputs are four buffers of their own, none of them ids (which are read twice).
 * Sorted rows from offsets[num_experts] on (as many as were dropped) get token 0 and the last expert, so that the
 * lists stay what gather_qmm wants; no slot names them.
 * num_experts and k in [1, 1024], R <= 2^30.  Above 2048 routed rows a cluster of 16 CTAs sorts, of eight or one where the
 * device has no room for them. */
fp4_status moe_sort(const int32_t* ids, int64_t tokens, int64_t k, int64_t num_experts, int32_t* lhs_idx,
                    int32_t* rhs_idx, int32_t* slot, int32_t* offsets, cudaStream_t stream);

/* moe_combine: the experts' rows back to their tokens, weighted.
 *   out[t] = residual[t] + sum over j of weights[t, j] * y[slot[t, j]]    (fp32, in order of j; one rounding to bf16)
 *   y         bf16[rows, cols], 16-byte aligned;  slot int32[tokens, k] (moe_sort's); a negative slot adds nothing,
 *             one that is rows or more adds nothing and makes the next fp4_check_device_error return FP4_ERR_INVALID_ARG
 *   weights   fp32[tokens, k] or NULL (1: with the gradient of the sorted rows as y, the gradient of their gather)
 *   residual  bf16[tokens, cols] or NULL (0), 16-byte aligned
 *   out       bf16[tokens, cols], 16-byte aligned; may be residual itself
 * Requires cols a multiple of 8, k in [1, 1024]. */
fp4_status moe_combine(const fp4_bf16* y, int64_t rows, const int32_t* slot, const float* weights,
                       const fp4_bf16* residual, int64_t tokens, int64_t k, int64_t cols, fp4_bf16* out,
                       cudaStream_t stream);

/* moe_combine_backward: the gradients of moe_combine (that of residual is dout).
 *   dy[slot[t, j]] = bf16(weights[t, j] * dout[t]);   dweights[t, j] = dout[t] . y[slot[t, j]]   (fp32, in a fixed order)
 *   dout      bf16[tokens, cols];  slot: as for moe_combine, no row named twice;  weights: fp32 or NULL (1)
 *   y         bf16[rows, cols], read only for dweights (NULL without it)
 *   rows_used device int32 or NULL: rows of dy from *rows_used on are set to zero (moe_sort's offsets + num_experts:
 *             the rows that no slot names); without it rows that no slot names are left as they were
 *   dy        bf16[rows, cols];  dweights fp32[tokens, k] or NULL; 0 where the slot is negative
 * All bf16 tensors 16-byte aligned.  Requires cols a multiple of 8, k in [1, 1024]. */
fp4_status moe_combine_backward(const fp4_bf16* dout, const fp4_bf16* y, const int32_t* slot, const float* weights,
                                int64_t tokens, int64_t k, int64_t cols, int64_t rows, const int32_t* rows_used,
                                fp4_bf16* dy, float* dweights, cudaStream_t stream);

/* Test hook, off by default: when `enable` is nonzero the next launches of the
 * tensor-core kernels -- qqmm, qmv's NVFP4/MXFP4 path, gather_qmm and kv_attention
 * (head_dim 64, 128 or 256) -- make
 * their MMA-issuing thread wait on a barrier nothing arrives at, with a 1 ms
 * limit, before doing their normal work.  The wait expires, the kernel records
 * FP4_ERR_TIMEOUT and still completes with a correct result; nothing faults or
 * hangs. */
fp4_status fp4_debug_inject_wait_timeout(int enable);

/* Test hook, off by default (0): the next launches of moe_sort use clusters of at most `most` CTAs, as they do where
 * the device has no room for more side by side (16, 8 or 1).  The results are the same. */
fp4_status fp4_debug_limit_sort_ctas(int most);

/* Measurement aid (no counterpart on the pages): moves NVFP4 weights from HBM
 * into shared memory exactly as qmv's tensor-core path streams them -- the same
 * split of K over CTAs, rows per CTA and ring of slots, one TMA box of R rows x
 * 128 bytes of codes and one of R rows x 16 bytes of scales per K = 256 stage,
 * programmatic dependent launch, consumption after the previous kernel -- and
 * computes nothing.  Timing it over the same weights as qmv gives the
 * launch-and-stream ceiling of that kernel shape.
 *   w       uint32[N, K/8], 16-byte aligned      scales  uint8[N, K/16], 16-byte aligned
 * Requires K % 256 == 0; a shape the tensor-core path does not take returns
 * FP4_ERR_UNSUPPORTED. */
fp4_status fp4_debug_stream_weights(const uint32_t* w, const uint8_t* scales, int64_t N, int64_t K,
                                    cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif
