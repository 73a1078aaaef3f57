"""Thin Python binding of libfp4gb300 (ctypes).

Functions carry the C ABI's names and only marshal arguments: shapes and
device pointers of torch tensors, the current CUDA stream, and output
allocation with torch (PyTorch is the memory allocator here, nothing more).
Every step of the computation runs in the library's CUDA kernels; there is no
CPU fallback -- if the shared library is missing the first call raises.

Packed 4-bit codes are held in ``torch.int32`` tensors (uint32 bit patterns),
scales in ``torch.uint8`` (NVFP4/MXFP4) or ``torch.bfloat16`` (affine).
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp4gb300.so")

FP4_OK, FP4_ERR_INVALID_ARG, FP4_ERR_UNSUPPORTED, FP4_ERR_ALIGNMENT, FP4_ERR_CUDA, FP4_ERR_TIMEOUT = range(6)
MODE_AFFINE, MODE_MXFP4, MODE_NVFP4 = 0, 1, 2
SCALES_LINEAR, SCALES_TILED = 0, 1
GROUP = {MODE_NVFP4: 16, MODE_MXFP4: 32, MODE_AFFINE: 64}

_lock = threading.Lock()
_lib = None

# (name, restype, argtypes) of every entry point the header declares
c = ctypes
_VP, _I64, _INT, _F = c.c_void_p, c.c_int64, c.c_int, c.c_float
SIGNATURES = {
    "fp4_init": (_INT, [_INT]),
    "fp4_status_string": (c.c_char_p, [_INT]),
    "fp4_check_device_error": (_INT, [_VP]),
    "fp4_padded_scale_dims": (None, [_I64, _I64, c.POINTER(_I64), c.POINTER(_I64)]),
    "fp4_amax_workspace_bytes": (c.c_size_t, [_I64]),
    "fp4_amax_global_scale": (_INT, [_VP, _I64, _VP, _VP, _VP, c.c_size_t, _VP]),
    "fp4_quantize": (_INT, [_VP, _I64, _I64, _INT, _INT, _INT, _VP, _VP, _VP, _INT, _VP]),
    "fp4_quantize_sr": (_INT, [_VP, _I64, _I64, _INT, _INT, _INT, _VP, c.c_uint64, c.c_uint64, _VP, _VP, _INT,
                               _VP]),
    "fp4_dequantize": (_INT, [_VP, _VP, _VP, _I64, _I64, _INT, _INT, _INT, _VP, _INT, _VP, _VP]),
    "qmv": (_INT, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _INT, _INT, _INT, _VP, _VP]),
    "qqmv": (_INT, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _INT, _VP, _VP]),
    "qqmm": (_INT, [_VP, _VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _INT, _VP, _VP]),
    "gather_rows": (_INT, [_VP, _I64, _VP, _I64, _I64, _VP, _VP]),
    "qmv_grouped": (_INT, [_VP, _VP, _INT, _INT, _INT, _VP, _VP, _VP]),
    "gather_qmm": (_INT, [_VP, _VP, _VP, _I64, _VP, _VP, _VP, _I64, _I64, _I64, _INT, _INT, _INT, _INT,
                          _VP, _VP]),
    "qqmm_batched": (_INT, [_VP, _VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64,
                            _INT, _VP, _VP]),
    "qqmm_quantize_x_workspace_bytes": (c.c_size_t, [_I64, _I64, _INT]),
    "qqmm_quantize_x": (_INT, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _INT, _VP, c.c_size_t, _VP, _VP, _VP]),
    "qmm": (_INT, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _INT, _INT, _INT, _VP, _VP]),
    "fp4_debug_inject_wait_timeout": (_INT, [_INT]),
    "fp4_debug_stream_weights": (_INT, [_VP, _VP, _I64, _I64, _VP]),
    "kv_plan": (_INT, [_VP, _VP, _I64, _INT, _VP, _I64, _VP, _I64, _I64, _VP, _VP, _VP, _VP, _I64, _VP, _VP]),
    "kv_append": (_INT, [_VP, _VP, _I64, _I64, _VP, _I64, _I64, _VP, _I64, _VP]),
    "kv_attention_workspace_bytes": (c.c_size_t, [_I64, _I64, _I64, _I64, _I64]),
    "kv_attention": (_INT, [_VP, _VP, _I64, _I64, _I64, _I64, _VP, _VP, _I64, _VP, _I64, _I64, _I64, _F, _I64, _VP,
                            c.c_size_t, _VP, _VP, _VP]),
    "fp4_amax_global_scale_noalloc": (_INT, [_VP, _I64, _VP, _VP, _VP]),
}


class Fp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def lib():
    """Load libfp4gb300.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is not None:  # set once, below, when it is complete
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fp4_status_string(int(status)).decode()


def _check(st: int, where: str):
    if st != FP4_OK:
        raise Fp4Error(st, where)


def _p(t):
    return None if t is None else t.data_ptr()


def _s(stream):
    """The raw handle of `stream`, or of the current stream of the current device.  (Without the stream object of
    torch.cuda.current_stream(), which costs ~3 us a call: as much as a launch.)"""
    if stream is not None:
        return stream.cuda_stream
    if torch.cuda.is_initialized():
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return torch.cuda.current_stream().cuda_stream


def padded_scale_dims(rows: int, scale_cols: int):
    pr, pc = c.c_int64(), c.c_int64()
    lib().fp4_padded_scale_dims(rows, scale_cols, c.byref(pr), c.byref(pc))
    return pr.value, pc.value


def fp4_init(device: int = 0):
    _check(lib().fp4_init(device), "fp4_init")


def fp4_check_device_error(stream=None) -> int:
    """Returns the status (FP4_OK or FP4_ERR_TIMEOUT...) without raising."""
    return lib().fp4_check_device_error(_s(stream))


def fp4_amax_global_scale(x: torch.Tensor, gs_out=None, amax_out=None, ws=None, stream=None):
    n = x.numel()
    if gs_out is None:
        gs_out = torch.empty((), dtype=torch.float32, device=x.device)
    wsb = lib().fp4_amax_workspace_bytes(n)
    if ws is None:
        ws = torch.empty(wsb, dtype=torch.uint8, device=x.device)
    _check(lib().fp4_amax_global_scale(_p(x), n, _p(gs_out), _p(amax_out), _p(ws), ws.numel() * ws.element_size(),
                                       _s(stream)), "fp4_amax_global_scale")
    return gs_out


def fp4_amax_global_scale_noalloc(x: torch.Tensor, gs_out=None, amax_out=None, stream=None):
    """Allocation-free global scale: the library uses its own fixed device scratch."""
    if gs_out is None:
        gs_out = torch.empty((), dtype=torch.float32, device=x.device)
    _check(lib().fp4_amax_global_scale_noalloc(_p(x), x.numel(), _p(gs_out), _p(amax_out), _s(stream)),
           "fp4_amax_global_scale_noalloc")
    return gs_out


def scales_shape(rows: int, cols: int, group: int, layout: int):
    if layout == SCALES_TILED:
        return padded_scale_dims(rows, cols // group)
    return rows, cols // group


def fp4_quantize(x: torch.Tensor, mode: int, group_size: int = None, global_scale=None,
                 layout: int = SCALES_LINEAR, xq=None, scales=None, stream=None):
    group_size = group_size or GROUP[mode]
    rows, cols = x.shape
    if xq is None:
        xq = torch.empty((rows, cols // 8), dtype=torch.int32, device=x.device)
    if scales is None:
        scales = torch.empty(scales_shape(rows, cols, group_size, layout), dtype=torch.uint8, device=x.device)
    _check(lib().fp4_quantize(_p(x), rows, cols, mode, 4, group_size, _p(global_scale), _p(xq), _p(scales), layout,
                              _s(stream)), "fp4_quantize")
    return xq, scales


def fp4_quantize_sr(x: torch.Tensor, mode: int, seed: int, offset: int = 0, group_size: int = None,
                    global_scale=None, layout: int = SCALES_LINEAR, xq=None, scales=None, stream=None):
    """fp_quantize with stochastic rounding of the elements (Philox4x32-10 words
    from seed and offset); block scales as fp4_quantize."""
    group_size = group_size or GROUP[mode]
    rows, cols = x.shape
    if xq is None:
        xq = torch.empty((rows, cols // 8), dtype=torch.int32, device=x.device)
    if scales is None:
        scales = torch.empty(scales_shape(rows, cols, group_size, layout), dtype=torch.uint8, device=x.device)
    _check(lib().fp4_quantize_sr(_p(x), rows, cols, mode, 4, group_size, _p(global_scale), int(seed), int(offset),
                                 _p(xq), _p(scales), layout, _s(stream)), "fp4_quantize_sr")
    return xq, scales


def fp4_dequantize(wq: torch.Tensor, scales: torch.Tensor, biases=None, mode: int = MODE_NVFP4,
                   group_size: int = None, global_scale=None, layout: int = SCALES_LINEAR, out=None,
                   stream=None, rows: int = None):
    group_size = group_size or GROUP[mode]
    rows = rows if rows is not None else wq.shape[0]
    cols = wq.shape[-1] * 8
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.bfloat16, device=wq.device)
    _check(lib().fp4_dequantize(_p(wq), _p(scales), _p(biases), rows, cols, mode, 4, group_size,
                                _p(global_scale), layout, _p(out), _s(stream)), "fp4_dequantize")
    return out


def qmv(x: torch.Tensor, w: torch.Tensor, scales: torch.Tensor, biases=None, global_scale_w=None,
        mode: int = MODE_NVFP4, group_size: int = None, y=None, stream=None):
    group_size = group_size or GROUP[mode]
    N, K = w.shape[0], w.shape[1] * 8
    if y is None:
        y = torch.empty((N,), dtype=torch.bfloat16, device=w.device)
    _check(lib().qmv(_p(x), _p(w), _p(scales), _p(biases), _p(global_scale_w), N, K, mode, 4, group_size, _p(y),
                     _s(stream)), "qmv")
    return y


def qqmv(x: torch.Tensor, w: torch.Tensor, scales: torch.Tensor, global_scale_x=None, global_scale_w=None,
         mode: int = MODE_NVFP4, y=None, stream=None):
    """One-row quantized-activation GEMV: x is quantized and dequantized (bf16)
    inside the kernel, then multiplied by the 4-bit W."""
    N, K = w.shape[0], w.shape[1] * 8
    if y is None:
        y = torch.empty((N,), dtype=torch.bfloat16, device=w.device)
    _check(lib().qqmv(_p(x), _p(global_scale_x), _p(w), _p(scales), _p(global_scale_w), N, K, mode, _p(y),
                      _s(stream)), "qqmv")
    return y


def qqmm(xq: torch.Tensor, sx: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor, global_scale_x=None,
         global_scale_w=None, mode: int = MODE_NVFP4, out=None, stream=None, M: int = None):
    M = M if M is not None else xq.shape[0]
    N, K = wq.shape[0], wq.shape[1] * 8
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=wq.device)
    _check(lib().qqmm(_p(xq), _p(sx), _p(wq), _p(sw), _p(global_scale_x), _p(global_scale_w), M, N, K, mode,
                      _p(out), _s(stream)), "qqmm")
    return out


def qqmm_batched(xq: torch.Tensor, sx: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor, global_scale_x=None,
                 global_scale_w=None, mode: int = MODE_NVFP4, out=None, stream=None):
    """Batched FP4 x FP4 GEMM: xq [B, M, K/8] and its tiled scales [B, Mp, Cp];
    wq [B, N, K/8] (or [N, K/8], shared) and scales; out [B, M, N]; global
    scales as [B] arrays or None."""
    Bt, M, K = xq.shape[0], xq.shape[1], xq.shape[2] * 8
    shared = wq.dim() == 2
    N = wq.shape[-2]
    if out is None:
        out = torch.empty((Bt, M, N), dtype=torch.bfloat16, device=wq.device)
    _check(lib().qqmm_batched(_p(xq), _p(sx), _p(wq), _p(sw), _p(global_scale_x), _p(global_scale_w), Bt, M, N, K,
                              xq.stride(0), sx.stride(0), 0 if shared else wq.stride(0), 0 if shared else sw.stride(0),
                              out.stride(0), mode, _p(out), _s(stream)), "qqmm_batched")
    return out


def qqmm_quantize_x_workspace(M: int, K: int, mode: int = MODE_NVFP4, device="cuda"):
    """A zero-filled workspace for qqmm_quantize_x (allocate once, reuse)."""
    n = lib().qqmm_quantize_x_workspace_bytes(M, K, mode)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def qqmm_quantize_x(x: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor, ws: torch.Tensor, global_scale_x=None,
                    global_scale_w=None, mode: int = MODE_NVFP4, global_scale_x_out=None, out=None, stream=None):
    """Quantize bf16 x [M, K] and multiply by FP4 W in one launch."""
    M, K = x.shape
    N = wq.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=wq.device)
    _check(lib().qqmm_quantize_x(_p(x), _p(global_scale_x), _p(wq), _p(sw), _p(global_scale_w), M, N, K, mode,
                                 _p(ws), ws.numel(), _p(global_scale_x_out), _p(out), _s(stream)), "qqmm_quantize_x")
    return out


def gather_qmm(x: torch.Tensor, lhs_idx: torch.Tensor, rhs_idx: torch.Tensor, w: torch.Tensor,
               scales: torch.Tensor, biases=None, mode: int = MODE_MXFP4, group_size: int = None,
               sorted_indices: bool = True, out=None, stream=None):
    group_size = group_size or GROUP[mode]
    R = lhs_idx.numel()
    E, N, K = w.shape[0], w.shape[1], w.shape[2] * 8
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=w.device)
    _check(lib().gather_qmm(_p(x), _p(lhs_idx), _p(rhs_idx), R, _p(w), _p(scales), _p(biases), E, N, K, mode, 4,
                            group_size, 1 if sorted_indices else 0, _p(out), _s(stream)), "gather_qmm")
    return out


class MatrixGroup(c.Structure):
    """fp4_matrix_group: up to 4 matrices of one K for qmv_grouped."""
    _fields_ = [("count", c.c_int), ("w", c.c_void_p * 4), ("scales", c.c_void_p * 4), ("biases", c.c_void_p * 4),
                ("global_scale_w", c.c_void_p * 4), ("N", c.c_int64 * 4), ("K", c.c_int64)]


def matrix_group(mats) -> MatrixGroup:
    """mats: a list of (w, scales, biases, global_scale_w) tuples (None where absent)."""
    g = MatrixGroup()
    g.count = len(mats)
    for i, (w, s, b, gs) in enumerate(mats):
        g.w[i] = w.data_ptr()
        g.scales[i] = s.data_ptr()
        g.biases[i] = b.data_ptr() if b is not None else None
        g.global_scale_w[i] = gs.data_ptr() if gs is not None else None
        g.N[i] = w.shape[0]
    g.K = mats[0][0].shape[1] * 8
    return g


def qmv_grouped(x: torch.Tensor, mats, mode: int = MODE_NVFP4, group_size: int = None, ys=None, stream=None,
                prefetch_next=None):
    """One x against up to 4 matrices of the same K in one launch.  mats: a list of
    (w, scales, biases, global_scale_w) tuples; prefetch_next: the same for the
    GEMV launched next (an L2 warm-up hint) or None.  Returns the y vectors."""
    group_size = group_size or GROUP[mode]
    g = mats if isinstance(mats, MatrixGroup) else matrix_group(mats)
    if ys is None:
        ys = [torch.empty((int(g.N[i]),), dtype=torch.bfloat16, device=x.device) for i in range(g.count)]
    yy = (c.c_void_p * g.count)(*[y.data_ptr() for y in ys])
    nx = None
    if prefetch_next is not None:
        nx = prefetch_next if isinstance(prefetch_next, MatrixGroup) else matrix_group(prefetch_next)
    _check(lib().qmv_grouped(_p(x), c.byref(g), mode, 4, group_size, yy, c.byref(nx) if nx is not None else None,
                             _s(stream)), "qmv_grouped")
    return ys


def gather_rows(x: torch.Tensor, idx: torch.Tensor, out=None, stream=None):
    """out[i] = x[idx[i]] (bf16 rows; the routed activations in routing order)."""
    R, (T, K) = idx.numel(), x.shape
    if out is None:
        out = torch.empty((R, K), dtype=x.dtype, device=x.device)
    _check(lib().gather_rows(_p(x), T, _p(idx), R, K, _p(out), _s(stream)), "gather_rows")
    return out


def qmm(x: torch.Tensor, w: torch.Tensor, scales: torch.Tensor, biases=None, global_scale_w=None,
        mode: int = MODE_NVFP4, group_size: int = None, out=None, stream=None):
    """Dense W4A16 GEMM: out = x . deq(W)^T with x bf16 [M, K] and 4-bit W [N, K]."""
    group_size = group_size or GROUP[mode]
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=w.device)
    _check(lib().qmm(_p(x), _p(w), _p(scales), _p(biases), _p(global_scale_w), M, N, K, mode, 4, group_size, _p(out),
                     _s(stream)), "qmm")
    return out


def _need(name: str, t: torch.Tensor, dtype, shape, rows: bool = False):
    """Refuses a tensor whose type, shape or layout the kernels would misread: contiguous, or with `rows` its rows."""
    if t.dtype is not dtype or t.shape != shape or not (t.is_contiguous() or rows and t.stride(-1) == 1):
        raise ValueError(f"{name}: a {dtype} tensor of shape {tuple(shape)} with {'contiguous rows' if rows else 'contiguous elements'} "
                         f"is needed, got {t.dtype} {tuple(t.shape)}, strides {t.stride()}")


def _need_vector(name: str, t: torch.Tensor, dtype, n: int):
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: {n} contiguous {dtype} are needed, got {t.dtype} {tuple(t.shape)}, strides {t.stride()}")


def _need_gpu(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}: the kernels read GPU memory")


class KvCache(c.Structure):
    """fp4_kv_cache: one layer's paged 4-bit cache (make it with kv_cache, which keeps the tensors alive)."""
    _fields_ = [("k_codes", c.c_void_p), ("k_scales", c.c_void_p), ("v_codes", c.c_void_p), ("v_scales", c.c_void_p),
                ("global_scale_k", c.c_void_p), ("global_scale_v", c.c_void_p), ("num_pages", c.c_int64),
                ("page_size", c.c_int32), ("kv_heads", c.c_int32), ("head_dim", c.c_int32), ("mode", c.c_int)]


def kv_cache(k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
             mode: int = MODE_NVFP4, global_scale_k=None, global_scale_v=None) -> KvCache:
    """A cache over the caller's tensors: codes int32 [pages, kv_heads, page_size, head_dim/8], scales uint8
    [pages, kv_heads, page_size, head_dim/group], all contiguous."""
    pages, heads, page, words = k_codes.shape
    if v_codes.shape != k_codes.shape:
        raise ValueError(f"k and v codes differ in shape: {tuple(k_codes.shape)}, {tuple(v_codes.shape)}")
    want = (pages, heads, page, words * 8 // GROUP[mode])
    for name, t, shape, dt in (("k_codes", k_codes, tuple(k_codes.shape), torch.int32),
                               ("v_codes", v_codes, tuple(k_codes.shape), torch.int32),
                               ("k_scales", k_scales, want, torch.uint8), ("v_scales", v_scales, want, torch.uint8)):
        _need(name, t, dt, shape)
    for name, t in (("global_scale_k", global_scale_k), ("global_scale_v", global_scale_v)):
        if t is not None and (t.dtype is not torch.float32 or t.numel() != 1):
            raise ValueError(f"{name}: one float32 is needed, got {t.dtype} {tuple(t.shape)}")
    cache = KvCache(_p(k_codes), _p(k_scales), _p(v_codes), _p(v_scales), _p(global_scale_k), _p(global_scale_v),
                    pages, page, heads, words * 8, mode)
    cache.tensors = (k_codes, k_scales, v_codes, v_scales, global_scale_k, global_scale_v)
    return cache


def kv_cache_empty(num_pages: int, kv_heads: int, page_size: int, head_dim: int, mode: int = MODE_NVFP4,
                   global_scale_k=None, global_scale_v=None, device="cuda") -> KvCache:
    """A zero-filled cache of one layer."""
    codes = [torch.zeros((num_pages, kv_heads, page_size, head_dim // 8), dtype=torch.int32, device=device)
             for _ in range(2)]
    scales = [torch.zeros((num_pages, kv_heads, page_size, head_dim // GROUP[mode]), dtype=torch.uint8, device=device)
              for _ in range(2)]
    return kv_cache(codes[0], scales[0], codes[1], scales[1], mode, global_scale_k, global_scale_v)


class KvPlan(NamedTuple):
    """kv_plan's outputs (device tensors)."""
    total_lens: torch.Tensor   # int32 [batch]
    query_start: torch.Tensor  # int32 [batch + 1]
    slot_map: torch.Tensor     # int64 [tokens]
    positions: torch.Tensor    # int32 [tokens]
    pages_taken: torch.Tensor  # int32 scalar


def kv_plan(cached_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor, block_table: torch.Tensor,
            page_size: int, tokens: int, plan: KvPlan = None, stream=None) -> KvPlan:
    """Places a step's tokens: completes block_table [batch, max_pages] in place from free_pages and returns the
    lengths, slots and positions of up to `tokens` tokens (entries past the step's own are -1)."""
    batch, i32 = cached_lens.numel(), torch.int32
    if not (plan is None and cached_lens.dtype is i32 and cached_lens.is_cuda and cached_lens.is_contiguous() and new_lens.dtype is i32 and new_lens.is_cuda
            and new_lens.is_contiguous() and new_lens.numel() == batch and free_pages.dtype is i32 and free_pages.is_cuda
            and free_pages.is_contiguous() and block_table.dtype is i32 and block_table.is_cuda and block_table.dim() == 2
            and block_table.shape[0] == batch and block_table.stride(1) == 1):
        _need_vector("cached_lens", cached_lens, i32, batch)
        _need_vector("new_lens", new_lens, i32, batch)
        _need_vector("free_pages", free_pages, i32, free_pages.numel())
        _need("block_table", block_table, i32, (batch, *block_table.shape[-1:]), rows=True)
        if plan is not None:
            for name, t, dt, n in zip(plan._fields, plan, (i32, i32, torch.int64, i32, i32), (batch, batch + 1, tokens, tokens, 1)):
                _need_vector(name, t, dt, n)
        _need_gpu(cached_lens, new_lens, free_pages, block_table, *(plan or ()))
    if plan is None:
        dev = cached_lens.device
        plan = KvPlan(torch.empty(batch, dtype=i32, device=dev), torch.empty(batch + 1, dtype=i32, device=dev),
                      torch.empty(tokens, dtype=torch.int64, device=dev), torch.empty(tokens, dtype=i32, device=dev),
                      torch.empty((), dtype=i32, device=dev))
    _check(lib().kv_plan(_p(cached_lens), _p(new_lens), batch, page_size, _p(free_pages), free_pages.numel(),
                         _p(block_table), block_table.stride(0), block_table.shape[1], _p(plan.total_lens),
                         _p(plan.query_start), _p(plan.slot_map), _p(plan.positions), tokens,
                         _p(plan.pages_taken), _s(stream)), "kv_plan")
    return plan


def kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, stream=None):
    """Quantizes k and v [tokens, kv_heads, head_dim] (views with strides are read in place) into their slots."""
    tokens = slot_map.numel()
    bf16, shape, ks, vs = torch.bfloat16, (tokens, cache.kv_heads, cache.head_dim), k.stride(), v.stride()
    if not (slot_map.dtype is torch.int64 and slot_map.is_cuda and slot_map.is_contiguous() and k.dtype is bf16 and k.is_cuda
            and k.shape == shape and ks[2] == 1 and v.dtype is bf16 and v.is_cuda and v.shape == shape and vs[2] == 1
            and cache.tensors[0].is_cuda):
        _need_vector("slot_map", slot_map, torch.int64, tokens)
        for name, t in (("k", k), ("v", v)):
            _need(name, t, bf16, shape, rows=True)
        _need_gpu(k, v, slot_map, cache.tensors[0])
    _check(lib().kv_append(c.byref(cache), k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], slot_map.data_ptr(), tokens,
                           _s(stream)), "kv_append")


def kv_attention_workspace(cache: KvCache, batch: int, q_heads: int, max_query_len: int = 1, device="cuda"):
    """A zero-filled workspace for kv_attention: allocate once, with the longest max_query_len, for calls of any batch and
    any max_query_len up to it."""
    n = lib().kv_attention_workspace_bytes(batch, q_heads, cache.kv_heads, cache.head_dim, max_query_len)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kv_attention(cache: KvCache, q: torch.Tensor, query_start: torch.Tensor, total_lens: torch.Tensor,
                 block_table: torch.Tensor, ws: torch.Tensor, max_query_len: int = 1, scale: float = None,
                 window: int = 0, out=None, lse=None, stream=None):
    """Causal attention of q [tokens, q_heads, head_dim] over the paged 4-bit cache; scale defaults to
    head_dim ** -0.5."""
    tokens, heads, dim = q.shape
    batch, i32 = total_lens.numel(), torch.int32
    bf16, qs, pages = torch.bfloat16, q.stride(), block_table.shape
    if not (q.dtype is bf16 and q.is_cuda and dim == cache.head_dim and qs[2] == 1 and total_lens.dtype is i32 and total_lens.is_cuda
            and total_lens.is_contiguous() and query_start.dtype is i32 and query_start.is_cuda and query_start.is_contiguous()
            and query_start.numel() == batch + 1 and block_table.dtype is i32 and block_table.is_cuda and len(pages) == 2
            and pages[0] == batch and block_table.stride(1) == 1 and ws.is_cuda and ws.is_contiguous() and out is None and lse is None
            and cache.tensors[0].is_cuda):
        _need("q", q, bf16, (tokens, heads, cache.head_dim), rows=True)
        _need_vector("total_lens", total_lens, i32, batch)
        _need_vector("query_start", query_start, i32, batch + 1)
        _need("block_table", block_table, i32, (batch, *pages[-1:]), rows=True)
        if out is not None:
            _need("out", out, bf16, (tokens, heads, dim))
        if lse is not None:
            _need("lse", lse, torch.float32, (tokens, heads))
        if not ws.is_contiguous():
            raise ValueError(f"ws: a contiguous tensor is needed, got strides {ws.stride()}")
        _need_gpu(q, total_lens, query_start, block_table, ws, out, lse, cache.tensors[0])
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=q.device)
    _check(lib().kv_attention(c.byref(cache), q.data_ptr(), qs[0], qs[1], tokens, heads, query_start.data_ptr(),
                              total_lens.data_ptr(), batch, block_table.data_ptr(), block_table.stride(0), pages[1], max_query_len,
                              dim ** -0.5 if scale is None else scale, window, ws.data_ptr(), ws.numel() * ws.element_size(),
                              out.data_ptr(), _p(lse), _s(stream)), "kv_attention")
    return out


def fp4_debug_stream_weights(wq: torch.Tensor, scales: torch.Tensor, stream=None):
    """Stream NVFP4 weights as qmv's tensor-core path does, computing nothing
    (the launch-and-stream ceiling of that kernel shape)."""
    N, K = wq.shape[0], wq.shape[1] * 8
    _check(lib().fp4_debug_stream_weights(_p(wq), _p(scales), N, K, _s(stream)), "fp4_debug_stream_weights")


def fp4_debug_inject_wait_timeout(enable: bool):
    _check(lib().fp4_debug_inject_wait_timeout(1 if enable else 0), "fp4_debug_inject_wait_timeout")
