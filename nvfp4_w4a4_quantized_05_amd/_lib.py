"""ctypes binding of ``libnvfp4.so``: argument marshalling only.

Names mirror the C ABI in ``include/nvfp4.h``.  torch supplies device memory
and the current stream; every step of the computation runs in the HIP
library.  There is no fallback: if the library is missing, or a tensor is not
on a GPU, the call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")

NVFP4_OK = 0
IN_F32, IN_BF16 = 0, 1
OUT_F32, OUT_BF16 = 0, 1
SCALE_GIVEN, SCALE_FROM_AMAX = 0, 1
KV_FORMATS = {"fp8": 0, "nvfp4": 1}  # NVFP4_KV_E4M3, NVFP4_KV_NVFP4
STATUS_NAMES = {0: "NVFP4_OK", 1: "NVFP4_ERR_NULL", 2: "NVFP4_ERR_SHAPE", 3: "NVFP4_ERR_DTYPE",
                4: "NVFP4_ERR_MODE", 5: "NVFP4_ERR_ALIGN", 6: "NVFP4_ERR_WORKSPACE",
                7: "NVFP4_ERR_HIP", 8: "NVFP4_ERR_ALIAS", 9: "NVFP4_ERR_TOO_LARGE"}
EXPORTS = ("nvfp4_quantize", "nvfp4_gemm", "nvfp4_gemm_segmented", "nvfp4_gemm_segmented_gates",
           "nvfp4_quantize_gemm", "nvfp4_gdn_recurrence", "nvfp4_gemm_swiglu_quantize",
           "nvfp4_quantize_gemm_workspace_size", "nvfp4_quantize_gemm_no_alloc",
           "nvfp4_quantize_gemm_no_alloc_max_bytes", "nvfp4_harmonize_fused_scales",
           "nvfp4_gdn_prefill", "nvfp4_gdn_prefill_workspace_size", "nvfp4_gdn_decode", "nvfp4_conv_silu",
           "nvfp4_add_rmsnorm", "nvfp4_rmsnorm_gated", "nvfp4_qk_norm_rope", "nvfp4_kv_cache_write",
           "nvfp4_kv_cache_read", "nvfp4_attn_cached", "nvfp4_attn_cached_workspace_size",
           "nvfp4_gemm_workspace_size", "nvfp4_status_string", "nvfp4_last_hip_error")

_lib = None


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = load().nvfp4_status_string(status).decode()
        if status == 7:
            msg += f" (hipError {load().nvfp4_last_hip_error()})"
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}: {msg}")


def load() -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m nvfp4_w4a4_quantized_05_amd.build` (needs hipcc)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.nvfp4_quantize.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, i32, vp]
    lib.nvfp4_quantize.restype = i32
    lib.nvfp4_gemm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, i32, i64, vp, sz, vp]
    lib.nvfp4_gemm.restype = i32
    lib.nvfp4_gemm_segmented.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.POINTER(i64), i32, i64, i64, vp, i32,
                                         i64, vp, sz, vp]
    lib.nvfp4_gemm_segmented.restype = i32
    lib.nvfp4_gemm_segmented_gates.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.POINTER(i64), i32, i32, vp, vp, i32,
                                               i64, i64, vp, i32, i64, vp, sz, vp]
    lib.nvfp4_gemm_segmented_gates.restype = i32
    lib.nvfp4_gemm_swiglu_quantize.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, i64, vp]
    lib.nvfp4_gemm_swiglu_quantize.restype = i32
    lib.nvfp4_gdn_recurrence.argtypes = [vp, i64, i64, i64, i64, i64, i64, i64, i32, i32, vp, vp, vp, i64, vp, vp,
                                         i32, vp, vp]
    lib.nvfp4_gdn_recurrence.restype = i32
    lib.nvfp4_quantize_gemm.argtypes = [vp, i32, i64, vp, vp, vp, vp, i64, i64, i64, vp, i32, i64, vp, sz, vp]
    lib.nvfp4_quantize_gemm.restype = i32
    lib.nvfp4_quantize_gemm_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    lib.nvfp4_quantize_gemm_workspace_size.restype = sz
    lib.nvfp4_quantize_gemm_no_alloc.argtypes = [vp, i32, i64, vp, vp, vp, vp, i64, i64, i64, vp, i32, i64, vp]
    lib.nvfp4_quantize_gemm_no_alloc.restype = i32
    lib.nvfp4_quantize_gemm_no_alloc_max_bytes.argtypes = []
    lib.nvfp4_quantize_gemm_no_alloc_max_bytes.restype = sz
    f32 = ctypes.c_float
    lib.nvfp4_gdn_prefill.argtypes = [vp, i64, i64, i64, i64, vp, i32, i64, i64, i64, vp, i32, i64, i32, i32, vp, vp,
                                      vp, i32, vp, i64, vp, sz, vp]
    lib.nvfp4_gdn_prefill.restype = i32
    lib.nvfp4_gdn_prefill_workspace_size.argtypes = [i64, i32, i32, i32]
    lib.nvfp4_gdn_prefill_workspace_size.restype = sz
    lib.nvfp4_gdn_decode.argtypes = [vp, i32, i64, i64, i64, i64, vp, i32, i64, i64, i64, i64, i32, i32, vp, vp, i32,
                                     vp, i32, i64, vp]
    lib.nvfp4_gdn_decode.restype = i32
    lib.nvfp4_conv_silu.argtypes = [vp, i32, i64, i64, vp, i32, vp, i32, i64, vp, vp, i32, vp, i64, vp]
    lib.nvfp4_conv_silu.restype = i32
    lib.nvfp4_add_rmsnorm.argtypes = [vp, i32, i64, vp, i32, i64, f32, vp, f32, i64, i64, vp, i64, vp, i32, i64, vp,
                                      vp, vp, vp]
    lib.nvfp4_add_rmsnorm.restype = i32
    lib.nvfp4_rmsnorm_gated.argtypes = [vp, i32, i64, vp, i32, i64, vp, f32, i64, i64, i32, vp, i32, i64, vp, vp, vp,
                                        vp]
    lib.nvfp4_rmsnorm_gated.restype = i32
    lib.nvfp4_qk_norm_rope.argtypes = [vp, i32, i64, i64, i64, i64, i32, i32, i32, vp, vp, f32, vp, i32, i32, vp, i32,
                                       ctypes.c_char_p, i32, vp, i64, vp, i64, vp]
    lib.nvfp4_qk_norm_rope.restype = i32
    for f in (lib.nvfp4_kv_cache_write, lib.nvfp4_kv_cache_read):
        f.argtypes = [vp, vp, i64, i32, vp, vp, i32, i64, vp, i64, vp, i64, i32, vp]
        f.restype = i32
    lib.nvfp4_attn_cached.argtypes = [vp, vp, i64, i32, vp, vp, i32, i64, vp, i64, i32, f32, vp, vp, i64, vp, sz, vp]
    lib.nvfp4_attn_cached.restype = i32
    lib.nvfp4_attn_cached_workspace_size.argtypes = [i64, i32, i32, i32, i32]
    lib.nvfp4_attn_cached_workspace_size.restype = sz
    lib.nvfp4_harmonize_fused_scales.argtypes = [vp, vp, ctypes.POINTER(i64), i32, i64, vp, vp, vp]
    lib.nvfp4_harmonize_fused_scales.restype = i32
    lib.nvfp4_gemm_workspace_size.argtypes = [i64, i64, i64, i32]
    lib.nvfp4_gemm_workspace_size.restype = sz
    lib.nvfp4_status_string.argtypes = [i32]
    lib.nvfp4_status_string.restype = ctypes.c_char_p
    lib.nvfp4_last_hip_error.argtypes = []
    lib.nvfp4_last_hip_error.restype = i32
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, what: str):
    if status != NVFP4_OK:
        raise Nvfp4Error(status, what)


def _need_gpu(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("nvfp4 calls take GPU tensors only")


def _u8_matrix(t, shape, what):
    """t must be a contiguous uint8 tensor of exactly `shape`."""
    if t.dtype != torch.uint8 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous uint8 {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _f32_scalars(t, n, what):
    """t must hold at least n contiguous float32 values (tensor scales)."""
    if t.dtype != torch.float32 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous float32 with {n} value(s)")


def _out_matrix(out, M, N, out_dtype):
    """out: 2-D, out_dtype, M rows, at least N columns, unit column stride."""
    if out.dtype != out_dtype or out.dim() != 2 or out.stride(1) != 1:
        raise ValueError("out must be 2-D with unit column stride and dtype out_dtype")
    if out.shape[0] != M or out.shape[1] < N:
        raise ValueError(f"out must be [{M}, >= {N}], got {tuple(out.shape)}")


def _operands(a_codes, a_scales, a_gs, w_codes, w_scales, k):
    """Shapes of the two NVFP4 operands; returns (M, N, K)."""
    M = a_codes.shape[0]
    N = w_codes.shape[0]
    K = a_codes.shape[1] * 2 if k is None else k
    if a_codes.dim() != 2 or w_codes.dim() != 2 or K <= 0 or K % 16:
        raise ValueError("codes must be 2-D and K a positive multiple of 16")
    _u8_matrix(a_codes, (M, K // 2), "a_codes")
    _u8_matrix(a_scales, (M, K // 16), "a_scales")
    _u8_matrix(w_codes, (N, K // 2), "w_codes")
    _u8_matrix(w_scales, (N, K // 16), "w_scales")
    _f32_scalars(a_gs, 1, "a_gs")
    return M, N, K


def quantize(x: torch.Tensor, global_scale: torch.Tensor | None = None, *, from_amax: bool | None = None,
             codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """NVFP4-encode a 2-D bf16 or fp32 GPU tensor (rows contiguous, any row stride).

    ``global_scale`` is a one-element fp32 GPU tensor: read when it is given
    (calibrated scale), written with RN32(amax/2688) when ``from_amax``
    (default: from_amax = global_scale is None).  Returns (codes, scales, gs).
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    if x.dtype == torch.bfloat16:
        dt = IN_BF16
    elif x.dtype == torch.float32:
        dt = IN_F32
    else:
        raise ValueError(f"unsupported input dtype {x.dtype}")
    rows, cols = x.shape
    if cols % 16:
        raise ValueError("columns must be a multiple of 16")
    if codes is not None:
        _u8_matrix(codes, (rows, cols // 2), "codes")
    if scales is not None:
        _u8_matrix(scales, (rows, cols // 16), "scales")
    if global_scale is not None:
        _f32_scalars(global_scale, 1, "global_scale")
    _need_gpu(x, global_scale, codes, scales)
    if from_amax is None:
        from_amax = global_scale is None
    if global_scale is None:
        global_scale = torch.empty(1, dtype=torch.float32, device=x.device)
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=x.device)
    st = load().nvfp4_quantize(_ptr(x), dt, rows, cols, x.stride(0), _ptr(codes), _ptr(scales),
                               _ptr(global_scale), SCALE_FROM_AMAX if from_amax else SCALE_GIVEN,
                               _stream(stream))
    _check(st, "nvfp4_quantize")
    return codes, scales, global_scale


def gemm(a_codes, a_scales, a_gs, w_codes, w_scales, w_gs, *, out_dtype=torch.float32,
         out: torch.Tensor | None = None, k: int | None = None, stream=None):
    """y[M, N] = RN32(g_a g_w) deq(A) deq(W)^T from NVFP4 A [M, K] and W [N, K]."""
    M, N, K = _operands(a_codes, a_scales, a_gs, w_codes, w_scales, k)
    _f32_scalars(w_gs, 1, "w_gs")
    od = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}[out_dtype]
    if out is not None:
        _out_matrix(out, M, N, out_dtype)
    _need_gpu(a_codes, a_scales, a_gs, w_codes, w_scales, w_gs, out)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    lib = load()
    ws_bytes = lib.nvfp4_gemm_workspace_size(M, N, K, od)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=a_codes.device) if ws_bytes else None
    st = lib.nvfp4_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(a_gs), _ptr(w_codes), _ptr(w_scales),
                        _ptr(w_gs), M, N, K, _ptr(out), od, out.stride(0), _ptr(ws), ws_bytes,
                        _stream(stream))
    _check(st, "nvfp4_gemm")
    return out


def gemm_segmented(a_codes, a_scales, a_gs, w_codes, w_scales, module_gs, module_rows, *,
                   out_dtype=torch.float32, out: torch.Tensor | None = None, k: int | None = None, stream=None):
    """One GEMM over modules concatenated along N (module_rows rows each): the
    columns of module i are RN32(g_a g_i) deq(A) deq(W_i)^T, g_i = module_gs[i]."""
    rows = [int(r) for r in module_rows]
    M, N, K = _operands(a_codes, a_scales, a_gs, w_codes, w_scales, k)
    if sum(rows) != N or module_gs.numel() != len(rows) or module_gs.dtype != torch.float32:
        raise ValueError("module_rows must sum to the weight rows, one float32 scale per module")
    od = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}[out_dtype]
    if out is not None:
        _out_matrix(out, M, N, out_dtype)
    _need_gpu(a_codes, a_scales, a_gs, w_codes, w_scales, module_gs, out)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    lib = load()
    ws_bytes = lib.nvfp4_gemm_workspace_size(M, N, K, od)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=a_codes.device) if ws_bytes else None
    host_rows = (ctypes.c_int64 * len(rows))(*rows)
    st = lib.nvfp4_gemm_segmented(_ptr(a_codes), _ptr(a_scales), _ptr(a_gs), _ptr(w_codes), _ptr(w_scales),
                                  _ptr(module_gs.contiguous()), host_rows, len(rows), M, K, _ptr(out), od,
                                  out.stride(0), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "nvfp4_gemm_segmented")
    return out


def gemm_segmented_gates(a_codes, a_scales, a_gs, w_codes, w_scales, module_gs, module_rows, *,
                         decay_module: int = -1, a_log: torch.Tensor | None = None,
                         dt_bias: torch.Tensor | None = None, write_module: int = -1,
                         out_dtype=torch.float32, out: torch.Tensor | None = None, stream=None):
    """gemm_segmented whose epilogue turns module `decay_module` into the decay
    gate -exp(a_log) softplus(v + dt_bias) and module `write_module` into
    sigmoid(v) (-1: none)."""
    rows = [int(r) for r in module_rows]
    M, N, K = _operands(a_codes, a_scales, a_gs, w_codes, w_scales, None)
    if sum(rows) != N or module_gs.numel() != len(rows) or module_gs.dtype != torch.float32:
        raise ValueError("module_rows must sum to the weight rows, one float32 scale per module")
    if decay_module >= 0:
        for t in (a_log, dt_bias):
            if t is None or t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != rows[decay_module]:
                raise ValueError("a_log and dt_bias: contiguous float32, one per decay-module row")
    od = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}[out_dtype]
    if out is not None:
        _out_matrix(out, M, N, out_dtype)
    _need_gpu(a_codes, a_scales, a_gs, w_codes, w_scales, module_gs, a_log, dt_bias, out)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a_codes.device)
    lib = load()
    ws_bytes = lib.nvfp4_gemm_workspace_size(M, N, K, od)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=a_codes.device) if ws_bytes else None
    host_rows = (ctypes.c_int64 * len(rows))(*rows)
    st = lib.nvfp4_gemm_segmented_gates(_ptr(a_codes), _ptr(a_scales), _ptr(a_gs), _ptr(w_codes), _ptr(w_scales),
                                        _ptr(module_gs.contiguous()), host_rows, len(rows), decay_module,
                                        _ptr(a_log), _ptr(dt_bias), write_module, M, K, _ptr(out), od,
                                        out.stride(0), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "nvfp4_gemm_segmented_gates")
    return out


def gemm_swiglu_quantize(a_codes, a_scales, a_gs, w_codes, w_scales, w_gs, h_gs, *, codes=None, scales=None,
                         h: torch.Tensor | None = None, stream=None):
    """h = silu(gate) * up of the gate/up GEMM (W = [gate; up], 2F rows),
    quantized with tensor scale h_gs in the epilogue.  Returns (codes
    [M, F/2], scales [M, F/16], h_gs); h [M, >= F] fp32 is filled if given."""
    M, N, K = _operands(a_codes, a_scales, a_gs, w_codes, w_scales, None)
    if N % 2:
        raise ValueError("the gate/up weight has 2F rows")
    F = N // 2
    _f32_scalars(w_gs, 1, "w_gs")
    _f32_scalars(h_gs, 1, "h_gs")
    _need_gpu(a_codes, a_scales, a_gs, w_codes, w_scales, w_gs, h_gs, codes, scales, h)
    if codes is None:
        codes = torch.empty((M, F // 2), dtype=torch.uint8, device=a_codes.device)
    if scales is None:
        scales = torch.empty((M, F // 16), dtype=torch.uint8, device=a_codes.device)
    if codes.shape != (M, F // 2) or scales.shape != (M, F // 16) or not codes.is_contiguous() \
            or not scales.is_contiguous():
        raise ValueError("codes [M, F/2] and scales [M, F/16], contiguous")
    if h is not None and (h.dtype != torch.float32 or h.dim() != 2 or h.shape[0] != M or h.stride(1) != 1):
        raise ValueError("h must be float32 [M, >= F] with unit column stride")
    st = load().nvfp4_gemm_swiglu_quantize(_ptr(a_codes), _ptr(a_scales), _ptr(a_gs), _ptr(w_codes),
                                           _ptr(w_scales), _ptr(w_gs), M, F, K, _ptr(h_gs), _ptr(codes),
                                           _ptr(scales), _ptr(h), h.stride(0) if h is not None else 0,
                                           _stream(stream))
    _check(st, "nvfp4_gemm_swiglu_quantize")
    return codes, scales, h_gs


def gdn_recurrence(x: torch.Tensor, *, q_col: int, k_col: int, v_col: int, g_col: int, beta_col: int,
                   n_qk_heads: int, n_v_heads: int, state_in: torch.Tensor | None = None,
                   state_out: torch.Tensor | None = None, o: torch.Tensor | None = None,
                   state_norms: torch.Tensor | None = None, snap_steps: torch.Tensor | None = None,
                   snaps: torch.Tensor | None = None, stream=None):
    """Gated DeltaNet recurrence over the T rows of x (fp32 [T, ldx]: q, k,
    v, g, beta at the given columns; v_col = -1 reads v as zero).  Writes
    whichever of state_out [Hv,128,128], o [T, >= Hv*128], state_norms
    [T, Hv] and snaps [n, Hv, 128, 128] (at int32 snap_steps) are given."""
    _need_gpu(x, state_in, state_out, o, state_norms, snap_steps, snaps)
    if x.dim() != 2 or x.dtype != torch.float32 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D float32 tensor with unit column stride")
    T = x.shape[0]
    st_shape = (n_v_heads, 128, 128)
    for t in (state_in, state_out):
        if t is not None and (t.shape != st_shape or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError("states must be contiguous float32 [n_v_heads, 128, 128]")
    if o is not None and (o.dtype != torch.float32 or o.dim() != 2 or o.shape[0] != T or o.stride(1) != 1):
        raise ValueError("o must be float32 [T, >= n_v_heads*128] with unit column stride")
    if state_norms is not None and (state_norms.shape != (T, n_v_heads) or state_norms.dtype != torch.float32
                                    or not state_norms.is_contiguous()):
        raise ValueError("state_norms must be contiguous float32 [T, n_v_heads]")
    n_snaps = 0
    if snap_steps is not None:
        n_snaps = snap_steps.numel()
        if snap_steps.dtype != torch.int32 or snaps is None or snaps.shape != (n_snaps, *st_shape) \
                or snaps.dtype != torch.float32 or not snaps.is_contiguous():
            raise ValueError("snap_steps int32 [n] with snaps float32 [n, n_v_heads, 128, 128]")
    st = load().nvfp4_gdn_recurrence(_ptr(x), x.stride(0), q_col, k_col, v_col, g_col, beta_col, T, n_qk_heads,
                                     n_v_heads, _ptr(state_in), _ptr(state_out), _ptr(o),
                                     o.stride(0) if o is not None else 0, _ptr(state_norms),
                                     _ptr(snap_steps), n_snaps, _ptr(snaps), _stream(stream))
    _check(st, "nvfp4_gdn_recurrence")
    return state_out


_DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1}  # NVFP4_IN_* and NVFP4_OUT_*

# The calls of a decode step take 2-5 us on the GPU, so what these do per call
# is kept short: one look at each tensor, addresses passed as plain integers.


def _new(shape, dtype, device, stream):
    """Memory that a call on `stream` makes itself, from that stream's pool: the
    current stream's may still be in use there, and what is freed when the
    call returns would be handed out to it while the kernels run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t, what):
    """(address, dtype code, rows, columns, row stride) of a 2-D bf16 or fp32
    GPU tensor with unit column stride.  One row or fewer has no stride, only a
    width: the next multiple of 8 that holds it (16 bytes), since a stride that
    no address is made of must not be refused."""
    code = _DTYPE_CODE.get(t.dtype)
    if code is None or t.dim() != 2:
        raise ValueError(f"{what} must be 2-D bf16 or fp32, got {t.dtype} {tuple(t.shape)}")
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{what} must have unit column stride")
    if not t.is_cuda:
        raise ValueError("nvfp4 calls take GPU tensors only")
    return t.data_ptr(), code, rows, cols, ld if rows > 1 else max(-(-cols // 8) * 8, 8)


def _vector(t, dtype, n, what):
    """Address of a contiguous GPU vector of n values."""
    if t.dtype != dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} vector of {n} values, got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError("nvfp4 calls take GPU tensors only")
    return t.data_ptr()


def _seqlens(t):
    """(address, sequences) of cu_seqlens."""
    n = t.shape[0] - 1 if t.dim() == 1 else 0
    if n < 1:
        raise ValueError("cu_seqlens must be a vector of n_seqs + 1 >= 2 row numbers")
    return _vector(t, torch.int32, n + 1, "cu_seqlens"), n


def _pool(t, dtype, shape, what):
    """(address, slots) of a contiguous [n_slots, *shape] state pool."""
    if t.dtype != dtype or t.shape[1:] != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} [n_slots, {', '.join(map(str, shape))}]")
    if not t.is_cuda:
        raise ValueError("nvfp4 calls take GPU tensors only")
    return t.data_ptr(), t.shape[0]


def _out_rows(t, rows, cols, what):
    """_rows of an output of `rows` rows and at least `cols` columns: (address, dtype code, row stride)."""
    ptr, code, r, c, ld = _rows(t, what)
    if r != rows or c < cols:
        raise ValueError(f"{what} must be [{rows}, >= {cols}], got {tuple(t.shape)}")
    return ptr, code, ld


def _raw_stream(stream):
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else stream.cuda_stream


def gdn_prefill(x: torch.Tensor, gates: torch.Tensor, cu_seqlens: torch.Tensor, *, q_col: int, k_col: int,
                v_col: int, g_col: int, beta_col: int, n_qk_heads: int, n_v_heads: int,
                state_in: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
                slots: torch.Tensor | None = None, o: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """Gated DeltaNet recurrence over packed prompts: sequence i is rows
    cu_seqlens[i] .. cu_seqlens[i + 1] - 1 (device int32) of x (bf16: q, k, v
    at their columns) and of gates (bf16 or fp32: g and beta at theirs).  It
    starts from slot slots[i] of state_in [n_slots, n_v_heads, 128, 128]
    (zeros if None) and leaves its state in that slot of state_out (which may
    be state_in).  Returns o, bf16 [T, >= n_v_heads * 128]; rows of no
    sequence are not written."""
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    xp, _, T, _, ldx = _rows(x, "x")
    gp, gates_dtype, g_rows, _, ldg = _rows(gates, "gates")
    if g_rows != T:
        raise ValueError("x and gates must have the same rows")
    cp, n_seqs = _seqlens(cu_seqlens)
    ip = op = sp = None
    n_slots = n_seqs
    if state_in is not None:
        ip, n_slots = _pool(state_in, torch.float32, (n_v_heads, 128, 128), "state_in")
    if state_out is state_in:
        op = ip
    elif state_out is not None:
        op, n_out = _pool(state_out, torch.float32, (n_v_heads, 128, 128), "state_out")
        if ip is not None and n_out != n_slots:
            raise ValueError("state_in and state_out must have the same slots")
        n_slots = n_out
    if slots is not None:
        if ip is None and op is None:
            raise ValueError("slots without a state pool")
        sp = _vector(slots, torch.int32, n_seqs, "slots")
    if o is None:
        o = _new((T, n_v_heads * 128), torch.bfloat16, x.device, stream)
    o_ptr, o_dtype, ldo = _out_rows(o, T, n_v_heads * 128, "o")
    if o_dtype != OUT_BF16:
        raise ValueError("o must be bf16")
    lib = load()
    need = lib.nvfp4_gdn_prefill_workspace_size(T, n_seqs, n_qk_heads, n_v_heads)
    if workspace is None:
        workspace = _new(need, torch.uint8, x.device, stream)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    st = lib.nvfp4_gdn_prefill(xp, ldx, q_col, k_col, v_col, gp, gates_dtype, ldg, g_col, beta_col, cp, n_seqs, T,
                               n_qk_heads, n_v_heads, ip, op, sp, n_slots, o_ptr, ldo, workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _raw_stream(stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_gdn_prefill")
    return o


def gdn_decode(x: torch.Tensor, gates: torch.Tensor, states: torch.Tensor, *, q_col: int, k_col: int, v_col: int,
               g_col: int, beta_col: int, n_qk_heads: int, n_v_heads: int, slots: torch.Tensor | None = None,
               o: torch.Tensor | None = None, stream=None):
    """The same recurrence for one new token of each request: row b of x and
    gates (bf16 or fp32) is request b's, slot slots[b] (b if None) of states
    [n_slots, n_v_heads, 128, 128] fp32 is updated in place.  Returns o
    [batch, >= n_v_heads * 128] (bf16 or fp32 as given, else x's type);
    requests whose slot is negative get a row of zeros."""
    xp, x_dtype, B, _, ldx = _rows(x, "x")
    gp, gates_dtype, g_rows, _, ldg = _rows(gates, "gates")
    if g_rows != B:
        raise ValueError("x and gates must have the same rows")
    pp, n_slots = _pool(states, torch.float32, (n_v_heads, 128, 128), "states")
    sp = _vector(slots, torch.int32, B, "slots") if slots is not None else None
    if o is None:
        o = _new((B, n_v_heads * 128), x.dtype, x.device, stream)
    op, o_dtype, ldo = _out_rows(o, B, n_v_heads * 128, "o")
    st = load().nvfp4_gdn_decode(xp, x_dtype, ldx, q_col, k_col, v_col, gp, gates_dtype, ldg, g_col, beta_col, B,
                                 n_qk_heads, n_v_heads, pp, sp, n_slots, op, o_dtype, ldo, _raw_stream(stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_gdn_decode")
    return o


def conv_silu(x: torch.Tensor, weight: torch.Tensor, *, cu_seqlens: torch.Tensor | None = None,
              state: torch.Tensor | None = None, slots: torch.Tensor | None = None,
              out: torch.Tensor | None = None, stream=None):
    """silu of the causal convolution of each column of x [T, channels] (bf16
    or fp32) with weight [channels, width] fp32, per packed sequence of
    cu_seqlens (device int32), or, without cu_seqlens, for one new row of each
    request.  state [n_slots, width - 1, channels] (x's type) holds the last
    inputs of each request, read and updated in slot slots[i].  Returns out
    [T, >= channels] of x's type."""
    xp, dtype, T, channels, ldx = _rows(x, "x")
    if weight.dtype != torch.float32 or weight.dim() != 2 or weight.shape[0] != channels \
            or not weight.is_contiguous() or not weight.is_cuda:
        raise ValueError("weight must be contiguous float32 [channels, width] on the GPU")
    width = weight.shape[1]
    cp, n_seqs = _seqlens(cu_seqlens) if cu_seqlens is not None else (None, T)
    pp, n_slots = _pool(state, x.dtype, (width - 1, channels), "state") if state is not None else (None, 0)
    sp = None
    if slots is not None:
        if state is None:
            raise ValueError("slots without a state pool")
        sp = _vector(slots, torch.int32, n_seqs, "slots")
    if out is None:
        out = _new((T, channels), x.dtype, x.device, stream)
    yp, y_dtype, ldy = _out_rows(out, T, channels, "out")
    if y_dtype != dtype:
        raise ValueError("out must have the dtype of x")
    st = load().nvfp4_conv_silu(xp, dtype, ldx, channels, weight.data_ptr(), width, cp, n_seqs if cp else 0, T, pp, sp,
                                n_slots, yp, ldy, _raw_stream(stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_conv_silu")
    return out


def _norm_out(rows, cols, out, out_dtype, y_gs, codes, scales, device, stream):
    """Destinations of a norm's y, made where they are not given: (out, its
    address, dtype code and row stride, codes, scales)."""
    if y_gs is not None:
        _f32_scalars(y_gs, 1, "y_gs")
        if cols % 16:
            raise ValueError("columns must be a multiple of 16 to be quantized")
        if codes is None:
            codes = _new((rows, cols // 2), torch.uint8, device, stream)
        if scales is None:
            scales = _new((rows, cols // 16), torch.uint8, device, stream)
        _u8_matrix(codes, (rows, cols // 2), "codes")
        _u8_matrix(scales, (rows, cols // 16), "scales")
        _need_gpu(y_gs, codes, scales)
    elif codes is not None or scales is not None:
        raise ValueError("codes and scales need y_gs, the tensor scale")
    if out is None and (y_gs is None or out_dtype is not None):
        out = _new((rows, cols), out_dtype or torch.bfloat16, device, stream)
    if out is None:
        return None, None, 0, 0, codes, scales
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out must have dtype out_dtype")
    yp, y_dtype, ldy = _out_rows(out, rows, cols, "out")
    return out, yp, y_dtype, ldy, codes, scales


def add_rmsnorm(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor | None = None, scale: float = 1.0,
                eps: float = 1e-6, residual_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                out_dtype=None, y_gs: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                scales: torch.Tensor | None = None, stream=None):
    """t = residual + scale * x (written to residual_out if given, which may be
    residual) and y = RMSNorm(t) * weight (float32 [cols]).  y goes to out
    (bf16 or fp32; made in bf16 if neither out nor y_gs is given) and, with
    y_gs, as NVFP4 codes and scales under that tensor scale.  Returns out, or
    with y_gs (out or None, codes, scales)."""
    xp, x_dtype, rows, cols, ldx = _rows(x, "x")
    wp = _vector(weight, torch.float32, cols, "weight")
    rp = tp = None
    r_dtype, ldr, ldt = x_dtype, 0, 0
    if residual is not None:
        rp, r_dtype, r, c, ldr = _rows(residual, "residual")
        if r != rows or c != cols:
            raise ValueError("residual must have the shape of x")
    if residual_out is not None:
        tp, t_dtype, r, c, ldt = _rows(residual_out, "residual_out")
        if r != rows or c != cols or (rp is not None and t_dtype != r_dtype):
            raise ValueError("residual_out must have the shape of x and the dtype of residual")
        r_dtype = t_dtype
    out, yp, y_dtype, ldy, codes, scales = _norm_out(rows, cols, out, out_dtype, y_gs, codes, scales, x.device, stream)
    st = load().nvfp4_add_rmsnorm(xp, x_dtype, ldx, rp, r_dtype, ldr, scale, wp, eps, rows, cols, tp, ldt, yp,
                                  y_dtype, ldy, _ptr(y_gs), _ptr(codes), _ptr(scales), _raw_stream(stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_add_rmsnorm")
    return out if y_gs is None else (out, codes, scales)


def rmsnorm_gated(o: torch.Tensor, z: torch.Tensor, weight: torch.Tensor, *, eps: float = 1e-6,
                  out: torch.Tensor | None = None, out_dtype=None, y_gs: torch.Tensor | None = None,
                  codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """y = RMSNorm of each group of weight.numel() columns of o, times weight,
    times silu(z); destinations and return value as for add_rmsnorm."""
    op, o_dtype, rows, cols, ldo = _rows(o, "o")
    zp, z_dtype, z_rows, z_cols, ldz = _rows(z, "z")
    if z_rows != rows or z_cols != cols:
        raise ValueError("z must have the shape of o")
    group = weight.numel()
    wp = _vector(weight, torch.float32, group, "weight")
    out, yp, y_dtype, ldy, codes, scales = _norm_out(rows, cols, out, out_dtype, y_gs, codes, scales, o.device, stream)
    st = load().nvfp4_rmsnorm_gated(op, o_dtype, ldo, zp, z_dtype, ldz, wp, eps, rows, cols, group, yp, y_dtype, ldy,
                                    _ptr(y_gs), _ptr(codes), _ptr(scales), _raw_stream(stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_rmsnorm_gated")
    return out if y_gs is None else (out, codes, scales)


class _KvCacheStruct(ctypes.Structure):  # nvfp4_kv_cache_t
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales", "k_gs", "v_gs")] + \
               [(n, ctypes.c_int32) for n in ("format", "n_pages", "page_size", "n_kv_heads", "head_dim")]


class KvCache:
    """A paged, quantised key/value cache of one layer (nvfp4_kv_cache_t): the
    given uint8 tensors, which it keeps alive, and their tensor scales.

    format "fp8":    k [n_pages, n_kv_heads, page_size, head_dim],
                     v [n_pages, n_kv_heads, head_dim, page_size] (E4M3 codes)
    format "nvfp4":  k [.., page_size, head_dim / 2], k_scales [.., page_size, head_dim / 16],
                     v [.., head_dim / 2, page_size], v_scales [.., head_dim / 16, page_size]
    k_gs, v_gs:      one float32 each, on the GPU
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_gs: torch.Tensor, v_gs: torch.Tensor,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None, *, format: str):
        if format not in KV_FORMATS:
            raise ValueError(f"format must be one of {tuple(KV_FORMATS)}")
        if k.dim() != 4 or v.dim() != 4:
            raise ValueError("k and v must be 4-D")
        fp4 = format == "nvfp4"
        n_pages, heads, page, width = k.shape
        dim = 2 * width if fp4 else width
        _u8_matrix(k, (n_pages, heads, page, width), "k")
        _u8_matrix(v, (n_pages, heads, width, page), "v")
        if fp4 and (k_scales is None or v_scales is None):
            raise ValueError("an nvfp4 cache needs k_scales and v_scales")
        if not fp4 and (k_scales is not None or v_scales is not None):
            raise ValueError("an fp8 cache has no k_scales or v_scales")
        if fp4:
            _u8_matrix(k_scales, (n_pages, heads, page, dim // 16), "k_scales")
            _u8_matrix(v_scales, (n_pages, heads, dim // 16, page), "v_scales")
        _f32_scalars(k_gs, 1, "k_gs")
        _f32_scalars(v_gs, 1, "v_gs")
        self._tensors = [t for t in (k, v, k_scales, v_scales, k_gs, v_gs) if t is not None]
        _need_gpu(*self._tensors)
        self.device = _one_device(*self._tensors)
        self.k, self.v, self.k_scales, self.v_scales, self.k_gs, self.v_gs = k, v, k_scales, v_scales, k_gs, v_gs
        self.format, self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = format, n_pages, page, heads, dim
        self._struct = _KvCacheStruct(k.data_ptr(), v.data_ptr(), k_scales.data_ptr() if fp4 else None,
                                      v_scales.data_ptr() if fp4 else None, k_gs.data_ptr(), v_gs.data_ptr(),
                                      KV_FORMATS[format], n_pages, page, heads, dim)
        self._ptr = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, k_gs: torch.Tensor,
              v_gs: torch.Tensor, *, format: str = "fp8") -> "KvCache":
        """A new cache of zeros beside its tensor scales."""
        fp4 = format == "nvfp4"
        width = head_dim // 2 if fp4 else head_dim

        def zeros(*shape):
            return torch.zeros((n_pages, n_kv_heads, *shape), dtype=torch.uint8, device=k_gs.device)

        return cls(zeros(page_size, width), zeros(width, page_size), k_gs, v_gs,
                   zeros(page_size, head_dim // 16) if fp4 else None, zeros(head_dim // 16, page_size) if fp4 else None,
                   format=format)


def _one_device(*ts):
    """Number of the GPU that all of them are on."""
    dev = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("the tensors of a call must be on one GPU")
    return dev


def _launch_stream(dev, stream):
    """The raw stream of a call on tensors of GPU `dev`, which must be the current one and the stream's."""
    if dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        raise ValueError("the tensors, the stream and the current device must be of one GPU")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _kv_rows(cache, page_table, kv_lens, cu_seqlens, T):
    """(page table, its row stride, pages a row, lengths, cu_seqlens, sequences) of a call on T rows."""
    n_seqs = kv_lens.shape[0] if kv_lens.dim() == 1 else 0
    lp = _vector(kv_lens, torch.int32, n_seqs, "kv_lens")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != n_seqs \
            or (page_table.stride(1) != 1 and page_table.shape[1] > 1) or not page_table.is_cuda:
        raise ValueError("page_table must be int32 [n_seqs, pages] with unit column stride on the GPU")
    cp = None
    if cu_seqlens is not None:
        cp = _vector(cu_seqlens, torch.int32, n_seqs + 1, "cu_seqlens")
    elif T != n_seqs:
        raise ValueError("without cu_seqlens there is one row for each sequence")
    pages = page_table.shape[1]
    return page_table.data_ptr(), page_table.stride(0) if n_seqs > 1 else max(pages, 1), pages, lp, cp, n_seqs


def qk_norm_rope(x: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor, cos_sin: torch.Tensor,
                 positions: torch.Tensor, *, q_col: int, k_col: int, n_q_heads: int, n_kv_heads: int,
                 eps: float = 1e-6, pair_axis: bytes | None = None, adjacent: bool = False,
                 q: torch.Tensor | None = None, k: torch.Tensor | None = None, stream=None):
    """RMSNorm of each query and key head of x (bf16 or fp32 [T, cols], q heads
    from column q_col, k heads from k_col) times q_weight / k_weight (float32
    [head_dim]), then the rotation of its first cos_sin.shape[1] dims by row
    positions[t] of cos_sin (float32 [n_pos, rot]: cosines, then sines).
    positions: int32 [T], or [axes, T] with pair_axis, rot / 2 bytes that name
    the axis of each pair.  Pairs are (p, p + rot / 2), or (2 p, 2 p + 1) if
    adjacent.  Returns (q, k), bf16 [T, heads * head_dim]."""
    xp, x_dtype, T, cols, ldx = _rows(x, "x")
    dim = q_weight.numel()
    if min(q_col, k_col) < 0 or max(q_col + n_q_heads * dim, k_col + n_kv_heads * dim) > cols:
        raise ValueError(f"the heads must lie in the {cols} columns of x")
    wq, wk = _vector(q_weight, torch.float32, dim, "q_weight"), _vector(k_weight, torch.float32, dim, "k_weight")
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous() or not cos_sin.is_cuda:
        raise ValueError("cos_sin must be contiguous float32 [n_pos, rot] on the GPU")
    n_pos, rot = cos_sin.shape
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    if positions.dtype != torch.int32 or positions.shape[-1] != T or positions.dim() not in (1, 2) \
            or not positions.is_contiguous() or not positions.is_cuda:
        raise ValueError("positions must be contiguous int32 [T] or [axes, T] on the GPU")
    if axes > 1 and (pair_axis is None or len(pair_axis) != rot // 2):
        raise ValueError("several axes need pair_axis, one byte for each of the rot / 2 pairs")
    if q is None:
        q = _new((T, n_q_heads * dim), torch.bfloat16, x.device, stream)
    if k is None:
        k = _new((T, n_kv_heads * dim), torch.bfloat16, x.device, stream)
    qp, q_dtype, ldq = _out_rows(q, T, n_q_heads * dim, "q")
    kp, k_dtype, ldk = _out_rows(k, T, n_kv_heads * dim, "k")
    if q_dtype != OUT_BF16 or k_dtype != OUT_BF16:
        raise ValueError("q and k must be bf16")
    dev = _one_device(x, q_weight, k_weight, cos_sin, positions, q, k)
    st = load().nvfp4_qk_norm_rope(xp, x_dtype, ldx, q_col, k_col, T, n_q_heads, n_kv_heads, dim, wq, wk, eps,
                                   cos_sin.data_ptr(), n_pos, rot, positions.data_ptr(), axes,
                                   bytes(pair_axis) if axes > 1 else None, int(adjacent), qp, ldq, kp, ldk,
                                   _launch_stream(dev, stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_qk_norm_rope")
    return q, k


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, cache: KvCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
                   cu_seqlens: torch.Tensor | None = None, *, stream=None) -> None:
    """Quantise rows of keys and values (bf16 or fp32 [T, n_kv_heads * head_dim])
    into the cache: row j of the n rows of sequence i (cu_seqlens, or one row
    each) goes to position kv_lens[i] - n + j, in page page_table[i, position
    // page_size]."""
    kp, dtype, T, cols, ldk = _rows(k, "k")
    vp, v_dtype, v_rows, v_cols, ldv = _rows(v, "v")
    want = cache.n_kv_heads * cache.head_dim
    if v_dtype != dtype or v_rows != T or cols != want or v_cols != want:
        raise ValueError(f"k and v must be [T, {want}] of one type")
    tp, ldt, pages, lp, cp, n_seqs = _kv_rows(cache, page_table, kv_lens, cu_seqlens, T)
    dev = _one_device(k, v, page_table, kv_lens, cu_seqlens if cp else kv_lens)
    if dev != cache.device:
        raise ValueError("the tensors of a call must be on one GPU")
    st = load().nvfp4_kv_cache_write(cache._ptr, tp, ldt, pages, lp, cp, n_seqs, T, kp, ldk, vp, ldv, dtype,
                                     _launch_stream(dev, stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_kv_cache_write")


def kv_cache_read(cache: KvCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
                  cu_seqlens: torch.Tensor | None = None, *, rows: int | None = None, out_dtype=torch.bfloat16,
                  k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """The values at the last n positions before kv_lens[i] of each sequence, n
    its rows in cu_seqlens (or one).  k and v: [rows, >= n_kv_heads * head_dim],
    bf16 or fp32, made in out_dtype where they are not given.  Returns (k, v)."""
    cols = cache.n_kv_heads * cache.head_dim
    if k is None or v is None:
        if rows is None:
            rows = k.shape[0] if k is not None else v.shape[0] if v is not None else \
                kv_lens.shape[0] if cu_seqlens is None else None
        if rows is None:
            raise ValueError("rows, or k and v, must be given with cu_seqlens")
        dtype = k.dtype if k is not None else v.dtype if v is not None else out_dtype
        k = _new((rows, cols), dtype, kv_lens.device, stream) if k is None else k
        v = _new((rows, cols), dtype, kv_lens.device, stream) if v is None else v
    T = k.shape[0]
    kp, dtype, ldk = _out_rows(k, T, cols, "k")
    vp, v_dtype, ldv = _out_rows(v, T, cols, "v")
    if dtype != v_dtype:
        raise ValueError("k and v must be of one type")
    tp, ldt, pages, lp, cp, n_seqs = _kv_rows(cache, page_table, kv_lens, cu_seqlens, T)
    dev = _one_device(k, v, page_table, kv_lens, cu_seqlens if cp else kv_lens)
    if dev != cache.device:
        raise ValueError("the tensors of a call must be on one GPU")
    st = load().nvfp4_kv_cache_read(cache._ptr, tp, ldt, pages, lp, cp, n_seqs, T, kp, ldk, vp, ldv, dtype,
                                    _launch_stream(dev, stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_kv_cache_read")
    return k, v


def attn_cached(q: torch.Tensor, cache: KvCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
                cu_seqlens: torch.Tensor | None = None, *, n_q_heads: int, scale: float | None = None,
                tree: torch.Tensor | None = None, o: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """Attention of the rows q (bf16 [T, n_q_heads * head_dim]) over a cache that
    holds their keys and values already.  A row sees the positions up to its
    own, or with tree (int64 [T], drafted tokens) every position before the
    sequence's first new row and new row b if bit b of its mask is set.  scale
    defaults to 1 / sqrt(head_dim).  Returns o, bf16 [T, n_q_heads * head_dim]."""
    qp, q_dtype, T, q_cols, ldq = _rows(q, "q")
    dim, heads = cache.head_dim, cache.n_kv_heads
    cols = n_q_heads * dim
    if q_dtype != IN_BF16 or q_cols < cols:
        raise ValueError(f"q must be bf16 [T, >= {cols}]")
    tp, ldt, pages, lp, cp, n_seqs = _kv_rows(cache, page_table, kv_lens, cu_seqlens, T)
    mp = _vector(tree, torch.int64, T, "tree") if tree is not None else None
    if o is None:
        o = _new((T, cols), torch.bfloat16, q.device, stream)
    op, o_dtype, ldo = _out_rows(o, T, cols, "o")
    if o_dtype != OUT_BF16:
        raise ValueError("o must be bf16")
    lib = load()
    need = lib.nvfp4_attn_cached_workspace_size(T, n_seqs, n_q_heads, heads, dim)
    if workspace is None:
        workspace = _new(need, torch.uint8, q.device, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    dev = _one_device(q, page_table, kv_lens, cu_seqlens if cp else q, tree if mp else q, o, workspace)
    if dev != cache.device:
        raise ValueError("the tensors of a call must be on one GPU")
    st = lib.nvfp4_attn_cached(cache._ptr, tp, ldt, pages, lp, cp, n_seqs, T, qp, ldq, n_q_heads,
                               dim ** -0.5 if scale is None else scale, mp, op, ldo, workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _launch_stream(dev, stream))
    if st:
        raise Nvfp4Error(st, "nvfp4_attn_cached")
    return o


def quantize_gemm(x: torch.Tensor, a_gs: torch.Tensor, w_codes, w_scales, w_gs, *, out_dtype=torch.float32,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """y = gemm(quantize(x, a_gs), W) in one call (one kernel for decode-sized x)."""
    if x.dim() != 2 or x.stride(1) != 1 or x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be a 2-D bf16 or fp32 tensor with unit column stride")
    M, K = x.shape
    N = w_codes.shape[0]
    if K % 16:
        raise ValueError("K must be a multiple of 16")
    _u8_matrix(w_codes, (N, K // 2), "w_codes")
    _u8_matrix(w_scales, (N, K // 16), "w_scales")
    _f32_scalars(a_gs, 1, "a_gs")
    _f32_scalars(w_gs, 1, "w_gs")
    dt = IN_BF16 if x.dtype == torch.bfloat16 else IN_F32
    od = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}[out_dtype]
    if out is not None:
        _out_matrix(out, M, N, out_dtype)
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _need_gpu(x, a_gs, w_codes, w_scales, w_gs, out, workspace)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    lib = load()
    ws_bytes = lib.nvfp4_quantize_gemm_workspace_size(M, N, K, dt, od)
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    ws_ptr = _ptr(workspace) if ws_bytes else None
    ws_have = workspace.numel() * workspace.element_size() if (ws_bytes and workspace is not None) else 0
    st = lib.nvfp4_quantize_gemm(_ptr(x), dt, x.stride(0), _ptr(a_gs), _ptr(w_codes), _ptr(w_scales), _ptr(w_gs),
                                 M, N, K, _ptr(out), od, out.stride(0), ws_ptr, ws_have, _stream(stream))
    _check(st, "nvfp4_quantize_gemm")
    return out


def quantize_gemm_no_alloc(x: torch.Tensor, a_gs: torch.Tensor, w_codes, w_scales, w_gs, *,
                           out_dtype=torch.float32, out: torch.Tensor | None = None, stream=None):
    """quantize_gemm without a workspace: the library's static device scratch
    holds the quantized activations (nvfp4_quantize_gemm_no_alloc; calls
    that overlap on one GPU race on it).  Allocates out only if not given."""
    if x.dim() != 2 or x.stride(1) != 1 or x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be a 2-D bf16 or fp32 tensor with unit column stride")
    M, K = x.shape
    N = w_codes.shape[0]
    if K % 16:
        raise ValueError("K must be a multiple of 16")
    _u8_matrix(w_codes, (N, K // 2), "w_codes")
    _u8_matrix(w_scales, (N, K // 16), "w_scales")
    _f32_scalars(a_gs, 1, "a_gs")
    _f32_scalars(w_gs, 1, "w_gs")
    dt = IN_BF16 if x.dtype == torch.bfloat16 else IN_F32
    od = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}[out_dtype]
    if out is not None:
        _out_matrix(out, M, N, out_dtype)
    _need_gpu(x, a_gs, w_codes, w_scales, w_gs, out)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    st = load().nvfp4_quantize_gemm_no_alloc(_ptr(x), dt, x.stride(0), _ptr(a_gs), _ptr(w_codes), _ptr(w_scales),
                                             _ptr(w_gs), M, N, K, _ptr(out), od, out.stride(0), _stream(stream))
    _check(st, "nvfp4_quantize_gemm_no_alloc")
    return out


def harmonize_fused_scales(scales: torch.Tensor, module_gs: torch.Tensor, module_rows, k: int, *,
                           shared_gs: torch.Tensor | None = None, counters: torch.Tensor | None = None,
                           stream=None):
    """Rescale (in place) the block scales of modules concatenated along N to
    the shared tensor scale g* = max(module_gs).  Returns (shared_gs, counters)."""
    _need_gpu(scales, module_gs, shared_gs, counters)
    rows = (ctypes.c_int64 * len(module_rows))(*[int(r) for r in module_rows])
    if shared_gs is None:
        shared_gs = torch.empty(1, dtype=torch.float32, device=scales.device)
    if counters is None:
        counters = torch.zeros(2, dtype=torch.int32, device=scales.device)
    st = load().nvfp4_harmonize_fused_scales(_ptr(scales), _ptr(module_gs), rows, len(module_rows), k,
                                              _ptr(shared_gs), _ptr(counters), _stream(stream))
    _check(st, "nvfp4_harmonize_fused_scales")
    return shared_gs, counters
