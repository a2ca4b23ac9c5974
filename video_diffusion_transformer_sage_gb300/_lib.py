"""ctypes binding of `libsage_gb300.so` (include/sage.h): argument marshalling only.

Every step of the attention path runs in the library's CUDA kernels; this module only turns
torch tensors into pointers, sizes and strides, allocates outputs and workspaces with
torch, and raises `SageError` on a non-OK status.  There is no fallback: if the library is
missing the import of any op raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import re
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libsage_gb300.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "sage.h")
PAGED_HEADER = os.path.join(os.path.dirname(_HERE), "include", "sage_paged.h")
TREE_HEADER = os.path.join(os.path.dirname(_HERE), "include", "sage_paged_tree.h")
POOL_HEADER = os.path.join(os.path.dirname(_HERE), "include", "sage_paged_pool.h")
PAGED_WS_HEADER = 4096   # SAGE_PAGED_WS_HEADER: the bytes of a paged workspace that start as zeros

STATUS = {0: "SAGE_OK", 1: "SAGE_ERR_INVALID_ARG", 2: "SAGE_ERR_ALIGNMENT", 3: "SAGE_ERR_UNSUPPORTED",
          4: "SAGE_ERR_WORKSPACE", 5: "SAGE_ERR_CUDA", 6: "SAGE_ERR_DEVICE_TIMEOUT"}


class SageError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


class SageView(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_tokens", ctypes.c_int64), ("n_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("stride_token", ctypes.c_int64),
                ("stride_head", ctypes.c_int64)]


class SageQuantizedC(ctypes.Structure):
    _fields_ = [("q_codes", ctypes.c_void_p), ("q_scales", ctypes.c_void_p), ("k_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("k_mean", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("q_block", ctypes.c_int64), ("v_format", ctypes.c_int64),
                ("v_mean", ctypes.c_void_p)]

V_FORMATS = {"e4m3": 0, "int8": 1}


_lib = None


class SagePagedKVC(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("n_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("k_stride_page", ctypes.c_int64), ("k_stride_token", ctypes.c_int64),
                ("k_stride_head", ctypes.c_int64), ("v_stride_page", ctypes.c_int64),
                ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64), ("format", ctypes.c_int64),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class SagePagedBatchC(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int64), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64)]


class SagePagedTreeMaskC(ctypes.Structure):
    _fields_ = [("mask", ctypes.c_void_p), ("mask_words", ctypes.c_int64), ("mask_stride", ctypes.c_int64),
                ("depth", ctypes.c_void_p)]


class SagePagedPoolC(ctypes.Structure):
    _fields_ = [("refs", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("n_rows", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int64)]


def header_functions(header: str = HEADER) -> list:
    """Names of the functions a header (include/sage.h, PAGED_HEADER, TREE_HEADER, POOL_HEADER) declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\**\s+\**(sage_[a-z_0-9]+)\s*\(", text, re.M)))


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        VP = ctypes.POINTER(SageView)
        QP = ctypes.POINTER(SageQuantizedC)
        KP, BP = ctypes.POINTER(SagePagedKVC), ctypes.POINTER(SagePagedBatchC)
        TP, OP = ctypes.POINTER(SagePagedTreeMaskC), ctypes.POINTER(SagePagedPoolC)
        sig = {
            "sage_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "sage_quant_scratch_bytes": ([I, I, I], S),
            "sage_workspace_bytes": ([I, I, I], S),
            "sage_status_block_bytes": ([], S),
            "sage_smooth_quant_qk": ([VP, VP, QP, P, S, P], ctypes.c_int),
            "sage_quant_v": ([VP, QP, P, S, P], ctypes.c_int),
            "sage_quant_qkv": ([VP, VP, VP, QP, P, S, P], ctypes.c_int),
            "sage_smooth_quant_qk_noalloc": ([VP, VP, QP, P], ctypes.c_int),
            "sage_attn_fwd_quantized": ([I, I, I, QP, F, P, I, I, P, P], ctypes.c_int),
            "sage_attn_fwd": ([VP, VP, VP, F, P, I, I, P, S, P], ctypes.c_int),
            "sage_attn_dense_bf16": ([VP, VP, VP, F, P, I, I, P], ctypes.c_int),
            "sage_dense_workspace_bytes": ([I, I, I], S),
            "sage_attn_dense_bf16_tc": ([VP, VP, VP, F, P, I, I, P, S, P], ctypes.c_int),
            "sage_debug_qk_int32": ([I, I, I, QP, I, I, I, I, I, P, P, P], ctypes.c_int),
            "sage_check_device_status": ([P, P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
            "sage_get_device_status": ([P, P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
            "sage_debug_wait_timeout": ([P, I, P], ctypes.c_int),
            "sage_measure_mma_rate": ([I, I, I, P, P], ctypes.c_int),
            "sage_qk_rmsnorm_rope": ([VP, VP, P, P, P, P, F, P], ctypes.c_int),
            "sage_smooth_quant_qk_rmsnorm_rope": ([VP, VP, P, P, P, P, F, QP, P, S, P], ctypes.c_int),
            "sage_paged_append": ([VP, VP, VP, P, P, P, P, I, P, F, KP, BP, P, I, I, P, P], ctypes.c_int),
            "sage_paged_workspace_bytes": ([I], S),
            "sage_paged_attn": ([VP, KP, BP, F, I, I, P, I, I, P, P, S, P], ctypes.c_int),
            "sage_paged_tree": ([BP, I, P, I, TP, P, P, P], ctypes.c_int),
            "sage_paged_pool_workspace_bytes": ([I, I], S),
            "sage_paged_release": ([OP, P, P, P, P], ctypes.c_int),
            "sage_paged_reserve": ([OP, P, P, P, P, S, P], ctypes.c_int),
            "sage_paged_fork": ([OP, P, P, P, I, P, P, P, P, P, S, P], ctypes.c_int),
            "sage_paged_copy": ([KP, P, P, P, I, P, P], ctypes.c_int),
            "sage_paged_compact": ([KP, BP, P, P, I, I, P, P, S, P], ctypes.c_int),
            "sage_paged_attn_tree": ([VP, KP, BP, TP, F, I, P, I, I, P, P, S, P], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(code: int, what: str) -> None:
    if code != 0:
        raise SageError(code, what)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def make_view(t: torch.Tensor) -> SageView:
    """A bf16 CUDA [N, H, D] tensor (any token / head strides, unit channel stride)."""
    if t.dim() != 3 or t.dtype != torch.bfloat16 or not t.is_cuda or t.stride(2) != 1:
        raise ValueError("expected a bf16 CUDA [N, H, D] tensor with unit channel stride")
    n, h, d = t.shape
    return SageView(t.data_ptr(), n, h, d, t.stride(0), t.stride(1))


def pad128(n: int) -> int:
    return (n + 127) // 128 * 128


class Quantized:
    """Device buffers of the quantised operands (layouts of sage_quantized in include/sage.h)."""

    def __init__(self, n: int, h: int, d: int, device="cuda", q_block: int = 128, v_format: str = "e4m3",
                 smooth_v: bool = False):
        """q_block: rows per Q scale (128, the method's default, or a smaller power of two).
        v_format: "e4m3" (the method's FP8 V and P) or "int8" (the INT8 P.V variant; codes held
        as fp16).  smooth_v: quantise V minus its channel mean and add the mean back."""
        np_ = pad128(n)
        if q_block not in (1, 2, 4, 8, 16, 32, 64, 128):
            raise ValueError(f"q_block must be a power of two <= 128, got {q_block}")
        if v_format not in V_FORMATS:
            raise ValueError(f"v_format must be one of {sorted(V_FORMATS)}, got {v_format!r}")
        self.n, self.h, self.d, self.q_block, self.v_format = n, h, d, q_block, v_format
        self.q_codes = torch.empty((h, np_, d), dtype=torch.float16, device=device)
        self.k_codes = torch.empty((h, np_, d), dtype=torch.float16, device=device)
        self.v_codes = torch.empty((h, d, np_), dtype=torch.float16 if v_format == "int8" else torch.uint8,
                                   device=device)
        self.v_mean = torch.empty((h, d), dtype=torch.float32, device=device) if smooth_v else None
        self.q_scales = torch.empty((h, np_ // q_block), dtype=torch.float32, device=device)
        self.k_scales = torch.empty((h, np_ // 64), dtype=torch.float32, device=device)
        self.k_mean = torch.empty((h, d), dtype=torch.float32, device=device)
        self.v_scales = torch.empty((h, d), dtype=torch.float32, device=device)

    def c(self) -> SageQuantizedC:
        return SageQuantizedC(self.q_codes.data_ptr(), self.q_scales.data_ptr(), self.k_codes.data_ptr(),
                              self.k_scales.data_ptr(), self.k_mean.data_ptr(), self.v_codes.data_ptr(),
                              self.v_scales.data_ptr(), self.q_block, V_FORMATS[self.v_format],
                              None if self.v_mean is None else self.v_mean.data_ptr())


def quant_scratch(n: int, h: int, d: int, device="cuda") -> torch.Tensor:
    return torch.empty(int(lib().sage_quant_scratch_bytes(n, h, d)), dtype=torch.uint8, device=device)


def status_block(device="cuda") -> torch.Tensor:
    return torch.zeros(int(lib().sage_status_block_bytes()), dtype=torch.uint8, device=device)


def workspace(n: int, h: int, d: int, device="cuda") -> torch.Tensor:
    """Workspace for sage_attn_fwd; its leading status block starts zeroed."""
    ws = torch.empty(int(lib().sage_workspace_bytes(n, h, d)) + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + int(lib().sage_workspace_bytes(n, h, d))]
    ws[:256].zero_()
    return ws


def sage_smooth_quant_qk(q: torch.Tensor, k: torch.Tensor, qz: Optional[Quantized] = None,
                         scratch: Optional[torch.Tensor] = None, stream=None, q_block: int = 128,
                         v_format: str = "e4m3", smooth_v: bool = False) -> Quantized:
    """When qz is None a Quantized is made here; q_block, v_format and smooth_v set it up
    (the V options take effect in sage_quant_v and the attention)."""
    n, h, d = q.shape
    qz = qz or Quantized(n, h, d, q.device, q_block, v_format, smooth_v)
    scratch = scratch if scratch is not None else quant_scratch(n, h, d, q.device)
    vq, vk, c = make_view(q), make_view(k), qz.c()
    _check(lib().sage_smooth_quant_qk(ctypes.byref(vq), ctypes.byref(vk), ctypes.byref(c), scratch.data_ptr(),
                                      scratch.numel(), _stream(stream)), "sage_smooth_quant_qk")
    return qz


def sage_smooth_quant_qk_noalloc(q: torch.Tensor, k: torch.Tensor, qz: Optional[Quantized] = None,
                                 stream=None) -> Quantized:
    """sage_smooth_quant_qk for callers that cannot allocate: the library's fixed device
    scratch array replaces the caller workspace (see include/sage.h for the size limit)."""
    n, h, d = q.shape
    qz = qz or Quantized(n, h, d, q.device)
    vq, vk, c = make_view(q), make_view(k), qz.c()
    _check(lib().sage_smooth_quant_qk_noalloc(ctypes.byref(vq), ctypes.byref(vk), ctypes.byref(c), _stream(stream)),
           "sage_smooth_quant_qk_noalloc")
    return qz


def sage_quant_v(v: torch.Tensor, qz: Quantized, scratch: Optional[torch.Tensor] = None, stream=None) -> Quantized:
    n, h, d = v.shape
    scratch = scratch if scratch is not None else quant_scratch(n, h, d, v.device)
    vv, c = make_view(v), qz.c()
    _check(lib().sage_quant_v(ctypes.byref(vv), ctypes.byref(c), scratch.data_ptr(), scratch.numel(),
                              _stream(stream)), "sage_quant_v")
    return qz


def sage_quant_qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, qz: Optional[Quantized] = None,
                   scratch: Optional[torch.Tensor] = None, stream=None, q_block: int = 128, v_format: str = "e4m3",
                   smooth_v: bool = False) -> Quantized:
    """sage_smooth_quant_qk then sage_quant_v in one call (5 launches on the default options).
    scratch: at least 2 * sage_quant_scratch_bytes bytes (made here when None)."""
    n, h, d = q.shape
    qz = qz or Quantized(n, h, d, q.device, q_block, v_format, smooth_v)
    if scratch is None:
        scratch = torch.empty(2 * int(lib().sage_quant_scratch_bytes(n, h, d)), dtype=torch.uint8, device=q.device)
    vq, vk, vv, c = make_view(q), make_view(k), make_view(v), qz.c()
    _check(lib().sage_quant_qkv(ctypes.byref(vq), ctypes.byref(vk), ctypes.byref(vv), ctypes.byref(c),
                                scratch.data_ptr(), scratch.numel(), _stream(stream)), "sage_quant_qkv")
    return qz


def _out_args(out: Optional[torch.Tensor], n: int, h: int, d: int, device):
    if out is None:
        out = torch.empty((n, h, d), dtype=torch.bfloat16, device=device)
    if out.dtype != torch.bfloat16 or out.stride(2) != 1 or tuple(out.shape) != (n, h, d):
        raise ValueError("out must be bf16 [N, H, D] with unit channel stride")
    return out, out.stride(0), out.stride(1)


def sage_attn_fwd_quantized(qz: Quantized, sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                            status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    sm_scale = 1.0 / math.sqrt(qz.d) if sm_scale is None else sm_scale
    out, ost, osh = _out_args(out, qz.n, qz.h, qz.d, qz.q_codes.device)
    status = status if status is not None else status_block(qz.q_codes.device)
    c = qz.c()
    _check(lib().sage_attn_fwd_quantized(qz.n, qz.h, qz.d, ctypes.byref(c), sm_scale, out.data_ptr(), ost, osh,
                                         status.data_ptr(), _stream(stream)), "sage_attn_fwd_quantized")
    return out


def sage_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, sm_scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    n, h, d = q.shape
    sm_scale = 1.0 / math.sqrt(d) if sm_scale is None else sm_scale
    out, ost, osh = _out_args(out, n, h, d, q.device)
    ws = ws if ws is not None else workspace(n, h, d, q.device)
    vq, vk, vv = make_view(q), make_view(k), make_view(v)
    _check(lib().sage_attn_fwd(ctypes.byref(vq), ctypes.byref(vk), ctypes.byref(vv), sm_scale, out.data_ptr(), ost,
                               osh, ws.data_ptr(), ws.numel(), _stream(stream)), "sage_attn_fwd")
    return out


def sage_attn_dense_bf16(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, sm_scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    n, h, d = q.shape
    sm_scale = 1.0 / math.sqrt(d) if sm_scale is None else sm_scale
    out, ost, osh = _out_args(out, n, h, d, q.device)
    vq, vk, vv = make_view(q), make_view(k), make_view(v)
    _check(lib().sage_attn_dense_bf16(ctypes.byref(vq), ctypes.byref(vk), ctypes.byref(vv), sm_scale,
                                      out.data_ptr(), ost, osh, _stream(stream)), "sage_attn_dense_bf16")
    return out


def dense_workspace(n: int, h: int, d: int, device="cuda") -> torch.Tensor:
    """Workspace for sage_attn_dense_bf16_tc; its leading status block starts zeroed."""
    need = int(lib().sage_dense_workspace_bytes(n, h, d))
    ws = torch.empty(need + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + need]
    ws[:256].zero_()
    return ws


def sage_attn_dense_bf16_tc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, sm_scale: Optional[float] = None,
                            out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    n, h, d = q.shape
    sm_scale = 1.0 / math.sqrt(d) if sm_scale is None else sm_scale
    out, ost, osh = _out_args(out, n, h, d, q.device)
    ws = dense_workspace(n, h, d, q.device) if ws is None else ws
    vq, vk, vv = make_view(q), make_view(k), make_view(v)
    _check(lib().sage_attn_dense_bf16_tc(ctypes.byref(vq), ctypes.byref(vk), ctypes.byref(vv), sm_scale,
                                         out.data_ptr(), ost, osh, ws.data_ptr(), ws.numel(), _stream(stream)),
           "sage_attn_dense_bf16_tc")
    return out


def sage_debug_qk_int32(qz: Quantized, head: int, i0: int, j0: int, row_tiles: int = 1, col_tiles: int = 1,
                        status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    out = torch.empty((128 * row_tiles, 128 * col_tiles), dtype=torch.int32, device=qz.q_codes.device)
    status = status if status is not None else status_block(qz.q_codes.device)
    c = qz.c()
    _check(lib().sage_debug_qk_int32(qz.n, qz.h, qz.d, ctypes.byref(c), head, i0, j0, row_tiles, col_tiles,
                                     out.data_ptr(), status.data_ptr(), _stream(stream)), "sage_debug_qk_int32")
    return out


def sage_debug_wait_timeout(status: torch.Tensor, limit_ns: int, stream=None) -> None:
    _check(lib().sage_debug_wait_timeout(status.data_ptr(), int(limit_ns), _stream(stream)), "sage_debug_wait_timeout")


# FLOPs per CTA and round of each sage_measure_mma_rate mode (2 M N K per MMA).
MMA_RATE_FLOPS = {0: 8 * 2 * 128 * 128 * 16, 1: 8 * 2 * 128 * 128 * 32, 2: 8 * 2 * 128 * 128 * 16 + 4 * 2 * 128 * 128 * 32,
                  3: 8 * 2 * 128 * 256 * 32, 4: 8 * 2 * 128 * 256 * 16, 5: 8 * 2 * 128 * 64 * 32,
                  6: 4 * 2 * 128 * 128 * 16 + 4 * 2 * 128 * 64 * 32}


def sage_measure_mma_rate(mode: int, iters: int, ctas: int, status: torch.Tensor, stream=None) -> None:
    _check(lib().sage_measure_mma_rate(int(mode), int(iters), int(ctas), status.data_ptr(), _stream(stream)),
           "sage_measure_mma_rate")


def sage_check_device_status(status: torch.Tensor, stream=None):
    """Synchronises `stream`; returns (status code, where) and clears a recorded timeout."""
    where = ctypes.c_int32(0)
    code = lib().sage_check_device_status(status.data_ptr(), _stream(stream), ctypes.byref(where))
    return int(code), int(where.value)


def sage_qk_rmsnorm_rope(q: torch.Tensor, k: torch.Tensor, gamma_q: torch.Tensor, gamma_k: torch.Tensor,
                         rope_cos: torch.Tensor, rope_sin: torch.Tensor, eps: float = 1e-6, stream=None) -> None:
    """In place on the bf16 [N, H, D] CUDA views q and k: RMSNorm over D (weights gamma_q /
    gamma_k, fp32 [D]) and the rotation of channel pairs by the fp32 [N, D/2] cos / sin table."""
    n, h, d = q.shape
    for t, shape in ((gamma_q, (d,)), (gamma_k, (d,)), (rope_cos, (n, d // 2)), (rope_sin, (n, d // 2))):
        if t.dtype != torch.float32 or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"expected a contiguous fp32 CUDA tensor of shape {shape}")
    vq, vk = make_view(q), make_view(k)
    _check(lib().sage_qk_rmsnorm_rope(ctypes.byref(vq), ctypes.byref(vk), gamma_q.data_ptr(), gamma_k.data_ptr(),
                                      rope_cos.data_ptr(), rope_sin.data_ptr(), float(eps), _stream(stream)),
           "sage_qk_rmsnorm_rope")


def _check_transform_tables(n: int, d: int, gamma_q, gamma_k, rope_cos, rope_sin) -> None:
    for t, shape in ((gamma_q, (d,)), (gamma_k, (d,)), (rope_cos, (n, d // 2)), (rope_sin, (n, d // 2))):
        if t.dtype != torch.float32 or not t.is_cuda or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"expected a contiguous fp32 CUDA tensor of shape {shape}")


def sage_smooth_quant_qk_rmsnorm_rope(q: torch.Tensor, k: torch.Tensor, gamma_q: torch.Tensor, gamma_k: torch.Tensor,
                                      rope_cos: torch.Tensor, rope_sin: torch.Tensor, eps: float = 1e-6,
                                      qz: Optional[Quantized] = None, scratch: Optional[torch.Tensor] = None,
                                      stream=None, q_block: int = 128, v_format: str = "e4m3",
                                      smooth_v: bool = False) -> Quantized:
    """sage_qk_rmsnorm_rope then sage_smooth_quant_qk in one pass, without modifying q and k:
    the transform runs in the quantise kernels' prologue."""
    n, h, d = q.shape
    _check_transform_tables(n, d, gamma_q, gamma_k, rope_cos, rope_sin)
    qz = qz or Quantized(n, h, d, q.device, q_block, v_format, smooth_v)
    scratch = scratch if scratch is not None else quant_scratch(n, h, d, q.device)
    vq, vk, c = make_view(q), make_view(k), qz.c()
    _check(lib().sage_smooth_quant_qk_rmsnorm_rope(ctypes.byref(vq), ctypes.byref(vk), gamma_q.data_ptr(),
                                                   gamma_k.data_ptr(), rope_cos.data_ptr(), rope_sin.data_ptr(),
                                                   float(eps), ctypes.byref(c), scratch.data_ptr(), scratch.numel(),
                                                   _stream(stream)), "sage_smooth_quant_qk_rmsnorm_rope")
    return qz


# ------------------------------------------------------------------- paged K/V cache (include/sage_paged.h)
@functools.lru_cache(maxsize=None)
def _driver():
    return ctypes.CDLL("libcuda.so.1")


@functools.lru_cache(maxsize=None)
def _side_stream(index: int) -> torch.cuda.Stream:
    """The stream of a device that status blocks are zeroed on, apart from whatever else goes on.  Not one of torch's: those are
    given out again after 32, and a capture on the same stream would take the zeroing in and fail at the wait for it."""
    driver, device = _driver(), ctypes.c_int()
    context, stream = ctypes.c_void_p(), ctypes.c_void_p()

    def call(name, *args):
        code = getattr(driver, name)(*args)
        if code != 0:
            raise RuntimeError(f"{name} failed: {code}")

    call("cuDeviceGet", ctypes.byref(device), index)
    call("cuDevicePrimaryCtxRetain", ctypes.byref(context), device)   # torch's context, for the life of the process
    call("cuCtxPushCurrent_v2", context)
    try:
        call("cuStreamCreate", ctypes.byref(stream), 1)               # 1: does not wait for the default stream
    finally:
        call("cuCtxPopCurrent_v2", ctypes.byref(context))
    return torch.cuda.ExternalStream(stream.value, device=torch.device("cuda", index))


@contextlib.contextmanager
def _capture_apart():
    """What this thread enqueues and waits for on streams that are not captured does not end a capture on another one
    (cuThreadExchangeStreamCaptureMode: relaxed)."""
    mode, driver = ctypes.c_int(2), _driver()
    if driver.cuThreadExchangeStreamCaptureMode(ctypes.byref(mode)) != 0:
        raise RuntimeError("cuThreadExchangeStreamCaptureMode failed")
    try:
        yield
    finally:
        driver.cuThreadExchangeStreamCaptureMode(ctypes.byref(mode))


class _StatusOwner:
    """Holds a status block (and scratch behind it), made when first needed; it may be used on any stream."""

    def _own_status(self, device, nbytes: int) -> None:
        self.device, self._status_bytes, self._status, self._status_streams = device, nbytes, None, set()

    @property
    def status(self) -> torch.Tensor:
        if self._status is None:
            # Zeroed before this returns, on a stream of its own: no call on whatever stream comes before that, and inside
            # a graph capture the zeroing is no part of the graph, whose replays would erase records.
            with _capture_apart():
                side = _side_stream(self.device.index)
                with torch.cuda.stream(side):
                    status = torch.zeros(self._status_bytes, dtype=torch.uint8, device=self.device)
                side.synchronize()
            self._status = status
        return self._status

    def _status_on(self, stream) -> torch.Tensor:
        """The block for a call on `stream`, whose kernels may outlive its owner."""
        status = self.status
        raw = torch._C._cuda_getCurrentRawStream(self.device.index) if stream is None else _stream(stream)
        if raw not in self._status_streams:
            self._status_streams.add(raw)
            status.record_stream(torch.cuda.ExternalStream(raw, device=self.device))
        return status


class PagedKV(_StatusOwner):
    """A paged K/V cache over the caller's page tensors [n_pages, page_size, n_heads, head_dim] (any page,
    slot and head strides, unit channel stride): bf16, or torch.float8_e4m3fn with fp32 scales
    k_scale and v_scale [n_heads].  `status` is the block that sage_paged_append records bad indices in
    (read it with sage_check_device_status); it is made when first needed and may be used on any stream."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
            raise ValueError("k_pages and v_pages must be [n_pages, page_size, n_heads, head_dim] of one shape and type")
        if k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"the cache holds bf16 or float8_e4m3fn, got {k_pages.dtype}")
        e4m3 = k_pages.dtype == torch.float8_e4m3fn
        if (k_scale is not None) != e4m3 or (v_scale is not None) != e4m3:
            raise ValueError("k_scale and v_scale belong to a float8_e4m3fn cache, and it needs both")
        n, ps, h, d = k_pages.shape
        for t in (k_pages, v_pages):
            if not t.is_cuda or t.device != k_pages.device or t.stride(3) != 1:
                raise ValueError("expected CUDA page tensors on one device with unit channel stride")
        for t in (k_scale, v_scale):
            if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (h,) or not t.is_contiguous()
                                  or t.device != k_pages.device):
                raise ValueError(f"expected contiguous fp32 scales of shape ({h},) on the pages' device")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.n_pages, self.page_size, self.n_heads, self.head_dim = n, ps, h, d
        self._own_status(k_pages.device, int(lib().sage_status_block_bytes()))
        self._c = SagePagedKVC(k_pages.data_ptr(), v_pages.data_ptr(), n, ps, h, d, *k_pages.stride()[:3],
                               *v_pages.stride()[:3], 1 if e4m3 else 0, k_scale.data_ptr() if e4m3 else None,
                               v_scale.data_ptr() if e4m3 else None)
        self._ref = ctypes.byref(self._c)


class PagedBatch:
    """The sequences of a call: int32 CUDA tensors cu_q [n + 1] (first row of each sequence's new
    tokens), kv_len [n] (tokens in the cache, the new ones included) and page_table [n, max_pages].  The
    tensors may be rewritten between calls (a captured graph reads them anew)."""

    def __init__(self, cu_q: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor):
        n = kv_len.numel()
        for t in (cu_q, kv_len, page_table):
            if t.dtype != torch.int32 or not t.is_cuda or t.device != cu_q.device:
                raise ValueError("expected int32 CUDA tensors on one device")
        if kv_len.dim() != 1 or tuple(cu_q.shape) != (n + 1,) or page_table.dim() != 2 or page_table.shape[0] != n:
            raise ValueError("expected cu_q [n + 1], kv_len [n] and page_table [n, max_pages]")
        if not cu_q.is_contiguous() or not kv_len.is_contiguous() or (page_table.shape[1] > 1
                                                                      and page_table.stride(1) != 1):
            raise ValueError("cu_q and kv_len must be contiguous, page_table's rows too")
        self.cu_q, self.kv_len, self.page_table, self.n_seqs = cu_q, kv_len, page_table, n
        self.device = cu_q.device
        self._c = SagePagedBatchC(n, cu_q.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), page_table.shape[1],
                                  page_table.stride(0))
        self._ref = ctypes.byref(self._c)


def paged_workspace(head_dim: int, device="cuda") -> torch.Tensor:
    """Workspace for sage_paged_attn; the part that has to start as zeros (the status block first) does."""
    need = int(lib().sage_paged_workspace_bytes(head_dim))
    ws = torch.empty(need + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + need]
    ws[:PAGED_WS_HEADER].zero_()
    return ws


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _paged_view(t: torch.Tensor, d: int, device, what: str) -> SageView:
    if t.dim() != 3:
        raise ValueError(f"{what}: expected a bf16 [N, H, {d}] tensor")
    n, h, channels = t.shape
    token, head, unit = t.stride()
    if channels != d or unit != 1 or t.dtype is not _BF16 or t.device != device:
        raise ValueError(f"{what}: expected a bf16 [N, H, {d}] tensor with unit channel stride on the cache's device")
    return SageView(t.data_ptr(), n, h, d, token, head)


def _paged_call(device, stream, fn, args) -> int:
    """fn(*args, raw stream) with the cache's device current, on `stream` or that device's current stream."""
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == index:
        return fn(*args, raw)
    with torch.cuda.device(device):
        return fn(*args, raw)


def _made_on(stream, device):
    """Where a call makes a buffer: on its own stream, so that zeroing comes before the kernel and the memory's next
    use after it."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream")
                             else torch.cuda.ExternalStream(int(stream), device=device))


def _fp32_table(t: Optional[torch.Tensor], shape: tuple, device, what: str):
    if t is None:
        return None
    if t.dtype is not _F32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous fp32 tensor of shape {shape} on the cache's device")
    return t.data_ptr()


def sage_paged_append(k: torch.Tensor, v: torch.Tensor, cache: PagedKV, batch: PagedBatch,
                      q: Optional[torch.Tensor] = None, gamma_q: Optional[torch.Tensor] = None,
                      gamma_k: Optional[torch.Tensor] = None, rope_cos: Optional[torch.Tensor] = None,
                      rope_sin: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """New tokens' K and V [N, n_heads, D] into the cache, after the optional per-head RMSNorm (gamma_q,
    gamma_k: fp32 [D]) and rotation (rope_cos, rope_sin: fp32 [rows, D / 2]; row = position in the
    sequence, or positions[t], int32) of Q and K.  Returns Q so treated (q_out, made here when None; it
    may be q itself, then with q's strides), or None without q."""
    d, dev = cache.head_dim, cache.device
    vk, vv = _paged_view(k, d, dev, "k"), _paged_view(v, d, dev, "v")
    if batch.device != dev:
        raise ValueError("the batch lies on another device than the cache")
    vq, oargs = None, (None, 0, 0)
    if q is not None:
        vq = _paged_view(q, d, dev, "q")
        if q_out is None:
            with _made_on(stream, dev):
                q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        vo = _paged_view(q_out, d, dev, "q_out")
        if vo.n_tokens != vq.n_tokens or vo.n_heads != vq.n_heads:
            raise ValueError("q_out must have q's shape")
        oargs = (vo.data, vo.stride_token, vo.stride_head)
    elif q_out is not None or gamma_q is not None:
        raise ValueError("q_out and gamma_q belong to q")
    if positions is not None and (positions.dtype is not _I32 or positions.shape != (k.shape[0],)
                                  or not positions.is_contiguous() or positions.device != dev):
        raise ValueError("positions: expected a contiguous int32 tensor [N] on the cache's device")
    if status is None:
        status = cache._status_on(stream)
    elif status.device != dev or status.nbytes < 256:
        raise ValueError("status: expected a zeroed block of 256 bytes on the cache's device")
    rows = rope_cos.shape[0] if rope_cos is not None else 0
    table, weight, by = (rows, d // 2), (d,), ctypes.byref
    _check(_paged_call(dev, stream, lib().sage_paged_append, (
        None if vq is None else by(vq), by(vk), by(vv), _fp32_table(gamma_q, weight, dev, "gamma_q"),
        _fp32_table(gamma_k, weight, dev, "gamma_k"), _fp32_table(rope_cos, table, dev, "rope_cos"),
        _fp32_table(rope_sin, table, dev, "rope_sin"), rows, None if positions is None else positions.data_ptr(), eps,
        cache._ref, batch._ref, *oargs, status.data_ptr())), "sage_paged_append")
    return q_out


def _paged_attn_call(q, cache, batch, between, out, lse, ws, stream, what) -> torch.Tensor:
    """The attention calls: `between` stands between the batch and the output."""
    d, dev = cache.head_dim, cache.device
    vq = _paged_view(q, d, dev, "q")
    if batch.device != dev:
        raise ValueError("the batch lies on another device than the cache")
    if out is None:
        with _made_on(stream, dev):
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    vo = _paged_view(out, d, dev, "out")
    if vo.n_tokens != vq.n_tokens or vo.n_heads != vq.n_heads:
        raise ValueError("out must have q's shape")
    if lse is not None and (lse.dtype is not _F32 or lse.shape != q.shape[:2]
                            or not lse.is_contiguous() or lse.device != dev):
        raise ValueError("lse: expected a contiguous fp32 tensor [N, Hq] on the cache's device")
    if ws is None:
        with _made_on(stream, dev):
            ws = paged_workspace(d, dev)
    elif ws.device != dev:
        raise ValueError("ws lies on another device than the cache")
    _check(_paged_call(dev, stream, getattr(lib(), what), (
        ctypes.byref(vq), cache._ref, batch._ref, *between, vo.data, vo.stride_token,
        vo.stride_head, None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes)), what)
    return out


def sage_paged_attn(q: torch.Tensor, cache: PagedKV, batch: PagedBatch, sm_scale: Optional[float] = None,
                    causal: bool = True, window: Optional[int] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the batch's new tokens q [N, Hq, D] over the cache: all stored tokens of their sequence
    (causal False), those up to their own position, or the last `window` of these (None or 0: all).  lse: optional fp32
    [N, Hq], receives the log of the sum of exponentials.  ws: a paged_workspace (made here when None)."""
    sm_scale = 1.0 / math.sqrt(cache.head_dim) if sm_scale is None else sm_scale
    return _paged_attn_call(q, cache, batch, (sm_scale, 1 if causal else 0, window or 0), out, lse, ws, stream,
                            "sage_paged_attn")


# ------------------------------------------------------------------- drafted trees (include/sage_paged_tree.h)
class PagedTree:
    """Which new tokens each row of a call sees: int32 CUDA tensors mask [N, words] (bit i % 32 of word i / 32: the row sees
    new token i of its sequence), depth [N] (its ancestors; needed with a window) and positions [N] (for sage_paged_append).
    sage_paged_tree fills all three from the tokens' parents."""

    def __init__(self, mask: torch.Tensor, depth: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None):
        if mask.dim() != 2 or mask.dtype != torch.int32 or not mask.is_cuda or mask.shape[1] < 1:
            raise ValueError("mask: expected an int32 CUDA tensor [N, words]")
        n, words = mask.shape
        if words > 1 and mask.stride(1) != 1:
            raise ValueError("mask's rows must be contiguous")
        for t in (depth, positions):
            if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (n,) or not t.is_contiguous()
                                  or t.device != mask.device):
                raise ValueError(f"depth and positions: expected contiguous int32 tensors ({n},) on the mask's device")
        self.mask, self.depth, self.positions, self.n_tokens, self.device = mask, depth, positions, n, mask.device
        self._c = SagePagedTreeMaskC(mask.data_ptr(), words, mask.stride(0), None if depth is None else depth.data_ptr())
        self._ref = ctypes.byref(self._c)


def sage_paged_tree(parents: torch.Tensor, batch: PagedBatch, tree: Optional[PagedTree] = None, *, status: torch.Tensor,
                    window: Optional[int] = None, words: Optional[int] = None, stream=None) -> PagedTree:
    """The tree of each sequence's new tokens from `parents`, int32 [N]: the parent's number among the sequence's new
    tokens, before the token's own, or -1 for one that continues the cached text.  Fills `tree`, or a new one of `words`
    words a row (32 tokens each).  window: that of the attention (ancestors further up are not seen).  status: a block or a
    workspace that records bad indices."""
    n, dev = parents.shape[0] if parents.dim() == 1 else -1, batch.device
    if n < 0 or parents.dtype is not _I32 or parents.device != dev or not parents.is_contiguous():
        raise ValueError("parents: expected a contiguous int32 tensor [N] on the batch's device")
    if tree is None:
        if words is None:
            raise ValueError("words (of 32 tokens each, enough for the longest sequence's new tokens) or tree has to be given")
        with _made_on(stream, dev):
            tree = PagedTree(torch.empty((n, words), dtype=torch.int32, device=dev),
                             *(torch.empty(n, dtype=torch.int32, device=dev) for _ in range(2)))
    elif words is not None:
        raise ValueError("words belongs to a tree that is made here")
    if tree.n_tokens != n or tree.device != dev:
        raise ValueError("tree must have the rows of parents, on the same device")
    if status.device != dev or status.nbytes < 256:
        raise ValueError("status: expected a zeroed block of 256 bytes on the batch's device")
    positions = tree.positions
    _check(_paged_call(dev, stream, lib().sage_paged_tree, (
        batch._ref, n, parents.data_ptr(), window or 0, tree._ref, None if positions is None else positions.data_ptr(),
        status.data_ptr())), "sage_paged_tree")
    return tree


def sage_paged_attn_tree(q: torch.Tensor, cache: PagedKV, batch: PagedBatch, tree: PagedTree,
                         sm_scale: Optional[float] = None, window: Optional[int] = None,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the batch's new tokens q [N, Hq, D], trees of drafted tokens, over the cache: the cached tokens before
    them (with a window, the last `window` before the token's own place) and the new tokens that the tree's mask shows.
    Otherwise as sage_paged_attn."""
    if tree.n_tokens != q.shape[0] or tree.device != cache.device:
        raise ValueError("tree must have q's rows, on the cache's device")
    if window and tree.depth is None:
        raise ValueError("a window needs the tree's depth")
    sm_scale = 1.0 / math.sqrt(cache.head_dim) if sm_scale is None else sm_scale
    return _paged_attn_call(q, cache, batch, (tree._ref, sm_scale, window or 0), out, lse, ws, stream,
                            "sage_paged_attn_tree")


# ------------------------------------------------------------------- the cache's pages (include/sage_paged_pool.h)
class PagedPool(_StatusOwner):
    """The pages of a cache and who holds them: int32 CUDA tensors refs [n_pages] (entries of page tables that hold the
    page; 0: free) and page_table [n_rows, max_pages] (-1: no page), whose rows a PagedBatch may use.  `status` is the block
    that the accounting calls record bad indices in, with their scratch behind it."""

    def __init__(self, refs: torch.Tensor, page_table: torch.Tensor, page_size: int):
        if refs.dim() != 1 or page_table.dim() != 2 or 0 in page_table.shape:
            raise ValueError("expected refs [n_pages] and page_table [n_rows, max_pages]")
        for t in (refs, page_table):
            if t.dtype != torch.int32 or not t.is_cuda or t.device != refs.device:
                raise ValueError("expected int32 CUDA tensors on one device")
        if not refs.is_contiguous() or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("refs must be contiguous, page_table's rows too")
        self.refs, self.page_table, self.page_size = refs, page_table, page_size
        self.n_rows, self.n_pages = page_table.shape[0], refs.numel()
        self._own_status(refs.device, max(256, int(lib().sage_paged_pool_workspace_bytes(self.n_rows, self.n_pages))))
        self._c = SagePagedPoolC(refs.data_ptr(), self.n_pages, page_table.data_ptr(), self.n_rows, page_table.shape[1],
                                 page_table.stride(0), page_size)
        self._ref = ctypes.byref(self._c)


def _int_list(t: Optional[torch.Tensor], n: Optional[int], device, what: str):
    if t is None:
        return None
    if t.dtype is not _I32 or t.dim() != 1 or (n is not None and t.shape[0] != n) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous int32 tensor [{'n' if n is None else n}] on the same device")
    return t.data_ptr()


def sage_paged_release(pool: PagedPool, hi: torch.Tensor, lo: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gives back the pages of each row whose positions all lie outside [lo, hi) (int32 [n_rows]; lo None: 0)."""
    dev, n = pool.device, pool.n_rows
    lo_at, hi_at = _int_list(lo, n, dev, "lo"), _int_list(hi, n, dev, "hi")
    status = pool._status_on(stream)
    _check(_paged_call(dev, stream, lib().sage_paged_release, (pool._ref, lo_at, hi_at, status.data_ptr())),
           "sage_paged_release")


def sage_paged_reserve(pool: PagedPool, hi: torch.Tensor, lo: Optional[torch.Tensor] = None,
                       ok: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gives each row a page for every entry without one among those of its positions [lo, hi) (int32 [n_rows]; lo None:
    0).  Returns ok, int32 [n_rows]: 1 where the row has all of them, 0 where the free pages did not last."""
    dev, n = pool.device, pool.n_rows
    lo_at, hi_at = _int_list(lo, n, dev, "lo"), _int_list(hi, n, dev, "hi")
    if ok is None:
        with _made_on(stream, dev):
            ok = torch.empty(n, dtype=torch.int32, device=dev)
    ok_at, ws = _int_list(ok, n, dev, "ok"), pool._status_on(stream)
    _check(_paged_call(dev, stream, lib().sage_paged_reserve, (pool._ref, lo_at, hi_at, ok_at, ws.data_ptr(), ws.nbytes)),
           "sage_paged_reserve")
    return ok


def sage_paged_fork(pool: PagedPool, src_rows: torch.Tensor, dst_rows: torch.Tensor, n_tokens: torch.Tensor,
                    out: Optional[torch.Tensor] = None, stream=None):
    """Row dst_rows[k], which holds no page, begins like row src_rows[k], n_tokens[k] positions long (int32 [n_forks] each):
    full pages are shared, a page begun gets a free one of the child's own.  Returns (copy_src, copy_dst, copy_tokens,
    ok), int32 [n_forks] each (rows of `out`, int32 [4, n_forks], made here when None): what sage_paged_copy has to copy
    in each layer's cache, and 1 where the child was made."""
    dev = pool.device
    src, dst = _int_list(src_rows, None, dev, "src_rows"), _int_list(dst_rows, src_rows.shape[0], dev, "dst_rows")
    n, tokens = src_rows.shape[0], _int_list(n_tokens, src_rows.shape[0], dev, "n_tokens")
    if out is None:
        with _made_on(stream, dev):
            out = torch.empty((4, n), dtype=torch.int32, device=dev)
    elif out.dtype is not _I32 or tuple(out.shape) != (4, n) or not out.is_contiguous() or out.device != dev:
        raise ValueError(f"out: expected a contiguous int32 tensor [4, {n}] on the pool's device")
    ws, at = pool._status_on(stream), out.data_ptr()
    _check(_paged_call(dev, stream, lib().sage_paged_fork, (
        pool._ref, src, dst, tokens, n, at, at + 4 * n, at + 8 * n, at + 12 * n, ws.data_ptr(), ws.nbytes)),
        "sage_paged_fork")
    return tuple(out.unbind(0))


def sage_paged_copy(cache: PagedKV, src: torch.Tensor, dst: torch.Tensor, n_tokens: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """K and V of the first n_tokens[i] slots (None: all) of page src[i] to page dst[i], int32 [n] each; an entry with a
    -1 is left out.  No page may be the target of two copies, or target and source."""
    dev = cache.device
    s = _int_list(src, None, dev, "src")
    n = src.shape[0]
    d, t = _int_list(dst, n, dev, "dst"), _int_list(n_tokens, n, dev, "n_tokens")
    if status is None:
        status = cache._status_on(stream)
    elif status.device != dev or status.nbytes < 256:
        raise ValueError("status: expected a zeroed block of 256 bytes on the cache's device")
    _check(_paged_call(dev, stream, lib().sage_paged_copy, (cache._ref, s, d, t, n, status.data_ptr())), "sage_paged_copy")


def sage_paged_compact(cache: PagedKV, batch: PagedBatch, first: torch.Tensor, keep: torch.Tensor, n_keep: torch.Tensor,
                       ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """K and V of position keep[b, i] of sequence b to position first[b] + i, for i < n_keep[b], in place: int32 first
    and n_keep [n_seqs], keep [n_seqs, max_keep], positions not before their new ones and below kv_len.  ws: a
    paged_workspace, or its first SAGE_PAGED_WS_HEADER bytes as zeros (made here when None)."""
    dev, n = cache.device, batch.n_seqs
    if batch.device != dev:
        raise ValueError("the batch lies on another device than the cache")
    if keep.dim() != 2 or keep.shape[0] != n or keep.dtype is not _I32 or keep.device != dev \
            or (keep.shape[1] > 1 and keep.stride(1) != 1):
        raise ValueError(f"keep: expected an int32 tensor [{n}, max_keep] with contiguous rows on the cache's device")
    f, k = _int_list(first, n, dev, "first"), _int_list(n_keep, n, dev, "n_keep")
    if ws is None:
        with _made_on(stream, dev):
            ws = torch.zeros(PAGED_WS_HEADER, dtype=torch.uint8, device=dev)
    elif ws.device != dev:
        raise ValueError("ws lies on another device than the cache")
    _check(_paged_call(dev, stream, lib().sage_paged_compact, (
        cache._ref, batch._ref, f, keep.data_ptr(), keep.shape[1], keep.stride(0), k, ws.data_ptr(), ws.nbytes)),
        "sage_paged_compact")
