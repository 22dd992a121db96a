"""ctypes binding of libsparse_mla.so (include/sparse_mla.h).

Argument marshalling only: every step of the computation runs in the CUDA
library. Functions keep the C names. torch supplies device memory and the
current stream; outputs and the workspace are allocated with torch when the
caller passes none (the library itself never allocates).

The library must exist: if it was not built, or fails to load, every call
raises — there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading
from typing import NamedTuple, Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsparse_mla.so")

SMLA_OK = 0
SMLA_ERR_NULL_POINTER = 1
SMLA_ERR_BAD_SHAPE = 2
SMLA_ERR_BAD_DTYPE = 3
SMLA_ERR_MISALIGNED = 4
SMLA_ERR_UNSUPPORTED = 5
SMLA_ERR_WORKSPACE_TOO_SMALL = 6
SMLA_ERR_CUDA = 7

SMLA_KV_BF16 = 0
SMLA_KV_FP8_E4M3 = 1
SMLA_DOT_AUTO = 0
SMLA_DOT_BF16 = 1
SMLA_DOT_FP8 = 2
_DOT = {"auto": SMLA_DOT_AUTO, "bf16": SMLA_DOT_BF16, "fp8": SMLA_DOT_FP8}
SMLA_KERNEL_AUTO = 0
SMLA_KERNEL_WARP_MMA = 1
SMLA_KERNEL_TCGEN05_BASIC = 2
_KERNEL = {"auto": SMLA_KERNEL_AUTO, "mma": SMLA_KERNEL_WARP_MMA, "basic": SMLA_KERNEL_TCGEN05_BASIC}

# every function the header declares, with its ctypes signature
_c = ctypes
SIGNATURES = {
    "smla_status_string": ([_c.c_int], _c.c_char_p),
    "smla_version": ([], _c.c_int),
    "smla_plan_num_splits": ([_c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int], _c.c_int),
    "sparse_mla_fwd_workspace_size": ([_c.c_int] * 7, _c.c_size_t),
    "sparse_mla_fwd": ([_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_void_p,
                        _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int64, _c.c_int,
                        _c.c_float, _c.c_int, _c.c_void_p, _c.c_void_p,
                        _c.c_void_p, _c.c_size_t, _c.c_int, _c.c_void_p], _c.c_int),
    "sparse_mla_fwd_q8": ([_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                           _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int64, _c.c_int, _c.c_float,
                           _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_size_t, _c.c_int, _c.c_void_p], _c.c_int),
    "sparse_mla_fwd_ex": ([_c.c_void_p], _c.c_int),
    "sparse_mla_fwd_ex_workspace_size": ([_c.c_void_p], _c.c_size_t),
    "smla_gather_probe": ([_c.c_void_p, _c.c_int64, _c.c_int, _c.c_void_p, _c.c_int64, _c.c_int, _c.c_int,
                           _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p], _c.c_int),
    "smla_l2_read_probe": ([_c.c_void_p, _c.c_int64, _c.c_int, _c.c_void_p, _c.c_int, _c.c_void_p], _c.c_int),
    "smla_compute_fp8_scale": ([_c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_void_p], _c.c_int),
    "smla_fp8_cache_write": ([_c.c_void_p, _c.c_void_p, _c.c_int64, _c.c_int, _c.c_void_p,
                              _c.c_void_p, _c.c_int64, _c.c_void_p], _c.c_int),
    "smla_validate_indices": ([_c.c_void_p, _c.c_int, _c.c_int, _c.c_int64, _c.c_void_p,
                               _c.c_void_p], _c.c_int),
    "smla_device_error": ([_c.c_void_p, _c.c_int], _c.c_int),
    "smla_fused_qk_rope_cache": ([_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_int64,
                                  _c.c_void_p, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_void_p,
                                  _c.c_void_p, _c.c_int64, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int,
                                  _c.c_int64, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_int,
                                  _c.c_int, _c.c_void_p], _c.c_int),
    "smla_last_error_string": ([], _c.c_char_p),
    "smla_build_block_tables_workspace_size": ([_c.c_int], _c.c_size_t),
    "smla_build_block_tables": ([_c.c_void_p] * 4 + [_c.c_int, _c.c_int, _c.c_void_p, _c.c_int64, _c.c_int,
                                _c.c_void_p, _c.c_int] + [_c.c_void_p] * 6 + [_c.c_int64, _c.c_void_p, _c.c_void_p,
                                _c.c_size_t, _c.c_void_p], _c.c_int),
    "smla_rope_cos_sin_cache": ([_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_int, _c.c_double, _c.c_int, _c.c_double,
                                 _c.c_int64, _c.c_double, _c.c_double, _c.c_double, _c.c_void_p], _c.c_int),
    "smla_rope": ([_c.c_void_p], _c.c_int),
    "smla_kv8_append": ([_c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p, _c.c_int64, _c.c_int64, _c.c_void_p,
                         _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                         _c.c_int64, _c.c_void_p], _c.c_int),
    "smla_kv8_attn_workspace_size": ([_c.c_int] * 6, _c.c_size_t),
    "smla_kv8_attn_workspace_size_of": ([_c.c_void_p], _c.c_size_t),
    "smla_kv8_attn_fwd": ([_c.c_void_p], _c.c_int),
    "sparse_mla_fwd_no_alloc": ([_c.c_void_p, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_void_p,
                                 _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int64, _c.c_int,
                                 _c.c_float, _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_int,
                                 _c.c_void_p], _c.c_int),
}


SMLA_BF16 = 0
SMLA_F16 = 1
SMLA_F32 = 2
_DTYPE = {torch.bfloat16: SMLA_BF16, torch.float16: SMLA_F16, torch.float32: SMLA_F32}
SMLA_ROPE_NONE = 0
SMLA_ROPE_LINEAR = 1
SMLA_ROPE_NTK = 2
SMLA_ROPE_YARN = 3
_ROPE = {"none": SMLA_ROPE_NONE, "linear": SMLA_ROPE_LINEAR, "ntk": SMLA_ROPE_NTK, "yarn": SMLA_ROPE_YARN}


class SmlaFwdParams(ctypes.Structure):
    """smla_fwd_params of include/sparse_mla.h."""
    _fields_ = [("size", _c.c_size_t), ("q", _c.c_void_p), ("q_scale", _c.c_void_p),
                ("kv_cache", _c.c_void_p), ("kv_dtype", _c.c_int), ("kv_scale", _c.c_void_p),
                ("indices", _c.c_void_p), ("T", _c.c_int), ("H", _c.c_int), ("D_qk", _c.c_int), ("D_v", _c.c_int),
                ("num_slots", _c.c_int64), ("topk", _c.c_int), ("scale", _c.c_float), ("dot_precision", _c.c_int),
                ("sinks", _c.c_void_p), ("out", _c.c_void_p), ("lse", _c.c_void_p), ("workspace", _c.c_void_p),
                ("workspace_bytes", _c.c_size_t), ("num_splits", _c.c_int), ("stream", _c.c_void_p),
                ("kernel", _c.c_int)]


class SmlaRopeParams(ctypes.Structure):
    """smla_rope_params of include/sparse_mla.h."""
    _fields_ = [("size", _c.c_size_t), ("dtype", _c.c_int), ("q", _c.c_void_p), ("q_stride_t", _c.c_int64),
                ("q_stride_h", _c.c_int64), ("q_out", _c.c_void_p), ("q_out_stride_t", _c.c_int64),
                ("q_out_stride_h", _c.c_int64), ("k", _c.c_void_p), ("k_stride_t", _c.c_int64),
                ("k_stride_h", _c.c_int64), ("k_out", _c.c_void_p), ("k_out_stride_t", _c.c_int64),
                ("k_out_stride_h", _c.c_int64), ("positions", _c.c_void_p), ("cos_sin_cache", _c.c_void_p),
                ("max_position", _c.c_int64), ("T", _c.c_int), ("H", _c.c_int), ("H_k", _c.c_int), ("D", _c.c_int),
                ("rot_dim", _c.c_int), ("rot_offset", _c.c_int), ("is_neox", _c.c_int), ("inverse", _c.c_int),
                ("stream", _c.c_void_p)]


class SmlaKv8AttnParams(ctypes.Structure):
    """smla_kv8_attn_params of include/sparse_mla.h."""
    _fields_ = [("size", _c.c_size_t), ("q", _c.c_void_p), ("q_stride_t", _c.c_int64), ("q_stride_h", _c.c_int64),
                ("k_cache", _c.c_void_p), ("v_cache", _c.c_void_p), ("k_scale", _c.c_void_p),
                ("v_scale", _c.c_void_p), ("num_blocks", _c.c_int64), ("block_table", _c.c_void_p),
                ("table_stride", _c.c_int64), ("table_width", _c.c_int), ("seq_lens", _c.c_void_p),
                ("query_start", _c.c_void_p), ("B", _c.c_int), ("T", _c.c_int), ("H", _c.c_int), ("H_kv", _c.c_int),
                ("D", _c.c_int), ("block_size", _c.c_int), ("max_query_len", _c.c_int), ("window", _c.c_int),
                ("scale", _c.c_float), ("sinks", _c.c_void_p), ("out", _c.c_void_p), ("lse", _c.c_void_p),
                ("workspace", _c.c_void_p), ("workspace_bytes", _c.c_size_t), ("stream", _c.c_void_p)]


_lock = threading.Lock()
_lib = None


class SmlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s: %s" % (where, status_string(status))
        if status == SMLA_ERR_CUDA:
            msg += " (%s)" % lib().smla_last_error_string().decode()
        super().__init__(msg)


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it is missing: build it first)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libsparse_mla.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
        return _lib


def status_string(status: int) -> str:
    return lib().smla_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != SMLA_OK:
        raise SmlaError(status, where)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(x: Optional[torch.Tensor]) -> Optional[int]:
    return None if x is None else x.data_ptr()


def _need(x: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if x.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, x.dtype))
    if x.dim() != ndim:
        raise ValueError("%s must have %d dims, got shape %s" % (name, ndim, tuple(x.shape)))
    if not x.is_contiguous():
        raise ValueError("%s must be contiguous (strided inputs are not accepted)" % name)
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)


def smla_device_error(reset: bool = False) -> int:
    """Error word of the device-side bounded waits (0 = none); synchronous."""
    v = ctypes.c_int(0)
    _check(lib().smla_device_error(ctypes.byref(v), int(reset)), "smla_device_error")
    return int(v.value)


def smla_version() -> int:
    return int(lib().smla_version())


def smla_plan_num_splits(T: int, H: int, D_qk: int, topk: int, kv_dtype: int, sm_count: int) -> int:
    return int(lib().smla_plan_num_splits(T, H, D_qk, topk, kv_dtype, sm_count))


def sparse_mla_fwd_workspace_size(T: int, H: int, D_qk: int, D_v: int, topk: int, kv_dtype: int,
                                  num_splits: int = 0) -> int:
    n = lib().sparse_mla_fwd_workspace_size(T, H, D_qk, D_v, topk, kv_dtype, num_splits)
    if n == ctypes.c_size_t(-1).value:
        raise SmlaError(SMLA_ERR_BAD_SHAPE, "sparse_mla_fwd_workspace_size")
    return int(n)


# zeroed workspaces, one per (device, stream); the kernel leaves them zeroed
_workspaces = {}


def workspace_for(nbytes: int, device: torch.device, stream_handle: int) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    key = (device.index, stream_handle)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def sparse_mla_fwd(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor, scale: float, *,
                   kv_scale: Optional[torch.Tensor] = None, dot_precision: str = "auto",
                   D_v: int = 512, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   return_lse: bool = True, workspace: Optional[torch.Tensor] = None,
                   num_splits: int = 0, stream=None,
                   sinks: Optional[torch.Tensor] = None,
                   kernel: str = "auto") -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """out[T,H,D_v] (bf16), lse[T,H] (fp32) of the sparse MLA forward
    (sinks: optional fp32 [H] per-head sink logits; kernel: "auto", "mma" for
    the warp-MMA kernel, or "basic" for the tcgen05 kernels that take a
    whole SM per CTA).

    q bf16 [T,H,D_qk]; kv_cache [num_slots, D_qk] bf16 or torch.float8_e4m3fn/uint8
    (E4M3 codes, then kv_scale: fp32 device scalar); indices int32 [T, topk].
    """
    _need(q, "q", torch.bfloat16, 3)
    T, H, D_qk = q.shape
    if kv_cache.dtype == torch.bfloat16:
        kv_dtype = SMLA_KV_BF16
    elif kv_cache.dtype in (torch.float8_e4m3fn, torch.uint8):
        kv_dtype = SMLA_KV_FP8_E4M3
    else:
        raise TypeError("kv_cache must be bf16 or E4M3 (float8_e4m3fn / uint8), got %s" % kv_cache.dtype)
    _need(kv_cache, "kv_cache", kv_cache.dtype, 2)
    if kv_cache.shape[1] != D_qk:
        raise ValueError("kv_cache row width %d != D_qk %d" % (kv_cache.shape[1], D_qk))
    _need(indices, "indices", torch.int32, 2)
    if indices.shape[0] != T:
        raise ValueError("indices has %d rows, q has %d" % (indices.shape[0], T))
    if kv_dtype == SMLA_KV_FP8_E4M3:
        if kv_scale is None:
            raise ValueError("an fp8 cache needs kv_scale (fp32 device scalar)")
        _need(kv_scale.reshape(1), "kv_scale", torch.float32, 1)
    if dot_precision not in _DOT:
        raise ValueError("dot_precision must be one of %s" % sorted(_DOT))
    if kernel not in _KERNEL:
        raise ValueError("kernel must be one of %s" % sorted(_KERNEL))
    topk = indices.shape[1]
    if out is None:
        out = torch.empty((T, H, D_v), dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, 3)
    if lse is None and return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    sh = _stream(stream)
    need = sparse_mla_fwd_workspace_size(T, H, D_qk, D_v, topk, kv_dtype, num_splits)
    if workspace is None:
        workspace = workspace_for(need, q.device, sh)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if sinks is None and kernel == "auto":
        st = lib().sparse_mla_fwd(
            _ptr(q), _ptr(kv_cache), kv_dtype, _ptr(kv_scale), _ptr(indices),
            T, H, D_qk, D_v, kv_cache.shape[0], topk, float(scale), _DOT[dot_precision],
            _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, int(num_splits), sh)
        _check(st, "sparse_mla_fwd")
    else:
        if sinks is not None:
            _need(sinks, "sinks", torch.float32, 1)
            if sinks.shape[0] != H:
                raise ValueError("sinks must be [H]")
        _fwd_ex(q, None, kv_cache, kv_dtype, kv_scale, indices, T, H, D_qk, D_v, topk, scale,
                _DOT[dot_precision], sinks, out, lse, workspace, ws_bytes, num_splits, sh, _KERNEL[kernel])
    return out, lse


def _fwd_ex(q, q_scale, kv_cache, kv_dtype, kv_scale, indices, T, H, D_qk, D_v, topk, scale, dot, sinks,
            out, lse, workspace, ws_bytes, num_splits, sh, kernel=SMLA_KERNEL_AUTO):
    p = SmlaFwdParams(ctypes.sizeof(SmlaFwdParams), _ptr(q), _ptr(q_scale), _ptr(kv_cache), kv_dtype,
                      _ptr(kv_scale), _ptr(indices), T, H, D_qk, D_v, kv_cache.shape[0], topk, float(scale), dot,
                      _ptr(sinks), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, int(num_splits), sh,
                      int(kernel))
    _check(lib().sparse_mla_fwd_ex(ctypes.byref(p)), "sparse_mla_fwd_ex")


def sparse_mla_fwd_q8(q8: torch.Tensor, q_scale: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                      scale: float, *, kv_scale: torch.Tensor, D_v: int = 512, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                      workspace: Optional[torch.Tensor] = None, num_splits: int = 0,
                      stream=None, sinks: Optional[torch.Tensor] = None,
                      kernel: str = "auto") -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The forward with a pre-quantized q: q8 E4M3 codes [T, H, D_qk] (uint8 or
    float8_e4m3fn) and q_scale, its per-tensor fp32 device scalar; an E4M3 cache
    with kv_scale; fp8 dots."""
    if q8.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("q8 must be E4M3 codes (uint8 / float8_e4m3fn), got %s" % q8.dtype)
    _need(q8, "q8", q8.dtype, 3)
    T, H, D_qk = q8.shape
    if kv_cache.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError("kv_cache must be E4M3 (float8_e4m3fn / uint8), got %s" % kv_cache.dtype)
    _need(kv_cache, "kv_cache", kv_cache.dtype, 2)
    if kv_cache.shape[1] != D_qk:
        raise ValueError("kv_cache row width %d != D_qk %d" % (kv_cache.shape[1], D_qk))
    _need(indices, "indices", torch.int32, 2)
    if indices.shape[0] != T:
        raise ValueError("indices has %d rows, q8 has %d" % (indices.shape[0], T))
    _need(q_scale.reshape(1), "q_scale", torch.float32, 1)
    _need(kv_scale.reshape(1), "kv_scale", torch.float32, 1)
    topk = indices.shape[1]
    if out is None:
        out = torch.empty((T, H, D_v), dtype=torch.bfloat16, device=q8.device)
    _need(out, "out", torch.bfloat16, 3)
    if lse is None and return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q8.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    sh = _stream(stream)
    need = sparse_mla_fwd_workspace_size(T, H, D_qk, D_v, topk, SMLA_KV_FP8_E4M3, num_splits)
    if workspace is None:
        workspace = workspace_for(need, q8.device, sh)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if kernel not in _KERNEL:
        raise ValueError("kernel must be one of %s" % sorted(_KERNEL))
    if sinks is None and kernel == "auto":
        st = lib().sparse_mla_fwd_q8(
            _ptr(q8), _ptr(q_scale), _ptr(kv_cache), _ptr(kv_scale), _ptr(indices),
            T, H, D_qk, D_v, kv_cache.shape[0], topk, float(scale),
            _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, int(num_splits), sh)
        _check(st, "sparse_mla_fwd_q8")
    else:
        if sinks is not None:
            _need(sinks, "sinks", torch.float32, 1)
            if sinks.shape[0] != H:
                raise ValueError("sinks must be [H]")
        _fwd_ex(q8, q_scale, kv_cache, SMLA_KV_FP8_E4M3, kv_scale, indices, T, H, D_qk, D_v, topk, scale,
                SMLA_DOT_FP8, sinks, out, lse, workspace, ws_bytes, num_splits, sh, _KERNEL[kernel])
    return out, lse


def smla_gather_probe(pool: torch.Tensor, indices: torch.Tensor, *, ctas_per_sm: int = 1, stages: int = 1,
                      hold_ns: int = 0, pair_mode: int = 0, issue_warps: int = 0, copy_mode: int = 0,
                      checksum: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The pure indexed-row copy probe: rows `indices` (int32, any shape,
    taken flat) of `pool` [num_rows, row_bytes] (any 1- or 2-byte dtype)
    gathered into shared memory (copy_mode 0: TMA gather4, 1: 16-byte cp.async)
    and folded into per-CTA checksums (uint32 device tensor
    [sm_count * ctas_per_sm], returned); pair_mode 1 / 2: CTA pairs sharing
    each tile by cluster multicast / by a bulk copy into the peer;
    issue_warps > 0: a tile's copies spread evenly over that many producer
    warps."""
    if pool.dim() != 2 or not pool.is_contiguous() or not pool.is_cuda:
        raise ValueError("pool must be a contiguous CUDA tensor [num_rows, row]")
    _need(indices.reshape(-1), "indices", torch.int32, 1)
    row_bytes = pool.shape[1] * pool.element_size()
    sms = torch.cuda.get_device_properties(pool.device).multi_processor_count
    if checksum is None:
        checksum = torch.zeros(sms * ctas_per_sm, dtype=torch.int32, device=pool.device)
    _check(lib().smla_gather_probe(_ptr(pool), pool.shape[0], row_bytes, _ptr(indices), indices.numel(),
                                   int(ctas_per_sm), int(stages), int(hold_ns), int(pair_mode), int(issue_warps),
                                   int(copy_mode), _ptr(checksum),
                                   _stream(stream)),
           "smla_gather_probe")
    return checksum


def smla_l2_read_probe(buf: torch.Tensor, reps: int, blocks: int, checksum: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Stream `buf` (contiguous CUDA tensor) `reps` times from `blocks` blocks."""
    if not buf.is_contiguous() or not buf.is_cuda:
        raise ValueError("buf must be a contiguous CUDA tensor")
    if checksum is None:
        checksum = torch.zeros(blocks, dtype=torch.int32, device=buf.device)
    nbytes = buf.numel() * buf.element_size()
    _check(lib().smla_l2_read_probe(_ptr(buf), nbytes - nbytes % 16, int(reps), _ptr(checksum), int(blocks),
                                    _stream(stream)), "smla_l2_read_probe")
    return checksum


def sparse_mla_fwd_ex_workspace_size(T: int, H: int, D_qk: int, D_v: int, topk: int, kv_dtype: int, *,
                                     dot_precision: str = "auto", q8: bool = False, num_splits: int = 0,
                                     kernel: str = "auto") -> int:
    """Exact workspace bytes of one call (its dot precision, q form, kernel and splits)."""
    p = SmlaFwdParams(ctypes.sizeof(SmlaFwdParams), None, 1 if q8 else None, None, kv_dtype, None, None,
                      T, H, D_qk, D_v, 0, topk, 1.0, _DOT[dot_precision], None, None, None, None, 0,
                      int(num_splits), None, _KERNEL[kernel])
    n = lib().sparse_mla_fwd_ex_workspace_size(ctypes.byref(p))
    if n == ctypes.c_size_t(-1).value:
        raise SmlaError(SMLA_ERR_BAD_SHAPE, "sparse_mla_fwd_ex_workspace_size")
    return int(n)


def smla_compute_fp8_scale(x: torch.Tensor, scale_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fp32 device scalar amax(|x|)/448 of a bf16 tensor."""
    if x.dtype != torch.bfloat16 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError("x must be a contiguous CUDA bf16 tensor")
    if scale_out is None:
        scale_out = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().smla_compute_fp8_scale(_ptr(x), x.numel(), _ptr(scale_out), _stream(stream)),
           "smla_compute_fp8_scale")
    return scale_out


def smla_fp8_cache_write(src: torch.Tensor, slot_mapping: torch.Tensor, kv_scale: torch.Tensor,
                         kv_cache: torch.Tensor, stream=None) -> torch.Tensor:
    """kv_cache[slot_mapping[n]] = E4M3(src[n] / kv_scale) (uint8 / float8_e4m3fn cache)."""
    _need(src, "src", torch.bfloat16, 2)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(kv_cache, "kv_cache", kv_cache.dtype, 2)
    if kv_cache.element_size() != 1 or kv_cache.shape[1] != src.shape[1]:
        raise ValueError("kv_cache must be 1-byte [num_slots, D]")
    N, D = src.shape
    _check(lib().smla_fp8_cache_write(_ptr(src), _ptr(slot_mapping), N, D, _ptr(kv_scale),
                                      _ptr(kv_cache), kv_cache.shape[0], _stream(stream)),
           "smla_fp8_cache_write")
    return kv_cache


def smla_validate_indices(indices: torch.Tensor, num_slots: int, bad_count: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """int32 device scalar: entries of indices that are neither -1 nor in [0, num_slots)."""
    _need(indices, "indices", torch.int32, 2)
    if bad_count is None:
        bad_count = torch.empty(1, dtype=torch.int32, device=indices.device)
    T, topk = indices.shape
    _check(lib().smla_validate_indices(_ptr(indices), T, topk, int(num_slots), _ptr(bad_count), _stream(stream)),
           "smla_validate_indices")
    return bad_count


def _strided(x: torch.Tensor, name: str, ndim: int):
    """A bf16 CUDA tensor whose last dimension is contiguous (other strides free)."""
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or not x.is_cuda:
        raise TypeError("%s must be a CUDA bf16 tensor" % name)
    if x.dim() != ndim:
        raise ValueError("%s must have %d dims, got shape %s" % (name, ndim, tuple(x.shape)))
    if x.stride(-1) != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)


def smla_fused_qk_rope_cache(ql_nope: torch.Tensor, q_pe: torch.Tensor, kv_c: torch.Tensor, k_pe: torch.Tensor,
                             positions: torch.Tensor, cos_sin_cache: torch.Tensor, slot_mapping: torch.Tensor,
                             kv_cache: torch.Tensor, *, is_neox: bool = True, kv_scale: Optional[torch.Tensor] = None,
                             q_out: Optional[torch.Tensor] = None, q_out_fp8: bool = False,
                             q_scale: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The fused producer step: q_out = concat(ql_nope, RoPE(q_pe)) (bf16, or E4M3
    codes of / q_scale) and kv_cache[slot_mapping[t]] = concat(kv_c, RoPE(k_pe))
    (bf16 cache, or a 1-byte E4M3 cache with kv_scale). ql_nope [T, H, 512] and
    q_pe [T, H, 64] may be strided (last dimension contiguous), as may kv_c
    [T, 512] and k_pe [T, 64]. Returns q_out [T, H, 576]."""
    _strided(ql_nope, "ql_nope", 3)
    _strided(q_pe, "q_pe", 3)
    _strided(kv_c, "kv_c", 2)
    _strided(k_pe, "k_pe", 2)
    T, H, Dn = ql_nope.shape
    if Dn != 512 or tuple(q_pe.shape) != (T, H, 64) or tuple(kv_c.shape) != (T, 512) or tuple(k_pe.shape) != (T, 64):
        raise ValueError("expected ql_nope [T, H, 512], q_pe [T, H, 64], kv_c [T, 512], k_pe [T, 64]")
    _need(positions, "positions", torch.int64, 1)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(cos_sin_cache, "cos_sin_cache", torch.float32, 2)
    if positions.shape[0] != T or slot_mapping.shape[0] != T or cos_sin_cache.shape[1] != 64:
        raise ValueError("positions and slot_mapping must be [T]; cos_sin_cache [max_position, 64]")
    _need(kv_cache, "kv_cache", kv_cache.dtype, 2)
    if kv_cache.shape[1] != 576:
        raise ValueError("kv_cache must be [num_slots, 576]")
    if kv_cache.element_size() == 1:
        kv_dtype = SMLA_KV_FP8_E4M3
        if kv_scale is None:
            raise ValueError("an E4M3 cache needs kv_scale")
    elif kv_cache.dtype == torch.bfloat16:
        kv_dtype = SMLA_KV_BF16
    else:
        raise TypeError("kv_cache must be bf16 or a 1-byte E4M3 cache")
    if q_out is None:
        q_out = torch.empty((T, H, 576), dtype=torch.uint8 if q_out_fp8 else torch.bfloat16, device=ql_nope.device)
    _need(q_out, "q_out", q_out.dtype, 3)
    if (q_out.element_size() == 1) != bool(q_out_fp8) or tuple(q_out.shape) != (T, H, 576):
        raise ValueError("q_out must be [T, H, 576], 1-byte when q_out_fp8 else bf16")
    if q_out_fp8 and q_scale is None:
        raise ValueError("E4M3 q_out needs q_scale")
    _check(lib().smla_fused_qk_rope_cache(
        _ptr(ql_nope), ql_nope.stride(0), ql_nope.stride(1), _ptr(q_pe), q_pe.stride(0), q_pe.stride(1),
        _ptr(kv_c), kv_c.stride(0), _ptr(k_pe), k_pe.stride(0), _ptr(positions), _ptr(cos_sin_cache),
        cos_sin_cache.shape[0], 1 if is_neox else 0, _ptr(slot_mapping), _ptr(kv_cache), kv_dtype,
        kv_cache.shape[0], _ptr(kv_scale), _ptr(q_out), SMLA_KV_FP8_E4M3 if q_out_fp8 else SMLA_KV_BF16,
        _ptr(q_scale), T, H, _stream(stream)), "smla_fused_qk_rope_cache")
    return q_out


def build_fp8_cache(kv_source: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Quantize a whole bf16 pool [num_slots, D] into a fresh E4M3 cache with its scale."""
    scale = smla_compute_fp8_scale(kv_source, stream=stream)
    cache = torch.empty(kv_source.shape, dtype=torch.uint8, device=kv_source.device)
    slots = torch.arange(kv_source.shape[0], dtype=torch.int64, device=kv_source.device)
    smla_fp8_cache_write(kv_source, slots, scale, cache, stream=stream)
    return cache, scale


# ---- the serving step around the forward: page maps, rotary positions, the block-scaled 8-bit cache


class _Launch:
    """Runs a call on the tensors' device and on its stream, with that stream
    current, so that what the call allocates belongs to it. `handle` is the
    stream's handle."""

    __slots__ = ("handle", "_device", "_stream")

    def __init__(self, device: torch.device, stream):
        self._device = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)
        self._stream = None
        self.handle = None
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self._stream = torch.cuda.stream(stream)
            self.handle = int(stream.cuda_stream)

    def __enter__(self):
        if self._device is not None:
            self._device.__enter__()
        if self._stream is not None:
            self._stream.__enter__()
        else:
            self.handle = int(torch.cuda.current_stream().cuda_stream)
        return self.handle

    def __exit__(self, *exc):
        if self._stream is not None:
            self._stream.__exit__(*exc)
        if self._device is not None:
            self._device.__exit__(*exc)


class _Here:
    """As _Launch for the usual call: the tensors are on the current device and no
    stream is given. One for each device, kept: such a call costs a few
    microseconds in all."""

    __slots__ = ("_index",)

    def __init__(self, index: int):
        self._index = index

    def __enter__(self):
        return _raw_stream(self._index)

    def __exit__(self, *exc):
        return None


def _raw_stream(index: int) -> int:
    return int(torch.cuda.current_stream(index).cuda_stream)


if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _raw_stream = torch._C._cuda_getCurrentRawStream
_here = {}


def _on(device: torch.device, stream):
    if stream is not None or device.index != torch.cuda.current_device():
        return _Launch(device, stream)
    on = _here.get(device.index)
    if on is None:
        on = _here[device.index] = _Here(device.index)
    return on


def _fits(x, name: str, dtype, ndim: int, device: torch.device):
    """_need, and on `device`."""
    if not (isinstance(x, torch.Tensor) and x.dtype is dtype and x.dim() == ndim and x.device == device
            and x.is_contiguous()):
        _need(x, name, dtype, ndim)
        raise ValueError("%s is on %s, the other tensors on %s" % (name, x.device, device))


def _rows(x: torch.Tensor, name: str, dtype, ndim: int, device: Optional[torch.device] = None):
    """A CUDA tensor whose last dimension is contiguous (other strides free)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if x.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, x.dtype))
    if x.dim() != ndim:
        raise ValueError("%s must have %d dims, got shape %s" % (name, ndim, tuple(x.shape)))
    if x.stride(-1) != 1 and x.shape[-1] > 1 and x.numel() > 0:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and x.device != device:
        raise ValueError("%s is on %s, the other tensors on %s" % (name, x.device, device))


def _out(x: Optional[torch.Tensor], name: str, shape, dtype, device) -> torch.Tensor:
    if x is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _fits(x, name, dtype, len(shape), device)
    if x.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(x.shape)))
    return x


def _workspace(x: Optional[torch.Tensor], need: int, device: torch.device):
    """The caller's workspace, or one of the current stream's pool (so that calls in
    flight and captured graphs never share one), and its size."""
    if x is None:
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if not x.is_contiguous() or x.device != device:
        raise ValueError("workspace must be contiguous and on %s" % device)
    return x, x.numel() * x.element_size()


class BlockTables(NamedTuple):
    """What smla_build_block_tables returns (device tensors)."""
    query_start: torch.Tensor    # int32 [B + 1]
    positions: torch.Tensor      # int64 [num_tokens]
    slot_mapping: torch.Tensor   # int64 [num_tokens], -1 past the last token
    token_request: torch.Tensor  # int32 [num_tokens], -1 past the last token
    counts: torch.Tensor         # int32 [4]: tokens, blocks taken, blocks given back, blocks lacking
    blocks_held: torch.Tensor    # int32 [B]
    ring_state: torch.Tensor     # int32 [2]: head, count


def smla_build_block_tables(seq_lens: torch.Tensor, query_lens: torch.Tensor, blocks_held: torch.Tensor,
                            block_table: torch.Tensor, free_ring: torch.Tensor, ring_state: torch.Tensor, *,
                            block_size: int, num_tokens: Optional[int] = None,
                            blocks_held_out: Optional[torch.Tensor] = None,
                            ring_state_out: Optional[torch.Tensor] = None, query_start: Optional[torch.Tensor] = None,
                            positions: Optional[torch.Tensor] = None, slot_mapping: Optional[torch.Tensor] = None,
                            token_request: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> BlockTables:
    """Block tables and slot maps of one step from the requests' lengths, all on
    the device (include/sparse_mla.h). seq_lens, query_lens, blocks_held int32
    [B]; block_table int32 [B, width] (rows may be strided; its new entries are
    written); free_ring int32, at least as long as the pool, and ring_state
    int32 [2] = (head, count). blocks_held and ring_state are updated in place
    unless *_out is given. num_tokens: entries of the token maps (taken from
    positions when that is given; needed otherwise), those past the last token
    padded. Nothing is taken when blocks lack: counts[3] says how many."""
    _need(seq_lens, "seq_lens", torch.int32, 1)
    dev = seq_lens.device
    B = seq_lens.shape[0]
    _fits(query_lens, "query_lens", torch.int32, 1, dev)
    _fits(blocks_held, "blocks_held", torch.int32, 1, dev)
    if query_lens.shape[0] != B or blocks_held.shape[0] != B:
        raise ValueError("query_lens and blocks_held must be [B] = [%d]" % B)
    _rows(block_table, "block_table", torch.int32, 2, dev)
    rows, width = block_table.shape
    if rows != B:
        raise ValueError("block_table has %d rows, seq_lens %d" % (rows, B))
    row_stride = block_table.stride(0)
    if row_stride < width:
        if B > 1:
            raise ValueError("block_table rows overlap")
        row_stride = width
    _fits(free_ring, "free_ring", torch.int32, 1, dev)
    _fits(ring_state, "ring_state", torch.int32, 1, dev)
    if ring_state.shape[0] != 2:
        raise ValueError("ring_state must be [2]: head, count")
    if num_tokens is None:
        if positions is None:
            raise ValueError("num_tokens or positions is needed")
        num_tokens = positions.shape[0]
    L = _lib or lib()
    with _on(dev, stream) as handle:
        held = blocks_held if blocks_held_out is None else _out(blocks_held_out, "blocks_held_out", (B,), torch.int32, dev)
        state = ring_state if ring_state_out is None else _out(ring_state_out, "ring_state_out", (2,), torch.int32, dev)
        need = _tables_workspace(B)
        if (query_start is None and positions is None and slot_mapping is None and token_request is None
                and counts is None and workspace is None):
            # two allocations for all (each is as dear as the kernel's launch); the workspace first, for its alignment
            positions, slot_mapping = torch.empty((2, num_tokens), dtype=torch.int64, device=dev).unbind(0)
            ints = need // 4
            workspace, counts, query_start, token_request = torch.empty(
                ints + 5 + B + num_tokens, dtype=torch.int32, device=dev).split_with_sizes((ints, 4, B + 1, num_tokens))
            ws_bytes = need
        else:
            query_start = _out(query_start, "query_start", (B + 1,), torch.int32, dev)
            positions = _out(positions, "positions", (num_tokens,), torch.int64, dev)
            slot_mapping = _out(slot_mapping, "slot_mapping", (num_tokens,), torch.int64, dev)
            token_request = _out(token_request, "token_request", (num_tokens,), torch.int32, dev)
            counts = _out(counts, "counts", (4,), torch.int32, dev)
            workspace, ws_bytes = _workspace(workspace, need, dev)
        st = L.smla_build_block_tables(
            seq_lens.data_ptr(), query_lens.data_ptr(), blocks_held.data_ptr(), held.data_ptr(), B, block_size,
            block_table.data_ptr(), row_stride, width, free_ring.data_ptr(), free_ring.shape[0], ring_state.data_ptr(),
            state.data_ptr(), query_start.data_ptr(), positions.data_ptr(), slot_mapping.data_ptr(),
            token_request.data_ptr(), num_tokens, counts.data_ptr(), workspace.data_ptr(), ws_bytes, handle)
    if st:
        _check(st, "smla_build_block_tables")
    return BlockTables(query_start, positions, slot_mapping, token_request, counts, held, state)


# Workspace bytes of recent sizes: a call to the library for each costs more than the rest of the binding's checks,
# but a server's sizes have no end.
@functools.lru_cache(maxsize=1024)
def _tables_workspace(B: int) -> int:
    return int((_lib or lib()).smla_build_block_tables_workspace_size(B))


@functools.lru_cache(maxsize=1024)
def _kv8_attn_workspace(device: int, B: int, T: int, H: int, H_kv: int, D: int, max_query_len: int, width: int,
                        block_size: int) -> int:
    """For `device`, which is the current one (its SM count decides). Raises where the library has no answer, which
    is not kept: a device query may have failed in passing."""
    need = (_lib or lib()).smla_kv8_attn_workspace_size_of(_KV8_ATTN_PARAMS.pack(
        _KV8_ATTN_PARAMS.size, *([0] * 10), width, 0, 0, B, T, H, H_kv, D, block_size, max_query_len, 0, 0.0, 0, 0, 0, 0,
        0, 0))
    if need == ctypes.c_size_t(-1).value:
        raise SmlaError(SMLA_ERR_BAD_SHAPE, "smla_kv8_attn_workspace_size_of")
    return int(need)


def smla_rope_cos_sin_cache(num_positions: int, rot_dim: int, *, base: float = 10000.0, scaling: str = "none",
                            factor: float = 1.0, original_max_position: int = 0, beta_fast: float = 32.0,
                            beta_slow: float = 1.0, attention_factor: Optional[float] = None, first_position: int = 0,
                            out: Optional[torch.Tensor] = None, device=None, stream=None) -> torch.Tensor:
    """The rotary table [num_positions, rot_dim] (fp32: rot_dim / 2 cosines, then
    as many sines) that smla_rope and smla_fused_qk_rope_cache (rot_dim 64) read.
    scaling: "none", "linear", "ntk" or "yarn" (which needs
    original_max_position); attention_factor multiplies the values (None: the
    scaling's own)."""
    if scaling not in _ROPE:
        raise ValueError("scaling must be one of %s" % sorted(_ROPE))
    if attention_factor is not None and not attention_factor > 0:
        raise ValueError("attention_factor must be positive")
    if out is not None:
        _need(out, "out", torch.float32, 2)
        if tuple(out.shape) != (num_positions, rot_dim):
            raise ValueError("out must have shape %s, got %s" % ((num_positions, rot_dim), tuple(out.shape)))
        dev = out.device
    else:
        dev = torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError("device must be a CUDA device")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
    L = _lib or lib()
    with _on(dev, stream) as handle:
        if out is None:
            out = torch.empty((num_positions, rot_dim), dtype=torch.float32, device=dev)
        st = L.smla_rope_cos_sin_cache(out.data_ptr(), num_positions, first_position, rot_dim, base, _ROPE[scaling],
                                       factor, original_max_position, beta_fast, beta_slow, attention_factor or 0.0,
                                       handle)
    if st:
        _check(st, "smla_rope_cos_sin_cache")
    return out


_LETTERS = {_c.c_size_t: "N", _c.c_int: "i", _c.c_int64: "q", _c.c_float: "f", _c.c_void_p: "P"}


def _packed(structure) -> struct.Struct:
    """A C structure packed in one call (native sizes and alignment) instead of built field by field."""
    packed = struct.Struct("@" + "".join(_LETTERS[t] for _, t in structure._fields_))
    assert packed.size == ctypes.sizeof(structure)
    return packed


_ROPE_PARAMS = _packed(SmlaRopeParams)
_KV8_ATTN_PARAMS = _packed(SmlaKv8AttnParams)


def smla_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, cos_sin_cache: torch.Tensor, *,
              rot_offset: int = 0, is_neox: bool = True, inverse: bool = False, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None,
              stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotary positions on columns [rot_offset, rot_offset + rot_dim) of each head
    of q [T, H, D] and k [T, H_k, D] (or None), rot_dim being cos_sin_cache's
    width; the other columns are copied. bf16, fp16 or fp32; rows may be strided.
    Halves (is_neox) or interleaved pairs; inverse turns back (the forward
    rotation's gradient). q_out / k_out may be q / k: rotated in place."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPE:
        raise TypeError("q must be a bf16, fp16 or fp32 tensor")
    dtype, dev = q.dtype, q.device
    _rows(q, "q", dtype, 3)
    T, H, D = q.shape
    if k is not None:
        _rows(k, "k", dtype, 3, dev)
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError("k must be [T, H_k, D] = [%d, *, %d], got %s" % (T, D, tuple(k.shape)))
    elif k_out is not None:
        raise ValueError("k_out without k")
    _fits(positions, "positions", torch.int64, 1, dev)
    if positions.shape[0] != T:
        raise ValueError("positions must be [T] = [%d]" % T)
    _fits(cos_sin_cache, "cos_sin_cache", torch.float32, 2, dev)
    for name, x, like in (("q_out", q_out, q), ("k_out", k_out, k)):
        if x is not None and x is not like:
            _rows(x, name, dtype, 3, dev)
            if x.shape != like.shape:
                raise ValueError("%s must have shape %s, got %s" % (name, tuple(like.shape), tuple(x.shape)))
    L = _lib or lib()
    with _on(dev, stream) as handle:
        if q_out is None:
            q_out = torch.empty((T, H, D), dtype=dtype, device=dev)
        qs, os = q.stride(), q_out.stride()
        if k is None:
            ks = (0, 0, 0, 0, 0, 0)
            Hk = 0
        else:
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=dtype, device=dev)
            Hk = k.shape[1]
            a, b = k.stride(), k_out.stride()
            ks = (k.data_ptr(), a[0], a[1], k_out.data_ptr(), b[0], b[1])
        P, rot = cos_sin_cache.shape
        st = L.smla_rope(_ROPE_PARAMS.pack(
            _ROPE_PARAMS.size, _DTYPE[dtype], q.data_ptr(), qs[0], qs[1], q_out.data_ptr(), os[0], os[1], *ks,
            positions.data_ptr(), cos_sin_cache.data_ptr(), P, T, H, Hk, D, rot, rot_offset, 1 if is_neox else 0,
            1 if inverse else 0, handle))
    if st:
        _check(st, "smla_rope")
    return q_out, k_out


def _kv8_cache(k_cache, v_cache, k_scale, v_scale):
    for name, x in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(x, torch.Tensor) or x.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise TypeError("%s must be E4M3 codes (uint8 / float8_e4m3fn)" % name)
    _need(k_cache, "k_cache", k_cache.dtype, 4)
    dev = k_cache.device
    _fits(v_cache, "v_cache", v_cache.dtype, 4, dev)
    shape = k_cache.shape
    if shape != v_cache.shape:
        raise ValueError("k_cache is %s, v_cache %s" % (tuple(shape), tuple(v_cache.shape)))
    _fits(k_scale, "k_scale", torch.float32, 2, dev)
    _fits(v_scale, "v_scale", torch.float32, 2, dev)
    if k_scale.shape != shape[:2] or v_scale.shape != shape[:2]:
        raise ValueError("k_scale and v_scale must be [num_blocks, H_kv] = %s" % (tuple(shape[:2]),))
    return shape


def smla_kv8_append(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, stream=None):
    """Writes bf16 rows k, v [T, H_kv, D] (may be strided) at their slots of the
    block-scaled cache: k_cache, v_cache [num_blocks, H_kv, block_size, D] E4M3
    codes, k_scale, v_scale fp32 [num_blocks, H_kv]. A block's scale grows with
    its largest value and its older codes follow. Returns (k_cache, v_cache)."""
    num_blocks, H_kv, block_size, D = _kv8_cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    _rows(k, "k", torch.bfloat16, 3, dev)
    _rows(v, "v", torch.bfloat16, 3, dev)
    T = k.shape[0]
    if k.shape != (T, H_kv, D) or v.shape != (T, H_kv, D):
        raise ValueError("k and v must be [T, %d, %d], got %s and %s" % (H_kv, D, tuple(k.shape), tuple(v.shape)))
    _fits(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    if slot_mapping.shape[0] != T:
        raise ValueError("slot_mapping must be [T] = [%d]" % T)
    ks, vs = k.stride(), v.stride()
    L = _lib or lib()
    with _on(dev, stream) as handle:
        st = L.smla_kv8_append(k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], slot_mapping.data_ptr(), T,
                               H_kv, D, block_size, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                               v_scale.data_ptr(), num_blocks, handle)
    if st:
        _check(st, "smla_kv8_append")
    return k_cache, v_cache


def smla_kv8_attn_workspace_size(B: int, T: int, H: int, H_kv: int, D: int, max_query_len: int) -> int:
    """Workspace bytes of smla_kv8_attn_fwd on the current device."""
    n = lib().smla_kv8_attn_workspace_size(B, T, H, H_kv, D, max_query_len)
    if n == ctypes.c_size_t(-1).value:
        raise SmlaError(SMLA_ERR_BAD_SHAPE, "smla_kv8_attn_workspace_size")
    return int(n)


def smla_kv8_attn_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                      v_scale: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                      query_start: torch.Tensor, scale: float, *, max_query_len: int, window: int = 0,
                      sinks: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                      workspace: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal attention of each request's last tokens over its pages of the
    block-scaled cache: out [T, H, D] (bf16) and lse [T, H] (fp32).

    q bf16 [T, H, D] (rows may be strided); the caches and scales as for
    smla_kv8_append, H a multiple of H_kv; block_table int32 [B, width] (rows
    may be strided); seq_lens int32 [B]; query_start int32 [B + 1] (rows of q
    past query_start[B] are left alone); max_query_len: a bound of the requests'
    tokens in q; window > 0: each token sees its last `window` positions; sinks
    fp32 [H]: logits that join the denominator."""
    num_blocks, H_kv, block_size, D = _kv8_cache(k_cache, v_cache, k_scale, v_scale)
    dev = k_cache.device
    _rows(q, "q", torch.bfloat16, 3, dev)
    T, H, Dq = q.shape
    if Dq != D or H_kv == 0 or H % H_kv != 0 or H == 0:
        raise ValueError("q is %s, the cache has %d heads of %d columns" % (tuple(q.shape), H_kv, D))
    _rows(block_table, "block_table", torch.int32, 2, dev)
    B, width = block_table.shape
    row_stride = block_table.stride(0)
    if B <= 1 and row_stride < width:
        row_stride = width
    _fits(seq_lens, "seq_lens", torch.int32, 1, dev)
    _fits(query_start, "query_start", torch.int32, 1, dev)
    if seq_lens.shape[0] != B or query_start.shape[0] != B + 1:
        raise ValueError("seq_lens must be [B], query_start [B + 1], B = %d" % B)
    if sinks is not None:
        _fits(sinks, "sinks", torch.float32, 1, dev)
        if sinks.shape[0] != H:
            raise ValueError("sinks must be [H]")
    L = _lib or lib()
    with _on(dev, stream) as handle:
        out = _out(out, "out", (T, H, D), torch.bfloat16, dev)
        if lse is not None or return_lse:
            lse = _out(lse, "lse", (T, H), torch.float32, dev)
        try:
            need = _kv8_attn_workspace(dev.index, B, T, H, H_kv, D, max_query_len, width, block_size)
        except SmlaError:
            need = 256  # (the call says what is wrong)
        workspace, ws_bytes = _workspace(workspace, need, dev)
        qs = q.stride()
        st = L.smla_kv8_attn_fwd(_KV8_ATTN_PARAMS.pack(
            _KV8_ATTN_PARAMS.size, q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), num_blocks, block_table.data_ptr(), row_stride, width,
            seq_lens.data_ptr(), query_start.data_ptr(), B, T, H, H_kv, D, block_size, max_query_len, window, scale,
            0 if sinks is None else sinks.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
            workspace.data_ptr(), ws_bytes, handle))
    if st:
        _check(st, "smla_kv8_attn_fwd")
    return out, lse


def new_kv8_cache(num_blocks: int, H_kv: int, block_size: int, D: int, device="cuda"):
    """An empty block-scaled cache: (k_cache, v_cache, k_scale, v_scale)."""
    shape = (num_blocks, H_kv, block_size, D)
    return (torch.zeros(shape, dtype=torch.uint8, device=device), torch.zeros(shape, dtype=torch.uint8, device=device),
            torch.ones((num_blocks, H_kv), dtype=torch.float32, device=device),
            torch.ones((num_blocks, H_kv), dtype=torch.float32, device=device))
