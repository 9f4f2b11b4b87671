"""Thin binding over libexattn.so (include/exattn.h): ctypes, and for the calls
whose kernels take a few microseconds the compiled _binding.so.

Argument marshalling only: every step of attention runs in the library's
CUDA kernels.  torch supplies device memory and the current stream.  There is
no fallback: if the library is missing or fails to load, these functions raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libexattn.so")

ATTN_OK = 0
STATUS_NAMES = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_MISALIGNED",
                4: "ATTN_ERR_CUDA", 5: "ATTN_ERR_TIMEOUT", 6: "ATTN_ERR_WORKSPACE", 7: "ATTN_ERR_NOT_IMPLEMENTED",
                8: "ATTN_ERR_PAGE", 9: "ATTN_ERR_TREE"}
ATTN_BF16, ATTN_FP16 = 0, 1
# attn_mask: none, top-left causal (query q sees keys k <= q), bottom-right causal (k <= q + Nk - Nq)
ATTN_MASK_NONE, ATTN_MASK_CAUSAL, ATTN_MASK_CAUSAL_BOTTOM_RIGHT = 0, 1, 2
_MASKS = {False: 0, True: 1, 0: 0, 1: 1, 2: 2, "none": 0, "top_left": 1, "bottom_right": 2}
# attn_dq_mode
DQ_MODES = {"atomic": 0, "deterministic": 1, "auto": 2}
# attn_bwd is these three C-ABI calls in this order
BWD_STEPS = ("attn_bwd_preprocess", "attn_bwd_kv_blocks", "attn_bwd_dq_convert")

_lock = threading.Lock()
_lib = None
_lib_path = None


class Strides(ctypes.Structure):
    """attn_strides: element strides of a [B][H][N][d] view with contiguous d."""
    _fields_ = [("batch", ctypes.c_longlong), ("head", ctypes.c_longlong), ("row", ctypes.c_longlong)]


class CacheStruct(ctypes.Structure):
    """attn_cache"""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "page_table")]
                + [(n, ctypes.c_int) for n in ("num_pages", "heads", "page_size", "d", "table_width", "format")])


class RopeStruct(ctypes.Structure):
    """attn_rope"""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("freq", "start", "offsets")] + [("offset_stride", ctypes.c_longlong)]
                + [(n, ctypes.c_void_p) for n in ("q_weight", "k_weight")]
                + [(n, ctypes.c_int) for n in ("rotary_dim", "layout", "weight_fp32")]
                + [(n, ctypes.c_float) for n in ("amplitude", "eps")])


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = last_error()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status_string(status)})"
                         + (f": {detail}" if detail else ""))


def last_error() -> str:
    """The library's description of its most recent failure on this thread ("" if none)."""
    return load().attn_last_error().decode()


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (raises OSError if it is missing).  With another one than that beside this file the calls of the compiled
    binding, which calls the latter, are not to be had."""
    global _lib, _lib_path
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise OSError(f"{path} not found: build it with exact_head_attention_gb300.build.build()")
            lib = ctypes.CDLL(path)
            vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
            lib.attn_fwd.restype = i
            st = Strides
            lib.attn_fwd_strided.argtypes = [vp, st, vp, st, vp, st, vp, st, vp, i, i, i, i, i, i, f, i, vp]
            lib.attn_fwd_strided.restype = i
            lib.attn_bwd_strided.argtypes = [vp, st, vp, st, vp, st, vp, st, vp, st, vp, vp, st, vp, st, vp, st,
                                             i, i, i, i, i, i, f, i, vp, sz, vp]
            lib.attn_bwd_strided.restype = i
            lib.attn_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp, sz, vp]
            lib.attn_fwd_splitkv.restype = i
            lib.attn_fwd_splitkv_strided.argtypes = [vp, st, vp, st, vp, st, vp, st, vp, i, i, i, i, i, i, f, i, i, vp,
                                                     sz, vp]
            lib.attn_fwd_splitkv_strided.restype = i
            lib.attn_fwd_splitkv_num_splits.argtypes = [i, i, i, i, i, i]
            lib.attn_fwd_splitkv_num_splits.restype = i
            lib.attn_fwd_splitkv_workspace_size.argtypes = [i, i, i, i, i, i]
            lib.attn_fwd_splitkv_workspace_size.restype = sz
            lib.attn_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp, sz, vp]
            lib.attn_bwd_ex.restype = i
            lib.attn_bwd_strided_ex.argtypes = [vp, st, vp, st, vp, st, vp, st, vp, st, vp, vp, st, vp, st, vp, st,
                                                i, i, i, i, i, i, f, i, i, vp, sz, vp]
            lib.attn_bwd_strided_ex.restype = i
            lib.attn_kl_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
            lib.attn_kl_fwd.restype = i
            lib.attn_kl_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, f, i, vp]
            lib.attn_kl_bwd.restype = i
            lib.attn_kl_bwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, f, i, i, vp,
                                           sz, vp]
            lib.attn_kl_bwd_ex.restype = i
            lib.attn_kl_bwd_workspace_size.argtypes = [i, i, i, i]
            lib.attn_kl_bwd_workspace_size.restype = sz
            lib.attn_selftest_wait_timeout.argtypes = [i, vp]
            lib.attn_selftest_wait_timeout.restype = i
            lib.attn_kl_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp, sz, vp]
            lib.attn_kl_fwd_splitkv.restype = i
            lib.attn_kl_fwd_splitkv_workspace_size.argtypes = [i, i, i, i, i, i]
            lib.attn_kl_fwd_splitkv_workspace_size.restype = sz
            lib.attn_fwd_schedule.argtypes = [i, i, i, i, i, i, i, vp, i, vp, i]
            lib.attn_fwd_schedule.restype = i
            lib.attn_bwd_head_group.argtypes = [i, i, i, i, i, i, i, sz]
            lib.attn_bwd_head_group.restype = i
            lib.attn_bwd_auto_dq_mode.argtypes = [i, i, i, i, i, i]
            lib.attn_bwd_auto_dq_mode.restype = i
            lib.attn_bwd_workspace_size.argtypes = [i, i, i, i]
            lib.attn_bwd_workspace_size.restype = sz
            for name in ("attn_bwd",) + BWD_STEPS:
                fn = getattr(lib, name)
                fn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, sz, vp]
                fn.restype = i
            cp = ctypes.POINTER(CacheStruct)
            lib.attn_cache_write.argtypes = [cp, vp, st, vp, st, vp, vp, i, i, i, vp]
            lib.attn_cache_write.restype = i
            lib.attn_cache_read.argtypes = [cp, vp, vp, vp, st, vp, st, i, i, i, vp]
            lib.attn_cache_read.restype = i
            lib.attn_fwd_cache.argtypes = [vp, st, cp, vp, vp, st, vp, i, i, i, i, f, i, vp, sz, vp]
            lib.attn_fwd_cache.restype = i
            lib.attn_fwd_cache_workspace_size.argtypes = [cp, i, i, i]
            lib.attn_fwd_cache_workspace_size.restype = sz
            lib.attn_fwd_cache_tree.argtypes = [vp, st, cp, vp, vp, ctypes.c_longlong, vp, st, vp, i, i, i, f, i, vp, sz, vp]
            lib.attn_fwd_cache_tree.restype = i
            lib.attn_draft_tree.argtypes = [vp, vp, vp, i, i, vp]
            lib.attn_draft_tree.restype = i
            rp = ctypes.POINTER(RopeStruct)
            lib.attn_rope_fwd.argtypes = [vp, st, vp, st, vp, st, vp, st, i, i, i, i, i, rp, i, vp]
            lib.attn_rope_fwd.restype = i
            lib.attn_rope_bwd.argtypes = [vp, st, vp, st, vp, st, vp, st, vp, st, vp, st, vp, vp, i, i, i, i, i, rp, i, vp,
                                          sz, vp]
            lib.attn_rope_bwd.restype = i
            lib.attn_cache_append.argtypes = [cp, vp, st, vp, st, vp, st, vp, st, vp, vp, i, i, i, rp, i, vp]
            lib.attn_cache_append.restype = i
            lib.attn_rope_bwd_workspace_size.argtypes = [i]
            lib.attn_rope_bwd_workspace_size.restype = sz
            lib.attn_status_string.argtypes = [i]
            lib.attn_status_string.restype = ctypes.c_char_p
            lib.attn_check_device_error.argtypes = [vp]
            lib.attn_check_device_error.restype = i
            lib.attn_last_error.argtypes = []
            lib.attn_last_error.restype = ctypes.c_char_p
            _lib_path = os.path.realpath(path)
            _lib = lib
    return _lib


_compiled = None


def binding():
    """The compiled binding (_binding.so), behind the library beside it (raises OSError if it is missing or stale)."""
    global _compiled
    if _compiled is None:
        load()
        if _lib_path != os.path.realpath(LIB_PATH):
            raise OSError(f"{_lib_path} is loaded, and the compiled binding calls {LIB_PATH}: these calls need the latter")
        from exact_head_attention_gb300 import build
        hint = "build it with exact_head_attention_gb300.build.build()"
        if os.path.exists(build.BINDING_STAMP):
            with open(build.BINDING_STAMP) as f:
                was = f.read()
            if was != build._torch_stamp():
                raise OSError(f"_binding.so is of torch and Python {was}, not {build._torch_stamp()}: {hint}")
        try:
            from exact_head_attention_gb300 import _binding
        except ImportError as e:
            raise OSError(f"_binding.so not found, or not to be loaded ({e}): {hint}") from e
        _binding.set_error_class(AttnError)
        _compiled = _binding
    return _compiled


def status_string(status: int) -> str:
    return load().attn_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    if t.dtype == torch.float16:
        return ATTN_FP16
    raise TypeError(f"unsupported dtype {t.dtype}; expected bfloat16 or float16")


def mask_code(causal) -> int:
    """attn_mask value of `causal`: False/0/"none", True/1/"top_left", 2/"bottom_right"."""
    if causal not in _MASKS:
        raise ValueError(f"unknown causal mask {causal!r}")
    return _MASKS[causal]


def _ptr(t):
    if t is None:
        return None
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("tensors must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _view(t):
    """(pointer, Strides) of a [B, H, N, d] CUDA tensor whose last dimension is contiguous."""
    if not t.is_cuda or t.dim() != 4 or t.stride(3) != 1:
        raise ValueError("tensors must be [B, H, N, d] CUDA tensors with a contiguous last dimension")
    return ctypes.c_void_p(t.data_ptr()), Strides(t.stride(0), t.stride(1), t.stride(2))


def _all_contiguous(*ts) -> bool:
    return all(t.is_contiguous() for t in ts)


# The current stream's raw handle without building a Stream object (several microseconds a call);
# the public call is the fallback where this accessor is absent.
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _RAW_STREAM is not None:
        return ctypes.c_void_p(_RAW_STREAM(torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, H, Nq, d = q.shape
    return B, H, Nq, k.shape[2], d


def _check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)


def fwd_raw(q, k, v, o, lse, causal, scale: float, stream=None) -> int:
    """Calls attn_fwd on caller-provided contiguous tensors; returns the status code."""
    B, H, Nq, Nk, d = _dims(q, k)
    return load().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d, mask_code(causal),
                           float(scale), _dtype_code(q), _stream(stream))


def fwd_strided_raw(q, k, v, o, lse, causal, scale: float, stream=None) -> int:
    """Calls attn_fwd_strided with each tensor's own strides; returns the status code."""
    B, H, Nq, Nk, d = _dims(q, k)
    return load().attn_fwd_strided(*_view(q), *_view(k), *_view(v), *_view(o), _ptr(lse), B, H, Nq, Nk, d,
                                   mask_code(causal), float(scale), _dtype_code(q), _stream(stream))


def forward(q, k, v, causal=False, scale: float | None = None, stream=None):
    """O [B,H,Nq,d] (dtype and, where dense, strides of q) and LSE [B,H,Nq] fp32.

    `causal`: False, True (top-left) or "bottom_right".  Non-contiguous views whose last
    dimension is contiguous (e.g. [B, N, H, d] storage seen as [B, H, N, d]) go through
    attn_fwd_strided without a copy."""
    B, H, Nq, Nk, d = _dims(q, k)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if _all_contiguous(q, k, v, o):
        _check(fwd_raw(q, k, v, o, lse, causal, scale, stream), "attn_fwd")
    else:
        _check(fwd_strided_raw(q, k, v, o, lse, causal, scale, stream), "attn_fwd_strided")
    return o, lse


def splitkv_num_splits(B: int, H: int, Nq: int, Nk: int, d: int, sm_count: int = 0) -> int:
    """Slices per query tile attn_fwd_splitkv picks for num_splits = 0 (sm_count 0: the current device)."""
    return int(load().attn_fwd_splitkv_num_splits(B, H, Nq, Nk, d, sm_count))


def splitkv_workspace_size(B: int, H: int, Nq: int, Nk: int, d: int, num_splits: int = 0) -> int:
    return int(load().attn_fwd_splitkv_workspace_size(B, H, Nq, Nk, d, num_splits))


def fwd_splitkv_raw(q, k, v, o, lse, causal, scale: float, num_splits: int, workspace, stream=None) -> int:
    """Calls attn_fwd_splitkv (contiguous tensors) or attn_fwd_splitkv_strided; returns the status code."""
    B, H, Nq, Nk, d = _dims(q, k)
    common = (B, H, Nq, Nk, d, mask_code(causal), float(scale), _dtype_code(q), int(num_splits),
              *_workspace(workspace), _stream(stream))
    if _all_contiguous(q, k, v, o):
        return load().attn_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), *common)
    return load().attn_fwd_splitkv_strided(*_view(q), *_view(k), *_view(v), *_view(o), _ptr(lse), *common)


def forward_splitkv(q, k, v, causal=False, scale: float | None = None, num_splits: int = 0, stream=None):
    """forward() for few query rows with the key dimension divided across blocks (decoding).

    num_splits = 0 lets the library choose (possibly 1, i.e. the plain forward)."""
    B, H, Nq, Nk, d = _dims(q, k)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    ws_bytes = splitkv_workspace_size(B, H, Nq, Nk, d, num_splits)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
    _check(fwd_splitkv_raw(q, k, v, o, lse, causal, scale, num_splits, ws, stream), "attn_fwd_splitkv")
    return o, lse


def workspace_size(B: int, H: int, Nq: int, d: int) -> int:
    return int(load().attn_bwd_workspace_size(B, H, Nq, d))


def _workspace(workspace):
    ws_ptr = None if workspace is None else ctypes.c_void_p(workspace.data_ptr())
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return ws_ptr, ws_bytes


def bwd_raw(q, k, v, o, do, lse, dq, dk, dv, causal, scale: float, workspace, stream=None,
            step: str = "attn_bwd") -> int:
    """Calls attn_bwd (or one of BWD_STEPS) on caller-provided contiguous tensors; returns the status code."""
    B, H, Nq, Nk, d = _dims(q, k)
    fn = getattr(load(), step)
    return fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
              B, H, Nq, Nk, d, mask_code(causal), float(scale), _dtype_code(q), *_workspace(workspace),
              _stream(stream))


def bwd_strided_raw(q, k, v, o, do, lse, dq, dk, dv, causal, scale: float, workspace, stream=None) -> int:
    """Calls attn_bwd_strided with each tensor's own strides; returns the status code."""
    B, H, Nq, Nk, d = _dims(q, k)
    return load().attn_bwd_strided(*_view(q), *_view(k), *_view(v), *_view(o), *_view(do), _ptr(lse),
                                   *_view(dq), *_view(dk), *_view(dv), B, H, Nq, Nk, d, mask_code(causal),
                                   float(scale), _dtype_code(q), *_workspace(workspace), _stream(stream))


def fwd_schedule(B: int, H: int, Nq: int, Nk: int, d: int, causal=False, sm_count: int = 0):
    """The forward's packed lists of query blocks (attn_fwd_schedule): a list of per-CTA lists of block
    ids (bh * ceil(Nq/256) + qb), or None when the plain launch is used."""
    cap = 2048
    blocks = (ctypes.c_uint32 * cap)()
    begin = (ctypes.c_int * 256)()
    n = int(load().attn_fwd_schedule(B, H, Nq, Nk, d, mask_code(causal), sm_count, blocks, cap, begin, 256))
    if n < 0:
        raise ValueError("invalid sizes")
    if n == 0:
        return None
    return [list(blocks[begin[c]:begin[c + 1]]) for c in range(n)]


def head_group(B: int, H: int, Nq: int, Nk: int, d: int, causal=False, sm_count: int = 0, l2_bytes: int = 0) -> int:
    """Heads per launch group of the reducing backward (attn_bwd_head_group); sm_count / l2_bytes 0 take
    the current device's values."""
    g = int(load().attn_bwd_head_group(B, H, Nq, Nk, d, mask_code(causal), sm_count, l2_bytes))
    if g < 0:
        raise ValueError("invalid sizes")
    return g


def auto_dq_mode(B: int, H: int, Nq: int, Nk: int, d: int, causal=False) -> str:
    """The mode "auto" resolves to for this backward (attn_bwd_auto_dq_mode)."""
    code = int(load().attn_bwd_auto_dq_mode(B, H, Nq, Nk, d, mask_code(causal)))
    if code < 0:
        raise ValueError("invalid sizes")
    return {v: k for k, v in DQ_MODES.items()}[code]


def dq_mode_code(dq_mode) -> int:
    if isinstance(dq_mode, str):
        if dq_mode not in DQ_MODES:
            raise ValueError(f"unknown dq_mode {dq_mode!r}")
        return DQ_MODES[dq_mode]
    return int(dq_mode)


def bwd_ex_raw(q, k, v, o, do, lse, dq, dk, dv, causal, scale: float, dq_mode, workspace, stream=None) -> int:
    """Calls attn_bwd_ex (contiguous) or attn_bwd_strided_ex with a dQ mode; returns the status code."""
    B, H, Nq, Nk, d = _dims(q, k)
    common = (B, H, Nq, Nk, d, mask_code(causal), float(scale), _dtype_code(q), dq_mode_code(dq_mode),
              *_workspace(workspace), _stream(stream))
    if _all_contiguous(q, k, v, o, do, dq, dk, dv):
        return load().attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                                  _ptr(dv), *common)
    return load().attn_bwd_strided_ex(*_view(q), *_view(k), *_view(v), *_view(o), *_view(do), _ptr(lse),
                                      *_view(dq), *_view(dk), *_view(dv), *common)


def backward(q, k, v, o, do, lse, causal=False, scale: float | None = None, workspace=None, stream=None,
             dq_mode="atomic"):
    """(dQ, dK, dV) for the loss sum(O * dO).  `workspace` (uint8 CUDA tensor) is allocated if omitted.

    dq_mode: "atomic" (attn_bwd), "deterministic" (dQ from a query-tile kernel, same bits on every
    run) or "auto".  Gradients take the strides of q, k, v where those are dense; views go through
    the strided entry points."""
    B, H, Nq, Nk, d = _dims(q, k)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    if workspace is None:
        workspace = torch.empty(workspace_size(B, H, Nq, d), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if dq_mode_code(dq_mode) != DQ_MODES["atomic"]:
        _check(bwd_ex_raw(q, k, v, o, do, lse, dq, dk, dv, causal, scale, dq_mode, workspace, stream), "attn_bwd_ex")
    elif _all_contiguous(q, k, v, o, do, dq, dk, dv):
        _check(bwd_raw(q, k, v, o, do, lse, dq, dk, dv, causal, scale, workspace, stream), "attn_bwd")
    else:
        _check(bwd_strided_raw(q, k, v, o, do, lse, dq, dk, dv, causal, scale, workspace, stream),
               "attn_bwd_strided")
    return dq, dk, dv


def selftest_wait_timeout(timeout_ms: int = 20, stream=None) -> int:
    """Runs attn_selftest_wait_timeout: a bounded device wait that nothing satisfies.  Returns the status
    (ATTN_ERR_TIMEOUT = 5 when the timeout path works)."""
    return int(load().attn_selftest_wait_timeout(int(timeout_ms), _stream(stream)))


def check_device_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error status."""
    return int(load().attn_check_device_error(_stream(stream)))


class _FirstGradients(torch.autograd.Function):
    @staticmethod
    def forward(ctx, n, *tensors):
        return tensors[:n]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("a gradient of these gradients is asked for: their kernels are differentiable once")


def _first_gradients(grads, *inputs):
    """`grads` of a backward pass, from `inputs` by kernels that record nothing.  Where they are recorded (create_graph=True) and
    depend on what needs gradients itself, a gradient of them raises instead of lacking their terms."""
    inputs = [t for t in inputs if t is not None and t.requires_grad]
    if not inputs or not torch.is_grad_enabled():
        return grads
    at = [i for i, g in enumerate(grads) if g is not None]
    out = list(grads)
    for i, g in zip(at, _FirstGradients.apply(len(at), *(grads[i] for i in at), *inputs)):
        out[i] = g
    return tuple(out)


class _AttnFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale, dq_mode):
        o, lse = forward(q, k, v, causal, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.scale, ctx.dq_mode = causal, scale, dq_mode
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        if do.stride(-1) != 1:
            do = do.contiguous()
        grads = backward(q, k, v, o, do, lse, ctx.causal, ctx.scale, dq_mode=ctx.dq_mode)
        return *_first_gradients(grads, q, k, v, do), None, None, None


def attention(q, k, v, causal=False, scale: float | None = None, dq_mode="atomic"):
    """Autograd-aware exact attention over [B, H, N, d] tensors (causal: False, True or "bottom_right";
    dq_mode: "atomic", "deterministic" or "auto"); a gradient of its gradients raises."""
    scale = (1.0 / q.shape[-1] ** 0.5) if scale is None else scale
    return _AttnFunction.apply(q, k, v, causal, scale, dq_mode)


# ------------------------------------------------------------------ attention KL divergence

KL_SETTINGS = {"student": 1, "teacher": 2, 1: 1, 2: 2}


def kl_fwd_raw(q1, k1, q2, k2, kl, lse1, lse2, causal, scale: float, stream=None) -> int:
    """Calls attn_kl_fwd on caller-provided contiguous tensors; returns the status code."""
    B, H, Nq, Nk, d = _dims(q1, k1)
    return load().attn_kl_fwd(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(kl), _ptr(lse1), _ptr(lse2), B, H, Nq,
                              Nk, d, mask_code(causal), float(scale), _dtype_code(q1), _stream(stream))


def kl_bwd_raw(q1, k1, q2, k2, kl, lse1, lse2, g, setting, dq, dk, causal, scale: float, stream=None) -> int:
    """Calls attn_kl_bwd on caller-provided contiguous tensors; returns the status code."""
    B, H, Nq, Nk, d = _dims(q1, k1)
    return load().attn_kl_bwd(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(kl), _ptr(lse1), _ptr(lse2), _ptr(g),
                              KL_SETTINGS[setting], _ptr(dq), _ptr(dk), B, H, Nq, Nk, d, mask_code(causal),
                              float(scale), _dtype_code(q1), _stream(stream))


def kl_bwd_workspace_size(B: int, H: int, Nq: int, d: int) -> int:
    """Workspace bytes of the one-pass KL backward (attn_kl_bwd_workspace_size)."""
    return int(load().attn_kl_bwd_workspace_size(B, H, Nq, d))


def kl_bwd_ex_raw(q1, k1, q2, k2, kl, lse1, lse2, g, setting, dq, dk, causal, scale: float, dq_mode, workspace,
                  stream=None) -> int:
    """Calls attn_kl_bwd_ex (dQ mode, workspace) on caller-provided contiguous tensors; returns the status."""
    B, H, Nq, Nk, d = _dims(q1, k1)
    return load().attn_kl_bwd_ex(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(kl), _ptr(lse1), _ptr(lse2), _ptr(g),
                                 KL_SETTINGS[setting], _ptr(dq), _ptr(dk), B, H, Nq, Nk, d, mask_code(causal),
                                 float(scale), _dtype_code(q1), dq_mode_code(dq_mode), *_workspace(workspace),
                                 _stream(stream))


def kl_forward(q1, k1, q2, k2, causal=False, scale: float | None = None, stream=None):
    """Row-wise KL(P1 || P2) of the student (q2, k2) from the teacher (q1, k1): (KL, LSE1, LSE2) [B,H,Nq] fp32."""
    B, H, Nq, Nk, d = _dims(q1, k1)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    kl, lse1, lse2 = (torch.empty((B, H, Nq), dtype=torch.float32, device=q1.device) for _ in range(3))
    _check(kl_fwd_raw(q1, k1, q2, k2, kl, lse1, lse2, causal, scale, stream), "attn_kl_fwd")
    return kl, lse1, lse2


def kl_forward_splitkv(q1, k1, q2, k2, causal=False, scale: float | None = None, num_splits: int = 0, stream=None):
    """kl_forward for few query rows with the key dimension divided across blocks (0: library's choice)."""
    B, H, Nq, Nk, d = _dims(q1, k1)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    kl, lse1, lse2 = (torch.empty((B, H, Nq), dtype=torch.float32, device=q1.device) for _ in range(3))
    nb = int(load().attn_kl_fwd_splitkv_workspace_size(B, H, Nq, Nk, d, num_splits))
    ws = torch.empty(nb, dtype=torch.uint8, device=q1.device) if nb else None
    st = load().attn_kl_fwd_splitkv(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), _ptr(kl), _ptr(lse1), _ptr(lse2), B, H,
                                    Nq, Nk, d, mask_code(causal), float(scale), _dtype_code(q1), int(num_splits),
                                    *_workspace(ws), _stream(stream))
    _check(st, "attn_kl_fwd_splitkv")
    return kl, lse1, lse2


def kl_backward(q1, k1, q2, k2, kl, lse1, lse2, g, train="student", causal=False, scale: float | None = None,
                stream=None, dq_mode="atomic", workspace=None):
    """(dQ, dK) of sum(g * KL) for the trained distribution ("student": Q2, K2; "teacher": Q1, K1).

    dq_mode: "atomic" / "auto" (one pass over key tiles, dQ added into an fp32 accumulator; `workspace`
    is allocated if omitted) or "deterministic" (attn_kl_bwd: two launches, the same bits on every run)."""
    B, H, Nq, Nk, d = _dims(q1, k1)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    dq, dk = torch.empty_like(q1), torch.empty_like(k1)
    g = g.contiguous().float()
    if dq_mode_code(dq_mode) == DQ_MODES["deterministic"]:
        _check(kl_bwd_raw(q1, k1, q2, k2, kl, lse1, lse2, g, train, dq, dk, causal, scale, stream), "attn_kl_bwd")
        return dq, dk
    if workspace is None:
        workspace = torch.empty(kl_bwd_workspace_size(B, H, Nq, d), dtype=torch.uint8, device=q1.device)
    _check(kl_bwd_ex_raw(q1, k1, q2, k2, kl, lse1, lse2, g, train, dq, dk, causal, scale, dq_mode, workspace, stream),
           "attn_kl_bwd_ex")
    return dq, dk


class _KlFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q1, k1, q2, k2, causal, scale, train, dq_mode):
        kl, lse1, lse2 = kl_forward(q1, k1, q2, k2, causal, scale)
        ctx.save_for_backward(q1, k1, q2, k2, kl, lse1, lse2)
        ctx.causal, ctx.scale, ctx.train, ctx.dq_mode = causal, scale, train, dq_mode
        return kl

    @staticmethod
    def backward(ctx, g):
        q1, k1, q2, k2, kl, lse1, lse2 = ctx.saved_tensors
        dq, dk = kl_backward(q1, k1, q2, k2, kl, lse1, lse2, g, ctx.train, ctx.causal, ctx.scale,
                             dq_mode=ctx.dq_mode)
        dq, dk = _first_gradients((dq, dk), q1, k1, q2, k2, g)
        if KL_SETTINGS[ctx.train] == 1:
            return None, None, dq, dk, None, None, None, None
        return dq, dk, None, None, None, None, None, None


def attention_kl(q1, k1, q2, k2, causal=False, scale: float | None = None, train="student", dq_mode="atomic"):
    """Autograd-aware row-wise KL(P1 || P2) [B,H,Nq]; gradients flow to the trained distribution only,
    and a gradient of those raises."""
    scale = (1.0 / q1.shape[-1] ** 0.5) if scale is None else scale
    return _KlFunction.apply(q1, k1, q2, k2, causal, scale, train, dq_mode)


# ------------------------------------------------------------------ 8-bit key/value cache

CACHE_FORMATS = {"e4m3": 0, "int8": 1}


_CACHE_DTYPES = {torch.float8_e4m3fn: 0, torch.int8: 1}
_cache_checks = None  # binding().cache_struct, False where there is no binding


def _cache_struct(k, v, k_scale, v_scale, page_table) -> CacheStruct:
    """The attn_cache of checked tensors.  The cache's calls need no compiled binding: it makes this 1.0 us where it is there,
    for 5.5."""
    global _cache_checks
    if _cache_checks is None:
        try:
            _cache_checks = binding().cache_struct
        except OSError:
            _cache_checks = False
    if _cache_checks:
        return CacheStruct.from_buffer_copy(_cache_checks(k, v, k_scale, v_scale, page_table))
    tensors = (k, v, k_scale, v_scale, page_table)
    if not all(isinstance(t, torch.Tensor) for t in tensors):
        raise TypeError("a tensor is wanted")
    fmt = _CACHE_DTYPES.get(k.dtype)
    if fmt is None or v.dtype != k.dtype:
        raise TypeError(f"unsupported cache dtypes {k.dtype}, {v.dtype}; expected float8_e4m3fn or int8 for both")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or page_table.dtype != torch.int32:
        raise TypeError("scales must be float32 and the page table int32")
    if k.dim() != 4 or v.shape != k.shape or page_table.dim() != 2:
        raise ValueError("k, v must be [num_pages, heads, page, d] and the page table [B, width]")
    if k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2]:
        raise ValueError("scales must be [num_pages, heads]")
    if not all(t.is_cuda and t.get_device() == k.get_device() and t.is_contiguous() for t in tensors):
        raise ValueError("cache tensors must be contiguous and on one CUDA device")
    if max(*k.shape, *page_table.shape) > 2 ** 31 - 1:
        raise ValueError("tensors are too large")
    return CacheStruct(*(t.data_ptr() for t in tensors), *k.shape, page_table.shape[1], fmt)


class QuantCache:
    """An 8-bit key/value cache in pages (attn_cache): the caller's tensors and the struct the library takes.

    k, v: [num_pages, heads, page, d] float8_e4m3fn or int8 codes; k_scale, v_scale: [num_pages, heads] fp32; a
    code stands for code * scale of its page and head.  page_table: [B, width] int32, the pages of each sequence
    in order.  All contiguous, on one CUDA device; the tensors are used in place."""
    __slots__ = ("k", "v", "k_scale", "v_scale", "page_table", "device", "index", "B", "heads", "d", "struct", "_ref",
                 "address")

    def __init__(self, k, v, k_scale, v_scale, page_table):
        self.struct = _cache_struct(k, v, k_scale, v_scale, page_table)
        self._ref = ctypes.byref(self.struct)
        self.address = ctypes.addressof(self.struct)
        self.k, self.v, self.k_scale, self.v_scale, self.page_table = k, v, k_scale, v_scale, page_table
        self.device, self.index, self.B = k.device, k.get_device(), page_table.shape[0]
        self.heads, self.d = self.struct.heads, self.struct.d

    @classmethod
    def empty(cls, num_pages: int, heads: int, page: int, d: int, page_table, format: str = "e4m3"):
        """A cache of zeros on the page table's device."""
        if format not in CACHE_FORMATS:
            raise ValueError(f"unknown cache format {format!r}")
        dtype = {0: torch.float8_e4m3fn, 1: torch.int8}[CACHE_FORMATS[format]]
        dev = page_table.device
        k, v = (torch.zeros((num_pages, heads, page, d), dtype=torch.uint8, device=dev).view(dtype) for _ in range(2))
        ks, vs = (torch.zeros((num_pages, heads), dtype=torch.float32, device=dev) for _ in range(2))
        return cls(k, v, ks, vs, page_table)


def _int32(t, cache: QuantCache, name: str):
    """Address of an int32 tensor of one entry a sequence, or None."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.shape != (cache.B,) or t.get_device() != cache.index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of one entry a sequence on the cache's device")
    return t.data_ptr()


_STRIDES: dict = {}  # Strides objects by their values (building one costs more than the rest of a view's marshalling)


def _cache_view(t, cache: QuantCache, dtype):
    """(pointer, Strides) of a 16-bit [B, H, N, d] view that goes with the cache."""
    shape = t.shape
    if len(shape) != 4 or shape[0] != cache.B or shape[3] != cache.d:
        raise ValueError("tensors must be [B, H, N, d] with the page table's B and the cache's d")
    if t.get_device() != cache.index or t.dtype != dtype:
        raise ValueError("tensors must be of one dtype, on the cache's device")
    sb, sh, sn, sd = t.stride()
    if sd != 1:
        raise ValueError("tensors must have a contiguous last dimension")
    st = _STRIDES.get((sb, sh, sn))
    if st is None:
        if len(_STRIDES) >= 4096:
            _STRIDES.clear()
        st = _STRIDES[(sb, sh, sn)] = Strides(sb, sh, sn)
    return t.data_ptr(), st


def _on(cache: QuantCache, stream, call):
    """Runs `call` with the cache's device current and, where given, on `stream`: what it allocates belongs to it."""
    with torch.cuda.device(cache.device):
        if stream is None:
            return call(_stream(None))
        with torch.cuda.stream(stream):
            return call(_stream(stream))


def _run(cache: QuantCache, stream, call):
    index = torch.cuda.current_device()
    if stream is None and index == cache.index and _RAW_STREAM is not None:
        return call(_RAW_STREAM(index))
    return _on(cache, stream, call)


def cache_write(cache: QuantCache, k, v, start=None, count=None, stream=None) -> None:
    """Quantises new tokens into the cache (attn_cache_write).

    k, v: [B, heads, N, d] bf16 or fp16, last dimension contiguous.  Row n of sequence b becomes its token
    start[b] + n for n < count[b]; start None: 0, count None: N (int32 CUDA tensors otherwise).  Tokens that a
    reached page already holds keep their codes, or are rounded again where its scale has to grow."""
    shape = k.shape
    if v.shape != shape or len(shape) != 4 or shape[1] != cache.heads:
        raise ValueError("k and v must be [B, heads, N, d] with the cache's heads")
    kp, ks = _cache_view(k, cache, k.dtype)
    vp, vs = _cache_view(v, cache, k.dtype)
    args = (cache._ref, kp, ks, vp, vs, _int32(start, cache, "start"), _int32(count, cache, "count"), shape[0], shape[2],
            _dtype_code(k))
    if shape[0] == 0 or shape[2] == 0:
        return
    st = _run(cache, stream, lambda handle: load().attn_cache_write(*args, handle))
    if st != ATTN_OK:
        raise AttnError(st, "attn_cache_write")


def cache_read(cache: QuantCache, lens, rows: int | None = None, start=None, dtype=torch.bfloat16, out=None, stream=None):
    """Cached tokens back in 16 bits (attn_cache_read): (K, V) [B, heads, rows, d], row n the token start[b] + n.

    Rows at or past lens[b] are left as they were in `out`, a pair of views whose dtype and rows are then taken;
    without it the result is allocated with zeros in them."""
    if out is None and rows is None:
        raise ValueError("rows or out is needed")
    lens_at, start_at = _int32(lens, cache, "lens"), _int32(start, cache, "start")

    def call(handle):
        k, v = out if out is not None else (
            torch.zeros((cache.B, cache.heads, rows, cache.d), dtype=dtype, device=cache.device) for _ in range(2))
        shape = k.shape
        if v.shape != shape or len(shape) != 4 or shape[1] != cache.heads:
            raise ValueError("outputs must be [B, heads, N, d] with the cache's heads")
        kp, ks = _cache_view(k, cache, k.dtype)
        vp, vs = _cache_view(v, cache, k.dtype)
        code = _dtype_code(k)
        if shape[0] and shape[2]:
            st = load().attn_cache_read(cache._ref, start_at, lens_at, kp, ks, vp, vs, shape[0], shape[2], code, handle)
            if st != ATTN_OK:
                raise AttnError(st, "attn_cache_read")
        return k, v

    return _run(cache, stream, call)


def _cache_workspace(workspace, cache: QuantCache):
    """(address, bytes) of a caller's workspace."""
    if workspace.get_device() != cache.index or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the cache's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def cache_workspace_size(cache: QuantCache, H: int, Nq: int) -> int:
    """Workspace bytes of forward_cache (attn_fwd_cache_workspace_size)."""
    return int(load().attn_fwd_cache_workspace_size(cache._ref, cache.B, H, Nq))


def fwd_cache_raw(q, cache: QuantCache, lens, o, lse, causal, scale: float, workspace, stream=None) -> int:
    """Calls attn_fwd_cache on caller-provided tensors; returns the status code."""
    B, H, Nq, _ = q.shape
    qp, qs = _cache_view(q, cache, q.dtype)
    op, os_ = _cache_view(o, cache, q.dtype)
    if o.shape != q.shape or lse.shape != (B, H, Nq) or lse.dtype != torch.float32 or lse.get_device() != cache.index:
        raise ValueError("o must be shaped as q, lse float32 [B, H, Nq], on the cache's device")
    return load().attn_fwd_cache(qp, qs, cache._ref, _int32(lens, cache, "lens"), op, os_, _ptr(lse), B, H, Nq,
                                 mask_code(causal), scale, _dtype_code(q), *_cache_workspace(workspace, cache), _stream(stream))


def forward_cache(q, cache: QuantCache, lens, causal="bottom_right", scale: float | None = None, workspace=None,
                  stream=None):
    """O [B,H,Nq,d] and LSE [B,H,Nq] fp32 of attention over the first lens[b] cached tokens of every sequence.

    q: [B, H, Nq, d] bf16 or fp16, H a multiple of the cache's heads (query head h reads key/value head
    h // (H // heads)).  causal "bottom_right" (the default): the queries are a sequence's last Nq tokens; also
    False and True (top-left) as in forward().  lens: int32 CUDA tensor [B].  `workspace` (uint8 CUDA tensor of
    cache_workspace_size bytes, one for each call that may run at the same time) is allocated if omitted."""
    qp, qs = _cache_view(q, cache, q.dtype)
    B, H, Nq, d = q.shape
    code, mask, lens_at = _dtype_code(q), mask_code(causal), _int32(lens, cache, "lens")
    scale = (1.0 / d ** 0.5) if scale is None else scale

    def call(handle):
        o = torch.empty_like(q)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=cache.device)
        if B and H and Nq:
            lib = load()
            if workspace is None:
                size = lib.attn_fwd_cache_workspace_size(cache._ref, B, H, Nq)
                space = torch.empty(size, dtype=torch.uint8, device=cache.device)
                at = space.data_ptr()
            else:
                at, size = _cache_workspace(workspace, cache)
            op, os_ = _cache_view(o, cache, q.dtype)
            st = lib.attn_fwd_cache(qp, qs, cache._ref, lens_at, op, os_, lse.data_ptr(), B, H, Nq, mask, scale, code,
                                    at, size, handle)
            if st != ATTN_OK:
                raise AttnError(st, "attn_fwd_cache")
        return o, lse

    return _run(cache, stream, call)


def _fast(stream, on, call):
    """Runs a call of the compiled binding on the tensor (or cache) `on`, on `stream` where that is given: what it allocates belongs
    to it."""
    if stream is None:
        return call()
    if stream.device != getattr(on, "device", stream.device):
        raise ValueError("the stream is of another device than the tensors")
    with torch.cuda.device(stream.device), torch.cuda.stream(stream):
        return call()


def draft_tree(parents, stream=None):
    """Masks and depths of trees of drafted tokens (attn_draft_tree): (mask [B, N, ceil(N / 32)], depth [B, N]), int32.

    parents: int32 CUDA tensor [B, N] (or [N], one tree for all sequences: B is 1), -1 or the number of an earlier token.
    The mask has each token's ancestors and itself as bits, for forward_cache_tree; the depth is its number of drafted
    ancestors, the offsets of rope_forward and cache_append."""
    return _fast(stream, parents, lambda: binding().draft_tree(parents))


def forward_cache_tree(q, cache: QuantCache, lens, tree, scale: float | None = None, workspace=None, stream=None):
    """forward_cache for a tree of drafted tokens (attn_fwd_cache_tree): the queries are a sequence's last Nq tokens; each
    sees what is before those, and of them what its bits in `tree` say.

    tree: int32 CUDA tensor [B, Nq, ceil(Nq / 32)], or [1, ...] for all sequences alike (draft_tree): bit j % 32 of word
    j // 32 of row i, for j <= i.  The other arguments as in forward_cache."""
    return _fast(stream, cache, lambda: binding().forward_cache_tree(cache.address, cache.index, cache.B, q, lens, tree, scale, workspace))


# ------------------------------------------------------------------ rotary positions and norms per head

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     trained: int | None = None, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(freq, amplitude) for rope_forward and cache_append: freq [rotary_dim / 2] fp64 on `device`, radians a position.

    Pair i turns by base^(-2 i / rotary_dim) a position.  scaling for contexts `factor` times the trained length:
      None      as they are
      "linear"  positions divided by the factor
      "ntk"     the base raised so that the slowest pair is interpolated and the fastest stays
      "yarn"    (Peng et al., 2023) pairs with more than `fast` turns over the `trained` positions as they are, with fewer
                than `slow` interpolated, between them by a ramp linear in the turns, as the paper's formula has it; the amplitude
                0.1 ln(factor) + 1 on queries and keys.  Models made with that paper's released code ramp linearly in the
                pair's number between two rounded bounds instead: their frequencies are to be given as they are."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and above 0")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be above 0")
    amplitude = 1.0
    if scaling == "ntk":
        if rotary_dim == 2:
            raise ValueError("the ntk scaling needs more than one pair")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        if not trained or not fast > slow:
            raise ValueError("the yarn scaling needs the trained length, and fast above slow")
        keep = [min(1.0, max(0.0, (trained * f / (2.0 * math.pi) - slow) / (fast - slow))) for f in freq]
        freq = [f * k + f / factor * (1.0 - k) for f, k in zip(freq, keep)]
        amplitude = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.tensor(freq, dtype=torch.float64, device=device), amplitude


def _layout(layout: str) -> int:
    code = ROPE_LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"unknown rotary layout {layout!r}")
    return code


def rope_forward(q, k, freq, start=None, offsets=None, layout="half", amplitude: float = 1.0, q_weight=None, k_weight=None,
                 eps: float = 1e-6, out=None, stream=None):
    """Queries [B, H, N, d] and keys [B, Hk, N, d] with their heads' norms and rotary positions (attn_rope_fwd): (q, k).

    freq: fp64 [rotary_dim / 2] (rope_frequencies), None for norms alone.  Row n of sequence b stands at position
    start[b] + offsets[b, n] (int32 CUDA tensors; None: 0, and n; offsets of one row are all sequences').  layout "half":
    pairs (i, i + rotary_dim / 2), or "interleaved": (2 i, 2 i + 1).  amplitude multiplies what turns.  q_weight, k_weight:
    the norms' [d] weights (fp32 or as the tensors), None: no norm.  q or k may be None.  out: a pair to write to, which may
    be (q, k) itself."""
    oq, ok = (None, None) if out is None else out
    if out is not None and oq is None and ok is None:
        raise ValueError("out must be a pair of what q and k are")
    code = _layout(layout)
    return _fast(stream, k if q is None else q,
                 lambda: binding().rope_forward(q, k, freq, start, offsets, code, amplitude, q_weight, k_weight, eps, oq, ok))


def rope_bwd_workspace_size(d: int) -> int:
    """Workspace bytes of rope_backward with weights (attn_rope_bwd_workspace_size)."""
    return int(load().attn_rope_bwd_workspace_size(d))


def rope_backward(dq, dk, q, k, freq, start=None, offsets=None, layout="half", amplitude: float = 1.0, q_weight=None,
                  k_weight=None, eps: float = 1e-6, workspace=None, stream=None):
    """Gradients of rope_forward (attn_rope_bwd): (dq, dk, dq_weight, dk_weight) from those of its outputs.

    q and k are its inputs (not read, and may be None, where that tensor has no weights); the other arguments as there.
    The weights' gradients are summed in a fixed order; None where there are no weights.  `workspace` (uint8 CUDA tensor of
    rope_bwd_workspace_size bytes, one for each call that may run at the same time) is allocated if omitted."""
    code = _layout(layout)
    return _fast(stream, dk if dq is None else dq,
                 lambda: binding().rope_backward(dq, dk, q, k, freq, start, offsets, code, amplitude, q_weight, k_weight, eps, workspace))


def _plain_strides(t):
    """t itself where the library takes its strides, else a contiguous copy (an expanded gradient, say)."""
    if t is None:
        return t
    sb, sh, sn, sd = t.stride()
    good = sd == 1 and sn >= t.shape[3] and sn % 8 == 0 and t.data_ptr() % 16 == 0
    if good and all(n == 1 or (s > 0 and s % 8 == 0) for n, s in ((t.shape[0], sb), (t.shape[1], sh))):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _RopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, freq, start, offsets, layout, amplitude, eps):
        need_q, need_k, need_qw, need_kw = ctx.needs_input_grad[:4]
        # the tensors whose gradients are computed: of a norm's weights with its input's
        ctx.sides = (q is not None and (need_q or need_qw), k is not None and (need_k or need_kw))
        sides = [(x, w) if some and w is not None else (None, w) for x, w, some in zip((q, k), (q_weight, k_weight), ctx.sides)]
        ctx.save_for_backward(sides[0][0], sides[1][0], q_weight, k_weight, freq, start, offsets)
        ctx.rest = (layout, amplitude, eps)
        return rope_forward(q, k, freq, start, offsets, layout, amplitude, q_weight, k_weight, eps)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, freq, start, offsets = ctx.saved_tensors
        layout, amplitude, eps = ctx.rest
        # weights of a tensor that is not there have gradients of zero
        weights = [w if some or g is None else None for w, g, some in zip((q_weight, k_weight), (dq, dk), ctx.sides)]
        dy = [_plain_strides(g) if some else None for g, some in zip((dq, dk), ctx.sides)]
        if dy[0] is None and dy[1] is None:
            grads = (None, None, *(None if w is None else torch.zeros_like(w) for w in weights))
        else:
            grads = rope_backward(*dy, q, k, freq, start, offsets, layout, amplitude, *weights, eps)
        return *_first_gradients(grads, *dy, q, k, *weights), None, None, None, None, None, None


def rope(q, k, freq, start=None, offsets=None, layout="half", amplitude: float = 1.0, q_weight=None, k_weight=None,
         eps: float = 1e-6):
    """Autograd-aware rope_forward: (q, k); gradients flow to q, k and the weights, once: a gradient of those raises.

    A step with its backward can be captured into a CUDA graph as long as no autograd graph of the same leaves that was
    recorded outside the capture is still alive: torch would join the two streams, which can end the process.  Where the
    leaves are this call's own tensors it is refused (RuntimeError), unless gradients are off: nothing is recorded then."""
    if torch.is_grad_enabled() and (q is not None and q.is_cuda or k is not None and k.is_cuda):
        if torch.cuda.is_current_stream_capturing() and binding().leaf_elsewhere(q, k, q_weight, k_weight):
            raise RuntimeError("rope is being captured, and an autograd graph of its leaves that was recorded outside lives")
    return _RopeFunction.apply(q, k, q_weight, k_weight, freq, start, offsets, layout, amplitude, eps)


def cache_append(cache: QuantCache, k, v, freq, start=None, count=None, offsets=None, q=None, layout="half",
                 amplitude: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6, position_start=None, out=None,
                 stream=None):
    """cache_write with norm and rotary positions of the keys on the way (attn_cache_append); returns the rotated queries.

    k, v, start, count as in cache_write; freq, offsets, layout, amplitude, weights and eps as in rope_forward, the position
    of row n of sequence b being start[b] + offsets[b, n] (position_start, where given, in place of start).  q: [B, H, N, d]
    of the same tokens, or None; all its rows are turned, into `out` (which may be q) where that is given."""
    code = _layout(layout)
    return _fast(stream, cache, lambda: binding().cache_append(cache.address, cache.index, cache.B, k, v, freq, start, count, offsets, q,
                                                               code, amplitude, q_weight, k_weight, eps, position_start, out))
