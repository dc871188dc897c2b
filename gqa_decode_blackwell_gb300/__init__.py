"""Python binding of the GB300 GQA decode library (``include/gqa_decode.h``,
``include/gqa_shared_keys.h`` and ``include/gqa_paged.h``).

Argument marshalling only: every function below turns PyTorch tensors into
the plain pointers and sizes of the C entry point of the same name and calls
it (those of ``include/gqa_paged.h`` by way of ``csrc/paged_binding.cpp``).
All computation happens in the sm_103a kernels of
``libgqa_decode_sm103.so``; there is no fallback.  If the library has not
been built, the first call raises ``RuntimeError`` (build it with
``gqa_decode_blackwell_gb300.build.build()``).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import re
import threading
from typing import Optional

from .build import HEADER, LIB, PAGED_HEADER, SHARED_KEYS_HEADER, binding_path

GQA_OK = 0
GQA_ERR_INVALID_ARG = 1
GQA_ERR_UNSUPPORTED = 2
GQA_ERR_WORKSPACE = 3
GQA_ERR_CUDA = 4
GQA_ERR_TIMEOUT = 5
GQA_ERR_BAD_SEQLEN = 6
GQA_ERR_BOUNDS = 7
GQA_ERR_BAD_INDEX = 8
GQA_DTYPE_BF16 = 0
GQA_DTYPE_FP32 = 1
GQA_DTYPE_FP16 = 2
GQA_REDUCE_AUTO = 0
GQA_REDUCE_COMBINE = 1
GQA_REDUCE_CLUSTER = 2
_REDUCTIONS = {"auto": GQA_REDUCE_AUTO, "combine": GQA_REDUCE_COMBINE, "cluster": GQA_REDUCE_CLUSTER}

GQA_MAX_TREE_TOKENS = 256
_ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}

_lock = threading.Lock()
_lib = None


class GQAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gqa_status_string(status)} (status {status})")


class gqa_desc_t(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int),
        ("q_tokens", ctypes.c_int),
        ("q_heads", ctypes.c_int),
        ("kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("max_seqlen", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("causal", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("in_dtype", ctypes.c_int),
        ("reduction", ctypes.c_int),
    ]


class gqa_pages_t(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("max_pages", ctypes.c_int),
        ("page_stride", ctypes.c_int64),
        ("pos_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
    ]


class gqa_rotary_t(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int),
        ("interleaved", ctypes.c_int),
        ("inverse", ctypes.c_int),
        ("magnitude", ctypes.c_float),
    ]


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB):
                raise RuntimeError(f"GQA decode CUDA library not built ({LIB}); run "
                                   "gqa_decode_blackwell_gb300.build.build() or __graft_entry__.build()")
            _lib = load_library(LIB)
        return _lib


def load_library(path: str) -> ctypes.CDLL:
    """A build of the C library at `path` (say the -DGQA_DEBUG one) with its
    functions' argument and result types declared."""
    L = ctypes.CDLL(path)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(gqa_desc_t)
    L.gqa_decode_workspace_size.argtypes = [D, I]
    L.gqa_decode_workspace_size.restype = SZ
    L.gqa_decode_attn.argtypes = [D, P, P, P, P, P, P, I, P, SZ, P]
    L.gqa_decode_attn.restype = I
    L.gqa_decode_attn_static_workspace.argtypes = [D, P, P, P, P, P, P, I, P]
    L.gqa_decode_attn_static_workspace.restype = I
    L.gqa_decode_attn_split.argtypes = [D, P, P, P, P, P, P, I, P, SZ, P]
    L.gqa_decode_attn_split.restype = I
    L.gqa_decode_attn_merge.argtypes = [D, P, P, I, P, SZ, P]
    L.gqa_decode_attn_merge.restype = I
    L.gqa_decode_splitkv.argtypes = [D, P, P, P, P, I, P, P, P]
    L.gqa_decode_splitkv.restype = I
    L.gqa_decode_combine.argtypes = [P, P, I, I64, I, P, I, P, P]
    L.gqa_decode_combine.restype = I
    L.gqa_decode_get_error.argtypes = [I]
    L.gqa_decode_get_error.restype = I
    L.gqa_status_string.argtypes = [I]
    L.gqa_status_string.restype = ctypes.c_char_p
    L.gqa_decode_plan.argtypes = [D, P, I, I, ctypes.POINTER(I), ctypes.POINTER(I), ctypes.POINTER(I), P,
                                  I64, ctypes.POINTER(I64)]
    L.gqa_decode_plan.restype = I
    L.gqa_decode_selftest_timeout.argtypes = [ctypes.c_uint, P]
    L.gqa_decode_selftest_timeout.restype = I
    L.gqa_cross_workspace_size.argtypes = [D]
    L.gqa_cross_workspace_size.restype = SZ
    L.gqa_cross_attn.argtypes = [D, P, P, P, P, P, P, P, SZ, P]
    L.gqa_cross_attn.restype = I
    L.gqa_prefix_workspace_size.argtypes = [D, I]
    L.gqa_prefix_workspace_size.restype = SZ
    L.gqa_prefix_attn.argtypes = [D, P, P, P, P, I, P, P, P, P, P, P, SZ, P]
    L.gqa_prefix_attn.restype = I
    L.gqa_shared_keys_plan.argtypes = [D, I, I, P, I, ctypes.POINTER(I), ctypes.POINTER(I), P, P, I64,
                                       ctypes.POINTER(I64)]
    L.gqa_shared_keys_plan.restype = I
    G, R, F64 = ctypes.POINTER(gqa_pages_t), ctypes.POINTER(gqa_rotary_t), ctypes.c_double
    L.gqa_rotary_turns.argtypes = [I, F64, I, F64, I, F64, F64, P]
    L.gqa_rotary_turns.restype = I
    L.gqa_rotary_apply.argtypes = [R, P, P, I64, I, I, I, P, I64, P, I64, P]
    L.gqa_rotary_apply.restype = I
    L.gqa_paged_append.argtypes = [D, G, R, P, P, P, I64, P, I64, P, I64, P, P, P, P, P, P, P]
    L.gqa_paged_append.restype = I
    L.gqa_tree_from_parents.argtypes = [I, I, I, P, P, P, P, P, P]
    L.gqa_tree_from_parents.restype = I
    L.gqa_tree_workspace_size.argtypes = [D, G]
    L.gqa_tree_workspace_size.restype = SZ
    L.gqa_tree_attn.argtypes = [D, G, P, P, P, P, P, P, P, P, P, P, SZ, P]
    L.gqa_tree_attn.restype = I
    L.gqa_paged_keep.argtypes = [D, G, P, P, P, P, P, P, I, P, P, P]
    L.gqa_paged_keep.restype = I
    return L


def header_functions(header: str = HEADER):
    """Names of the functions a header (``include/gqa_decode.h``) declares."""
    with open(header) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gqa_[a-z_0-9]+)\s*\(", text)))


def _check(status: int, where: str):
    if status != GQA_OK:
        raise GQAError(status, where)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(dtype, allowed):
    import torch

    code = {torch.bfloat16: GQA_DTYPE_BF16, torch.float32: GQA_DTYPE_FP32, torch.float16: GQA_DTYPE_FP16}.get(dtype)
    if code is None or code not in allowed:
        raise ValueError(f"unsupported dtype {dtype}")
    return code


def _reduction_code(reduction) -> int:
    if isinstance(reduction, str):
        if reduction not in _REDUCTIONS:
            raise ValueError(f"reduction must be one of {sorted(_REDUCTIONS)}")
        return _REDUCTIONS[reduction]
    return int(reduction)


def make_desc(q, k_cache, *, scale: float = 0.0, causal: bool = False, out_dtype=None,
              reduction="auto") -> gqa_desc_t:
    """Problem description from q [B, nq, Hq, d] and a cache [B, S_max, Hkv, d]
    (inputs bf16 or fp16; out_dtype fp32 or the inputs' type, the default;
    reduction "auto", "combine" or "cluster", see gqa_reduction_t)."""
    import torch

    B, nq, Hq, d = q.shape
    Bk, s_max, Hkv, dk = k_cache.shape
    if Bk != B or dk != d:
        raise ValueError(f"q {tuple(q.shape)} and cache {tuple(k_cache.shape)} disagree")
    if out_dtype is None:
        out_dtype = q.dtype
    code = _dtype_code(out_dtype, (GQA_DTYPE_BF16, GQA_DTYPE_FP32, GQA_DTYPE_FP16))
    in_code = _dtype_code(q.dtype, (GQA_DTYPE_BF16, GQA_DTYPE_FP16))
    return gqa_desc_t(B, nq, Hq, Hkv, d, s_max, float(scale), int(bool(causal)), code, in_code,
                      _reduction_code(reduction))


def _inputs_ok(q, k_cache, v_cache, seqlens):
    import torch

    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype not in (torch.bfloat16, torch.float16) or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 or fp16 tensor, all three of one type")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    if seqlens.dtype != torch.int32 or not seqlens.is_contiguous():
        raise ValueError("seqlens must be a contiguous int32 tensor")


def gqa_decode_workspace_size(q, k_cache, num_splits: int = 0, *, causal: bool = False, out_dtype=None,
                              reduction="auto") -> int:
    desc = make_desc(q, k_cache, causal=causal, out_dtype=out_dtype, reduction=reduction)
    return int(lib().gqa_decode_workspace_size(ctypes.byref(desc), int(num_splits)))


def gqa_decode_attn(q, k_cache, v_cache, seqlens, out, lse=None, num_splits: int = 0, workspace=None, *,
                    scale: float = 0.0, causal: bool = False, reduction="auto", stream=None) -> None:
    """Full decode into ``out`` (and ``lse``); see gqa_decode_attn in the C header."""
    _inputs_ok(q, k_cache, v_cache, seqlens)
    desc = make_desc(q, k_cache, scale=scale, causal=causal, out_dtype=out.dtype, reduction=reduction)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().gqa_decode_attn(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens),
                               _ptr(out), _ptr(lse), int(num_splits), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "gqa_decode_attn")


def gqa_decode_attn_static_workspace(q, k_cache, v_cache, seqlens, out, lse=None, num_splits: int = 0, *,
                                     scale: float = 0.0, causal: bool = False, reduction="auto",
                                     stream=None) -> None:
    """gqa_decode_attn using the library's static device workspace instead of a
    caller-allocated one (for callers that cannot allocate; see the C header)."""
    _inputs_ok(q, k_cache, v_cache, seqlens)
    desc = make_desc(q, k_cache, scale=scale, causal=causal, out_dtype=out.dtype, reduction=reduction)
    rc = lib().gqa_decode_attn_static_workspace(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                                _ptr(seqlens), _ptr(out), _ptr(lse), int(num_splits),
                                                _stream(stream))
    _check(rc, "gqa_decode_attn_static_workspace")


def gqa_decode_attn_split(q, k_cache, v_cache, seqlens, out, lse=None, num_splits: int = 0, workspace=None, *,
                          scale: float = 0.0, causal: bool = False, reduction="auto", stream=None) -> None:
    """The decode-kernel half of gqa_decode_attn (see the C header)."""
    _inputs_ok(q, k_cache, v_cache, seqlens)
    desc = make_desc(q, k_cache, scale=scale, causal=causal, out_dtype=out.dtype, reduction=reduction)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().gqa_decode_attn_split(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens),
                                     _ptr(out), _ptr(lse), int(num_splits), _ptr(workspace), ws_bytes,
                                     _stream(stream))
    _check(rc, "gqa_decode_attn_split")


def gqa_decode_attn_merge(q, k_cache, out, lse=None, num_splits: int = 0, workspace=None, *, causal: bool = False,
                          reduction="auto", stream=None) -> None:
    """The combine half of gqa_decode_attn over the workspace of gqa_decode_attn_split."""
    desc = make_desc(q, k_cache, causal=causal, out_dtype=out.dtype, reduction=reduction)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().gqa_decode_attn_merge(ctypes.byref(desc), _ptr(out), _ptr(lse), int(num_splits), _ptr(workspace),
                                     ws_bytes, _stream(stream))
    _check(rc, "gqa_decode_attn_merge")


def gqa_decode_splitkv(q, k_cache, v_cache, seqlens, num_splits: int, o_part, lse_part, *, scale: float = 0.0,
                       causal: bool = False, stream=None) -> None:
    """Per-split partials (o_part fp32 [S, B, nq, Hq, d], lse_part fp32 [S, B, nq, Hq])."""
    _inputs_ok(q, k_cache, v_cache, seqlens)
    desc = make_desc(q, k_cache, scale=scale, causal=causal)
    rc = lib().gqa_decode_splitkv(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens),
                                  int(num_splits), _ptr(o_part), _ptr(lse_part), _stream(stream))
    _check(rc, "gqa_decode_splitkv")


def gqa_decode_combine(o_part, lse_part, out, lse=None, stream=None) -> None:
    """Merge partials o_part fp32 [S, rows..., d] / lse_part [S, rows...] into out [rows..., d]."""
    import torch

    S, d = o_part.shape[0], o_part.shape[-1]
    rows = lse_part[0].numel()
    code = _dtype_code(out.dtype, (GQA_DTYPE_BF16, GQA_DTYPE_FP32, GQA_DTYPE_FP16))
    rc = lib().gqa_decode_combine(_ptr(o_part), _ptr(lse_part), int(S), int(rows), int(d), _ptr(out), code,
                                  _ptr(lse), _stream(stream))
    _check(rc, "gqa_decode_combine")


def gqa_decode_get_error(clear: bool = True) -> int:
    return int(lib().gqa_decode_get_error(1 if clear else 0))


def gqa_status_string(status: int) -> str:
    try:
        return lib().gqa_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def gqa_decode_plan(desc: gqa_desc_t, seqlens_host, num_splits: int = 0, sm_count: int = 0, max_items=None):
    """Work decomposition as (num_ctas, plan_mode, num_slots, items int32 [n, 8])."""
    import numpy as np

    sl = np.ascontiguousarray(np.asarray(seqlens_host, dtype=np.int32))
    nc, mode, slots = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    n = ctypes.c_int64()
    L = lib()
    rc = L.gqa_decode_plan(ctypes.byref(desc), sl.ctypes.data, int(num_splits), int(sm_count), ctypes.byref(nc),
                           ctypes.byref(mode), ctypes.byref(slots), None, 0, ctypes.byref(n))
    _check(rc, "gqa_decode_plan")
    cap = n.value if max_items is None else min(n.value, max_items)
    items = np.zeros((max(cap, 1), 8), dtype=np.int32)
    rc = L.gqa_decode_plan(ctypes.byref(desc), sl.ctypes.data, int(num_splits), int(sm_count), ctypes.byref(nc),
                           ctypes.byref(mode), ctypes.byref(slots), items.ctypes.data, cap, ctypes.byref(n))
    _check(rc, "gqa_decode_plan")
    return nc.value, mode.value, slots.value, items[:cap]


def gqa_decode_selftest_timeout(timeout_us: int, stream=None) -> None:
    _check(lib().gqa_decode_selftest_timeout(int(timeout_us), _stream(stream)), "gqa_decode_selftest_timeout")


def decode(q, k_cache, v_cache, seqlens, *, num_splits: int = 0, scale: float = 0.0, causal: bool = False,
           out_dtype=None, reduction="auto", stream=None):
    """Allocates out / lse / workspace with torch and calls gqa_decode_attn."""
    import torch

    out_dtype = q.dtype if out_dtype is None else out_dtype
    B, nq, Hq, d = q.shape
    out = torch.empty(B, nq, Hq, d, dtype=out_dtype, device=q.device)
    lse = torch.empty(B, nq, Hq, dtype=torch.float32, device=q.device)
    ws_bytes = gqa_decode_workspace_size(q, k_cache, num_splits, causal=causal, out_dtype=out_dtype,
                                         reduction=reduction)
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device) if ws_bytes else None
    gqa_decode_attn(q, k_cache, v_cache, seqlens, out, lse, num_splits, ws, scale=scale, causal=causal,
                    reduction=reduction, stream=stream)
    return out, lse


_TYPE_CODES = None


def _type_codes():
    """gqa_dtype_t of each torch type (built on first use: torch is imported then)."""
    global _TYPE_CODES
    if _TYPE_CODES is None:
        import torch

        _TYPE_CODES = {torch.bfloat16: GQA_DTYPE_BF16, torch.float16: GQA_DTYPE_FP16, torch.float32: GQA_DTYPE_FP32}
    return _TYPE_CODES


def _shared_desc(q, k, out_dtype, scale, causal):
    """Description of q [B, nq, Hq, d] against k [B, S_max, Hkv, d], and q's device index."""
    codes = _type_codes()
    in_code = codes.get(q.dtype)
    if in_code != GQA_DTYPE_BF16 and in_code != GQA_DTYPE_FP16:
        raise ValueError(f"q must be bf16 or fp16, not {q.dtype}")
    out_code = in_code if out_dtype is None else codes.get(out_dtype)
    if out_code is None:
        raise ValueError(f"unsupported output type {out_dtype}")
    device = q.get_device()
    if device < 0:
        raise ValueError("q must be a CUDA tensor")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and the keys must have four dimensions")
    B, nq, Hq, d = q.shape
    Bk, s_max, Hkv, dk = k.shape
    if Bk != B or dk != d:
        raise ValueError(f"q {tuple(q.shape)} and keys {tuple(k.shape)} disagree")
    return gqa_desc_t(B, nq, Hq, Hkv, d, s_max, scale, 1 if causal else 0, out_code, in_code, GQA_REDUCE_AUTO), device


def _check_call(device, q, keys, lengths, out, lse, workspace, stream):
    """Types, layouts and devices of a call's tensors (their shapes beyond q and
    k are the caller's to check).  Returns the raw stream."""
    import torch

    dtype = q.dtype
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    for t in keys:
        if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != device:
            raise ValueError("keys and values must be contiguous, of q's type and on its device")
    for t, n in lengths:
        if t.dtype is not torch.int32 or t.numel() != n or not t.is_contiguous() or t.get_device() != device:
            raise ValueError(f"lengths must be {n} contiguous int32 on q's device")
    if out.shape != q.shape or not out.is_contiguous() or out.get_device() != device:
        raise ValueError("out must be contiguous, of q's shape and on its device")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != q.shape[:3] or not lse.is_contiguous()
                            or lse.get_device() != device):
        raise ValueError("lse must be contiguous fp32 [B, nq, Hq] on q's device")
    if workspace is not None and (not workspace.is_contiguous() or workspace.get_device() != device):
        raise ValueError("workspace must be contiguous and on q's device")
    return _raw_stream(stream, device)


def _raw_stream(stream, device) -> int:
    """The cudaStream_t of a call on `device` (None: torch's current stream there)."""
    import torch

    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if not hasattr(stream, "cuda_stream"):
        return int(stream)
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, not on cuda:{device}")
    return stream.cuda_stream


def _on_device(device, fn, *args):
    """fn(*args) with `device` current (the C library computes on the current device)."""
    import torch

    if torch._C._cuda_getDevice() == device:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _bytes_of(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def gqa_cross_workspace_size(q, k, *, out_dtype=None) -> int:
    """Bytes gqa_cross_attn needs for q [B, nq, Hq, d] against keys [B, S_max, Hkv, d]."""
    desc, device = _shared_desc(q, k, out_dtype, 0.0, False)
    return int(_on_device(device, lib().gqa_cross_workspace_size, ctypes.byref(desc)))


def gqa_cross_attn(q, k, v, kv_lens, out, lse=None, workspace=None, *, scale: float = 0.0, stream=None) -> None:
    """Cross attention into ``out`` (and ``lse``); see gqa_cross_attn in ``include/gqa_shared_keys.h``."""
    desc, device = _shared_desc(q, k, out.dtype, scale, False)
    if v.shape != k.shape:
        raise ValueError("k and v shapes differ")
    raw = _check_call(device, q, (k, v), ((kv_lens, desc.batch),), out, lse, workspace, stream)
    rc = _on_device(device, lib().gqa_cross_attn, ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                    kv_lens.data_ptr(), out.data_ptr(), _ptr(lse), _ptr(workspace), _bytes_of(workspace), raw)
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_cross_attn")


def gqa_prefix_workspace_size(q, k_prefix, k_cache, *, causal: bool = False, out_dtype=None) -> int:
    """Bytes gqa_prefix_attn needs for a decode step q, k_cache behind k_prefix [max_prefix, Hkv, d]."""
    desc, device = _shared_desc(q, k_cache, out_dtype, 0.0, causal)
    return int(_on_device(device, lib().gqa_prefix_workspace_size, ctypes.byref(desc), int(k_prefix.shape[0])))


def gqa_prefix_attn(q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, seqlens, out, lse=None, workspace=None, *,
                    scale: float = 0.0, causal: bool = False, stream=None) -> None:
    """Decode attention behind a shared prefix into ``out`` (and ``lse``); see
    gqa_prefix_attn in ``include/gqa_shared_keys.h``."""
    desc, device = _shared_desc(q, k_cache, out.dtype, scale, causal)
    if v_cache.shape != k_cache.shape or v_prefix.shape != k_prefix.shape:
        raise ValueError("k and v shapes differ")
    if k_prefix.dim() != 3 or k_prefix.shape[1:] != k_cache.shape[2:]:
        raise ValueError(f"prefix {tuple(k_prefix.shape)} and cache {tuple(k_cache.shape)} disagree")
    raw = _check_call(device, q, (k_prefix, v_prefix, k_cache, v_cache), ((prefix_len, 1), (seqlens, desc.batch)), out,
                      lse, workspace, stream)
    rc = _on_device(device, lib().gqa_prefix_attn, ctypes.byref(desc), q.data_ptr(), k_prefix.data_ptr(),
                    v_prefix.data_ptr(), prefix_len.data_ptr(), k_prefix.shape[0], k_cache.data_ptr(),
                    v_cache.data_ptr(), seqlens.data_ptr(), out.data_ptr(), _ptr(lse), _ptr(workspace),
                    _bytes_of(workspace), raw)
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_prefix_attn")


def _torch_stream(stream, device):
    import torch

    if stream is None:
        return torch.cuda.current_stream(device)
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)


def _allocate(q, out_dtype, workspace_bytes, stream):
    """out, lse and a workspace of the call's own stream, so that the caching
    allocator hands none of them on while that stream still uses it."""
    import torch

    with torch.cuda.stream(_torch_stream(stream, q.device)):
        out = torch.empty(q.shape, dtype=q.dtype if out_dtype is None else out_dtype, device=q.device)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        ws = torch.empty(workspace_bytes, dtype=torch.uint8, device=q.device) if workspace_bytes else None
    return out, lse, ws


def cross_attention(q, k, v, kv_lens, *, scale: float = 0.0, out_dtype=None, stream=None):
    """Allocates out / lse / workspace with torch and calls gqa_cross_attn."""
    out, lse, ws = _allocate(q, out_dtype, gqa_cross_workspace_size(q, k, out_dtype=out_dtype), stream)
    gqa_cross_attn(q, k, v, kv_lens, out, lse, ws, scale=scale, stream=stream)
    return out, lse


def prefix_decode(q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, seqlens, *, scale: float = 0.0,
                  causal: bool = False, out_dtype=None, stream=None):
    """Allocates out / lse / workspace with torch and calls gqa_prefix_attn."""
    ws_bytes = gqa_prefix_workspace_size(q, k_prefix, k_cache, causal=causal, out_dtype=out_dtype)
    out, lse, ws = _allocate(q, out_dtype, ws_bytes, stream)
    gqa_prefix_attn(q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, seqlens, out, lse, ws, scale=scale,
                    causal=causal, stream=stream)
    return out, lse


def gqa_shared_keys_plan(desc: gqa_desc_t, kv_lens_host, prefix_len: int = 0, max_prefix: int = 0,
                         sm_count: int = 0):
    """The tiled kernel's decomposition as (num_ctas, every_piece, info int32 [2, 4], items int32 [n, 9]);
    see gqa_shared_keys_plan in ``include/gqa_shared_keys.h``."""
    import numpy as np

    sl = np.ascontiguousarray(np.asarray(kv_lens_host, dtype=np.int32))
    nc, every, n = ctypes.c_int(), ctypes.c_int(), ctypes.c_int64()
    info = np.zeros((2, 4), dtype=np.int32)

    def call(items, cap):
        _check(lib().gqa_shared_keys_plan(ctypes.byref(desc), int(prefix_len), int(max_prefix), sl.ctypes.data,
                                          int(sm_count), ctypes.byref(nc), ctypes.byref(every), info.ctypes.data,
                                          None if items is None else items.ctypes.data, cap, ctypes.byref(n)),
               "gqa_shared_keys_plan")

    call(None, 0)
    items = np.zeros((n.value, 9), dtype=np.int32)
    call(items, n.value)
    return nc.value, bool(every.value), info, items


# ------------------------------------------------------- include/gqa_paged.h
# A step of a few tokens is shorter on the GPU than calls marshalled here would be,
# so what follows goes through csrc/paged_binding.cpp, which looks at the tensors.
def rotary_turns(dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                 original_length: int = 0, slow: float = 1.0, fast: float = 32.0, device=None):
    """The table the rotation turns by, int64 [dim / 2] (the bits of the C table's
    uint64) on ``device``; scaling "none", "linear", "base" or "parts", see
    gqa_rotary_scaling_t in ``include/gqa_paged.h``."""
    import torch

    if scaling not in _ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROTARY_SCALINGS)}")
    turns = torch.empty(max(int(dim) // 2, 1), dtype=torch.int64)
    _check(lib().gqa_rotary_turns(int(dim), float(base), _ROTARY_SCALINGS[scaling], float(factor),
                                  int(original_length), float(slow), float(fast), turns.data_ptr()),
           "gqa_rotary_turns")
    return turns if device is None else turns.to(device)


_binding, _bound = None, None


def _paged():
    """csrc/paged_binding.cpp, calling the loaded library."""
    global _binding, _bound
    if _bound is None or _bound is not _lib:
        with _lock:
            if _binding is None:
                import torch  # noqa: F401  (whose libraries it is linked against)

                path = binding_path()
                if not os.path.exists(path):
                    raise RuntimeError(f"binding of the paged calls not built ({path}); run "
                                       "gqa_decode_blackwell_gb300.build.build() or __graft_entry__.build()")
                loader = importlib.machinery.ExtensionFileLoader("_paged_binding", path)
                _binding = importlib.util.module_from_spec(importlib.util.spec_from_loader("_paged_binding", loader))
        L = lib()
        _binding.use(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.gqa_rotary_apply, L.gqa_paged_append, L.gqa_tree_from_parents, L.gqa_tree_workspace_size, L.gqa_tree_attn,
            L.gqa_paged_keep)))
        _bound = L
    return _binding


def gqa_rotary_apply(x, positions, turns, out, *, interleaved: bool = False, inverse: bool = False,
                     magnitude: float = 0.0, stream=None) -> None:
    """Rotates x [..., heads, d] to positions int32 [...] into ``out`` (x itself, or
    apart from it); see gqa_rotary_apply in ``include/gqa_paged.h``.  No gradient is
    recorded (``rotary`` records it)."""
    if stream is not None:
        stream = _raw_stream(stream, x.get_device())
    rc = _paged().rotary_apply(x, positions, turns, out, interleaved, inverse, magnitude, stream)
    if rc:
        raise GQAError(rc, "gqa_rotary_apply")


_rotation = None


def _recorded_rotation():
    """The rotation as autograd records it: linear, so that its gradient is the inverse
    rotation of the incoming one (of the same magnitude)."""
    global _rotation
    if _rotation is None:
        import torch

        class Rotation(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, positions, turns, interleaved, inverse, magnitude):
                out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
                gqa_rotary_apply(x, positions, turns, out, interleaved=interleaved, inverse=inverse, magnitude=magnitude)
                ctx.save_for_backward(positions, turns)
                ctx.how = interleaved, inverse, magnitude
                return out

            @staticmethod
            def backward(ctx, grad):
                positions, turns = ctx.saved_tensors
                interleaved, inverse, magnitude = ctx.how
                grad = rotary(grad.contiguous(), positions, turns, interleaved=interleaved, inverse=not inverse,
                              magnitude=magnitude)
                return grad, None, None, None, None, None

        _rotation = Rotation
    return _rotation


def rotary(x, positions, turns, *, interleaved: bool = False, inverse: bool = False, magnitude: float = 0.0,
           stream=None):
    """Allocates the result with torch and calls gqa_rotary_apply.  Differentiable in
    x: the backward pass reads positions and turns again, which have to stay as they
    are until then."""
    import torch

    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if stream is not None:
        _raw_stream(stream, x.get_device())  # refuses another device's
    with torch.cuda.stream(_torch_stream(stream, x.device)):
        if x.requires_grad and torch.is_grad_enabled():  # (recorded on the stream it runs on: the backward pass's too)
            return _recorded_rotation().apply(x, positions, turns, interleaved, inverse, magnitude)
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    gqa_rotary_apply(x, positions, turns, out, interleaved=interleaved, inverse=inverse, magnitude=magnitude,
                     stream=stream)
    return out


def gqa_paged_append(q, k, v, q_out, k_cache, v_cache, page_table, seqlens, *, new_lens=None, positions=None,
                     turns=None, interleaved: bool = False, magnitude: float = 0.0, stream=None) -> None:
    """Rotates the new tokens' q [B, nq, Hq, d] into ``q_out`` and puts k (rotated)
    and v [B, nq, Hkv, d] into the paged caches; q, k and v may be views of one
    tensor, q and q_out may be None, turns None rotates nothing.  See
    gqa_paged_append in ``include/gqa_paged.h``."""
    if stream is not None:
        stream = _raw_stream(stream, k.get_device())
    rc = _paged().paged_append(q, k, v, q_out, k_cache, v_cache, page_table, seqlens, new_lens, positions, turns,
                               interleaved, magnitude, stream)
    if rc:
        raise GQAError(rc, "gqa_paged_append")


def gqa_tree_from_parents(parents, seqlens, tree, positions=None, *, new_lens=None, max_seqlen: int = 1 << 30,
                          stream=None) -> None:
    """The drafts' tree of parents int32 [B, nq] as bits, int32 [B, nq, ceil(nq / 32)],
    and their positions int32 [B, nq]; see gqa_tree_from_parents in
    ``include/gqa_paged.h``."""
    if stream is not None:
        stream = _raw_stream(stream, parents.get_device())
    rc = _paged().tree_from_parents(parents, seqlens, tree, positions, new_lens, max_seqlen, stream)
    if rc:
        raise GQAError(rc, "gqa_tree_from_parents")


def gqa_tree_workspace_size(q, k_cache, page_table, *, out_dtype=None) -> int:
    """Bytes gqa_tree_attn needs for q [B, nq, Hq, d] over the paged caches."""
    code = -1 if out_dtype is None else _dtype_code(out_dtype, (GQA_DTYPE_BF16, GQA_DTYPE_FP32, GQA_DTYPE_FP16))
    return _paged().tree_workspace_size(q, k_cache, page_table, code)


def gqa_tree_attn(q, k_cache, v_cache, page_table, seqlens, out, lse=None, workspace=None, *, new_lens=None,
                  tree=None, causal: bool = False, scale: float = 0.0, stream=None) -> None:
    """Attention of new tokens over the paged caches into ``out`` (and ``lse``); see
    gqa_tree_attn in ``include/gqa_paged.h``."""
    if stream is not None:
        stream = _raw_stream(stream, q.get_device())
    rc = _paged().tree_attn(q, k_cache, v_cache, page_table, seqlens, out, lse, workspace, new_lens, tree, causal, scale,
                            stream)
    if rc:
        raise GQAError(rc, "gqa_tree_attn")


def tree_attention(q, k_cache, v_cache, page_table, seqlens, *, new_lens=None, tree=None, causal: bool = False,
                   scale: float = 0.0, out_dtype=None, stream=None):
    """Allocates out / lse / workspace with torch and calls gqa_tree_attn."""
    ws_bytes = gqa_tree_workspace_size(q, k_cache, page_table, out_dtype=out_dtype)
    out, lse, ws = _allocate(q, out_dtype, ws_bytes, stream)
    gqa_tree_attn(q, k_cache, v_cache, page_table, seqlens, out, lse, ws, new_lens=new_lens, tree=tree, causal=causal,
                  scale=scale, stream=stream)
    return out, lse


def gqa_paged_keep(k_cache, v_cache, page_table, seqlens, path, keep_lens, seqlens_out=None, *, tokens: int,
                   new_lens=None, stream=None) -> None:
    """Moves each sequence's accepted branch, path int32 [B, n] of which keep_lens
    [B] count, together behind the positions before its new tokens (``tokens`` of
    them, or new_lens); seqlens_out int32 [B] gets the new lengths and may be
    seqlens.  See gqa_paged_keep in ``include/gqa_paged.h``."""
    if stream is not None:
        stream = _raw_stream(stream, k_cache.get_device())
    rc = _paged().paged_keep(k_cache, v_cache, page_table, seqlens, path, keep_lens, seqlens_out, new_lens, tokens, stream)
    if rc:
        raise GQAError(rc, "gqa_paged_keep")
