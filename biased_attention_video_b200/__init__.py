"""Python binding of libh3attn (biased, block-routed attention over MiniMax-H3's
packed sequence on B200).

Argument marshalling only: every step of the computation runs in the CUDA
library.  PyTorch supplies device memory and the current stream.  There is no
fallback: if libh3attn.so cannot be loaded, every call raises.

Tensors: q, k, v, o bf16 [H, S, d] contiguous CUDA; seg uint8 [S]; times
float32 [S]; kv_sel int32 [H, n_video_blocks, k].
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from . import build as _build

OK, EINVAL, EUNSUPPORTED, EALIGN, ECUDA, ETIMEOUT, EWORKSPACE, EDATA = 0, -1, -2, -3, -4, -5, -6, -7
SEG_TEXT, SEG_IMAGE_REF, SEG_AUDIO, SEG_GUIDE, SEG_OUTPUT = 0, 1, 2, 3, 4

# every symbol the C header declares
EXPORTS = ("h3attn_plan_init", "h3attn_workspace_bytes", "h3attn_pool", "h3attn_route", "h3attn_route_static",
           "h3attn_route_static_check",
           "h3attn_forward",
           "h3attn_dense_workspace_bytes", "h3attn_dense_biased", "h3attn_check", "h3attn_selftest_timeout", "h3attn_set_wait_polls",
           "h3attn_attend_host", "h3attn_merge", "h3attn_tail_workspace_bytes", "h3attn_tail_correct",
           "h3attn_qk8_workspace_bytes", "h3attn_quantize_qk", "h3attn_forward_qk8",
           "h3attn_cache_workspace_bytes", "h3attn_cache_append", "h3attn_cache_read", "h3attn_cache_forward",
           "h3attn_strerror")


class H3Error(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {lib().h3attn_strerror(code).decode()} ({code})")


class Plan(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("S", ctypes.c_int32), ("d", ctypes.c_int32), ("block", ctypes.c_int32),
                ("sparsity", ctypes.c_double), ("n_blocks", ctypes.c_int32), ("prefix_rows", ctypes.c_int32),
                ("first_video_block", ctypes.c_int32), ("n_forced", ctypes.c_int32),
                ("n_video_blocks", ctypes.c_int32), ("k", ctypes.c_int32)]

    def __repr__(self):
        return "Plan(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class Penalty(ctypes.Structure):
    _fields_ = [("strength", ctypes.c_float), ("window", ctypes.c_float), ("falloff", ctypes.c_float),
                ("cap", ctypes.c_float)]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("H", ctypes.c_int32), ("d", ctypes.c_int32), ("block", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("times", ctypes.c_void_p)]


class _BatchStruct(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("row_start", ctypes.c_void_p), ("length", ctypes.c_void_p), ("page_table", ctypes.c_void_p)]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("index", ctypes.c_void_p),
                ("n_pos", ctypes.c_int32), ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


DEFAULT_PENALTY = (2.0, 0.20, 0.25, 6.0)

_lib = None
_P = ctypes.c_void_p


def lib_path() -> str:
    return _build.LIB


def lib():
    """Load libh3attn.so (building it in-tree with nvcc if it is missing or stale)."""
    global _lib
    if _lib is None:
        path = _build.build()
        L = ctypes.CDLL(path)
        PP = ctypes.POINTER(Plan)
        L.h3attn_plan_init.argtypes = [PP, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_double, _P]
        L.h3attn_plan_init.restype = ctypes.c_int
        L.h3attn_workspace_bytes.argtypes = [PP]
        L.h3attn_workspace_bytes.restype = ctypes.c_size_t
        L.h3attn_pool.argtypes = [PP, _P, ctypes.c_int, ctypes.c_int, _P, _P]
        L.h3attn_pool.restype = ctypes.c_int
        L.h3attn_route.argtypes = [PP, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.h3attn_route.restype = ctypes.c_int
        L.h3attn_route_static.argtypes = [PP, _P, _P, _P, _P]
        L.h3attn_route_static.restype = ctypes.c_int
        L.h3attn_route_static_check.argtypes = [_P]
        L.h3attn_route_static_check.restype = ctypes.c_int
        L.h3attn_forward.argtypes = [PP, _P, _P, _P, _P, _P, ctypes.POINTER(Penalty), _P, _P, _P, _P,
                                     ctypes.c_size_t, _P]
        L.h3attn_forward.restype = ctypes.c_int
        L.h3attn_dense_workspace_bytes.argtypes = [ctypes.c_int]
        L.h3attn_dense_workspace_bytes.restype = ctypes.c_size_t
        L.h3attn_dense_biased.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P, _P,
                                          ctypes.POINTER(Penalty), _P, _P, _P, ctypes.c_size_t, _P]
        L.h3attn_dense_biased.restype = ctypes.c_int
        L.h3attn_attend_host.argtypes = [PP, _P, _P, _P, _P, _P, ctypes.POINTER(Penalty), _P, _P, _P, _P, _P, _P,
                                         _P, _P, _P, _P, _P, ctypes.c_size_t, ctypes.c_int, _P, _P, _P]
        L.h3attn_attend_host.restype = ctypes.c_int
        L.h3attn_merge.argtypes = [ctypes.c_int, ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_float),
                                   ctypes.c_int, ctypes.c_int, ctypes.c_int, _P, _P, _P]
        L.h3attn_merge.restype = ctypes.c_int
        L.h3attn_tail_workspace_bytes.argtypes = [PP]
        L.h3attn_tail_workspace_bytes.restype = ctypes.c_size_t
        L.h3attn_tail_correct.argtypes = [PP, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, ctypes.c_size_t, _P]
        L.h3attn_tail_correct.restype = ctypes.c_int
        L.h3attn_qk8_workspace_bytes.argtypes = [PP]
        L.h3attn_qk8_workspace_bytes.restype = ctypes.c_size_t
        L.h3attn_quantize_qk.argtypes = [PP, _P, _P, _P, ctypes.c_size_t, _P]
        L.h3attn_quantize_qk.restype = ctypes.c_int
        L.h3attn_forward_qk8.argtypes = [PP, _P, _P, _P, _P, _P, ctypes.POINTER(Penalty), _P, _P, _P, _P,
                                         ctypes.c_size_t, _P, ctypes.c_size_t, _P]
        L.h3attn_forward_qk8.restype = ctypes.c_int
        CP, BP, I64 = ctypes.POINTER(_CacheStruct), ctypes.POINTER(_BatchStruct), ctypes.c_int64
        L.h3attn_cache_workspace_bytes.argtypes = [CP, ctypes.c_int, ctypes.c_int, ctypes.c_int]
        L.h3attn_cache_workspace_bytes.restype = ctypes.c_size_t
        L.h3attn_cache_append.argtypes = [CP, BP, _P, I64, I64, _P, I64, I64, ctypes.POINTER(_RopeStruct), _P, _P,
                                          ctypes.c_size_t, _P]
        L.h3attn_cache_append.restype = ctypes.c_int
        L.h3attn_cache_read.argtypes = [CP, BP, _P, _P, _P, ctypes.c_size_t, _P]
        L.h3attn_cache_read.restype = ctypes.c_int
        L.h3attn_cache_forward.argtypes = [CP, BP, ctypes.c_int, ctypes.c_int, _P, I64, I64, ctypes.c_int,
                                           ctypes.POINTER(Penalty), _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.h3attn_cache_forward.restype = ctypes.c_int
        L.h3attn_check.argtypes = [_P, _P]
        L.h3attn_check.restype = ctypes.c_int
        L.h3attn_set_wait_polls.argtypes = [ctypes.c_uint32]
        L.h3attn_set_wait_polls.restype = ctypes.c_int
        L.h3attn_selftest_timeout.argtypes = [_P, ctypes.c_uint32, _P]
        L.h3attn_selftest_timeout.restype = ctypes.c_int
        L.h3attn_strerror.argtypes = [ctypes.c_int]
        L.h3attn_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _raise(code: int, what: str):
    if code != OK:
        raise H3Error(code, what)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _dptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_qkv(*ts):
    for t in ts:
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous() and t.dim() == 3):
            raise ValueError("q/k/v/o must be contiguous CUDA bf16 [H, S, d]")


def _pen(pen) -> Optional[Penalty]:
    if pen is None:
        return None
    if isinstance(pen, Penalty):
        return pen
    s, w, f, c = pen
    return Penalty(s, w, f, c)


def plan(H: int, S: int, d: int, seg_host, sparsity: float = 0.0, block: int = 64) -> Plan:
    """Block plan from the host copy of seg (numpy or CPU tensor, uint8 [S])."""
    seg = np.ascontiguousarray(seg_host.cpu().numpy() if isinstance(seg_host, torch.Tensor) else seg_host,
                               dtype=np.uint8)
    if seg.shape != (S,):
        raise ValueError("seg must have S entries")
    p = Plan()
    _raise(lib().h3attn_plan_init(ctypes.byref(p), H, S, d, block, sparsity, seg.ctypes.data), "plan_init")
    return p


def workspace(p: Plan, device="cuda") -> torch.Tensor:
    n = lib().h3attn_workspace_bytes(ctypes.byref(p))
    if n == 0:
        raise H3Error(EINVAL, "workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def dense_workspace(S: int, device="cuda") -> torch.Tensor:
    return torch.zeros(lib().h3attn_dense_workspace_bytes(S), dtype=torch.uint8, device=device)


def pool(p: Plan, x: torch.Tensor, first_block: int = 0, n_out: Optional[int] = None, out=None, stream=None):
    """Block means (fp32 [H, n_out, d]) of blocks [first_block, first_block + n_out)."""
    _check_qkv(x)
    n_out = p.n_blocks - first_block if n_out is None else n_out
    if out is None:
        out = torch.empty((p.H, n_out, p.d), dtype=torch.float32, device=x.device)
    _raise(lib().h3attn_pool(ctypes.byref(p), x.data_ptr(), first_block, n_out, out.data_ptr(), _stream(stream)),
           "pool")
    return out


def route(p: Plan, q: torch.Tensor, k: torch.Tensor, ws: torch.Tensor, kv_sel=None, stream=None) -> torch.Tensor:
    """Routed key blocks int32 [H, n_video_blocks, k] (absolute block ids, ascending)."""
    _check_qkv(q, k)
    if kv_sel is None:
        kv_sel = torch.empty((p.H, p.n_video_blocks, p.k), dtype=torch.int32, device=q.device)
    _raise(lib().h3attn_route(ctypes.byref(p), q.data_ptr(), k.data_ptr(), kv_sel.data_ptr(), ws.data_ptr(),
                              ws.numel(), _stream(stream)), "route")
    return kv_sel


def route_static(p: Plan, q: torch.Tensor, k: torch.Tensor, kv_sel=None, stream=None) -> torch.Tensor:
    """Same result as route(), for callers that cannot allocate device memory: the
    pooled centroids live in a fixed 64 MiB array inside the library (no workspace).
    The output buffer kv_sel may be passed in; concurrent calls share that array."""
    _check_qkv(q, k)
    if kv_sel is None:
        kv_sel = torch.empty((p.H, p.n_video_blocks, p.k), dtype=torch.int32, device=q.device)
    _raise(lib().h3attn_route_static(ctypes.byref(p), q.data_ptr(), k.data_ptr(), kv_sel.data_ptr(),
                                     _stream(stream)), "route_static")
    return kv_sel


def route_static_check(stream=None) -> int:
    """Synchronise and return (then clear) the status word of the route_static calls on the current device."""
    return lib().h3attn_route_static_check(_stream(stream))


def forward(p: Plan, q, k, v, seg, times, pen=DEFAULT_PENALTY, kv_sel=None, ws=None, out=None,
            lse: bool | torch.Tensor = False, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention over the routed tiles (kv_sel None = dense) with the temporal penalty (pen None = off)."""
    _check_qkv(q, k, v)
    if ws is None:
        ws = workspace(p, q.device)
    o = torch.empty_like(q) if out is None else out
    lse_t = lse if isinstance(lse, torch.Tensor) else (
        torch.empty((p.H, p.S), dtype=torch.float32, device=q.device) if lse else None)
    pn = _pen(pen)
    _raise(lib().h3attn_forward(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), seg.data_ptr(),
                                _dptr(times), ctypes.byref(pn) if pn is not None else None, _dptr(kv_sel),
                                o.data_ptr(), _dptr(lse_t), ws.data_ptr(), ws.numel(), _stream(stream)), "forward")
    return o, lse_t


def qk8_workspace(p: Plan, device="cuda") -> torch.Tensor:
    """Scratch of the int8-QK path: codes and per-token scales of Q and K."""
    n = lib().h3attn_qk8_workspace_bytes(ctypes.byref(p))
    if n == 0:
        raise H3Error(EINVAL, "qk8_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _align256(x: int) -> int:
    return (x + 255) // 256 * 256


def quantize_qk(p: Plan, q, k, qk8_ws=None, stream=None):
    """Per-token int8 quantisation of Q and K (h3attn_quantize_qk).  Returns views of the scratch:
    (q8 int8 [H, S, d], k8 int8 [H, S, d], q_scale float32 [H, 64 n_blocks], k_scale float32 [H, 64 n_blocks])."""
    _check_qkv(q, k, k)
    if qk8_ws is None:
        qk8_ws = qk8_workspace(p, q.device)
    _raise(lib().h3attn_quantize_qk(ctypes.byref(p), q.data_ptr(), k.data_ptr(), qk8_ws.data_ptr(), qk8_ws.numel(),
                                    _stream(stream)), "quantize_qk")
    codes = p.H * p.S * p.d
    stride = p.n_blocks * 64
    o_k8 = _align256(codes)
    o_sq = o_k8 + _align256(codes)
    o_sk = o_sq + _align256(p.H * stride * 4)
    q8 = qk8_ws[:codes].view(torch.int8).view(p.H, p.S, p.d)
    k8 = qk8_ws[o_k8:o_k8 + codes].view(torch.int8).view(p.H, p.S, p.d)
    sq = qk8_ws[o_sq:o_sq + p.H * stride * 4].view(torch.float32).view(p.H, stride)
    sk = qk8_ws[o_sk:o_sk + p.H * stride * 4].view(torch.float32).view(p.H, stride)
    return q8, k8, sq, sk


def forward_qk8(p: Plan, q, k, v, seg, times, pen=DEFAULT_PENALTY, kv_sel=None, ws=None, qk8_ws=None, out=None,
                lse: bool | torch.Tensor = False, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """forward with Q and K quantised per token to int8 before the QK product (h3attn_forward_qk8)."""
    _check_qkv(q, k, v)
    if ws is None:
        ws = workspace(p, q.device)
    if qk8_ws is None:
        qk8_ws = qk8_workspace(p, q.device)
    o = torch.empty_like(q) if out is None else out
    lse_t = lse if isinstance(lse, torch.Tensor) else (
        torch.empty((p.H, p.S), dtype=torch.float32, device=q.device) if lse else None)
    pn = _pen(pen)
    _raise(lib().h3attn_forward_qk8(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), seg.data_ptr(),
                                    _dptr(times), ctypes.byref(pn) if pn is not None else None, _dptr(kv_sel),
                                    o.data_ptr(), _dptr(lse_t), ws.data_ptr(), ws.numel(), qk8_ws.data_ptr(),
                                    qk8_ws.numel(), _stream(stream)), "forward_qk8")
    return o, lse_t


def dense_biased(q, k, v, seg, times, pen=DEFAULT_PENALTY, ws=None, out=None, lse: bool = False, stream=None):
    """Dense attention with the temporal penalty on output -> guide pairs."""
    _check_qkv(q, k, v)
    H, S, d = q.shape
    if ws is None:
        ws = dense_workspace(S, q.device)
    o = torch.empty_like(q) if out is None else out
    lse_t = torch.empty((H, S), dtype=torch.float32, device=q.device) if lse else None
    pn = _pen(pen)
    _raise(lib().h3attn_dense_biased(H, S, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), seg.data_ptr(),
                                     _dptr(times), ctypes.byref(pn) if pn is not None else None, o.data_ptr(),
                                     _dptr(lse_t), ws.data_ptr(), ws.numel(), _stream(stream)), "dense_biased")
    return o, lse_t


def attend_host(p: Plan, q_host, k_host, v_host, seg_host, times_host, o_host, *, q, k, v, seg, times, o, ws,
                kv_sel=None, pen=DEFAULT_PENALTY, lse_host=None, lse=None, chunk_heads: int = 4, stream=None,
                copy_in_stream=None, copy_out_stream=None) -> None:
    """The whole call from (page-locked) host tensors, copies overlapped with the kernels per chunk of heads.

    Host tensors: q_host/k_host/v_host/o_host bf16 or int16 [H, S, d]; seg_host uint8 [S]; times_host float32 [S];
    device buffers q/k/v/o/seg/times (and kv_sel, lse) of the same shapes.  Streams are torch.cuda.Stream
    objects (None = the current stream)."""
    pn = _pen(pen)
    _raise(lib().h3attn_attend_host(
        ctypes.byref(p), q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(), seg_host.data_ptr(),
        _dptr(times_host), ctypes.byref(pn) if pn is not None else None, o_host.data_ptr(), _dptr(lse_host),
        q.data_ptr(), k.data_ptr(), v.data_ptr(), seg.data_ptr(), _dptr(times), _dptr(kv_sel), o.data_ptr(),
        _dptr(lse), ws.data_ptr(), ws.numel(), chunk_heads, _stream(stream), _stream(copy_in_stream),
        _stream(copy_out_stream)), "attend_host")


def merge(o_parts, lse_parts, log_w=None, out=None, lse: bool | torch.Tensor = False, stream=None):
    """Merge normalised partition results (forward outputs o [H, S, d] bf16 and lse [H, S] float32 over key
    sets) with multipliers exp(log_w[i]); returns (O, LSE or None)."""
    n = len(o_parts)
    if n != len(lse_parts) or n == 0:
        raise ValueError("o_parts and lse_parts must be non-empty and of equal length")
    _check_qkv(*o_parts)
    H, S, d = o_parts[0].shape
    for t in lse_parts:
        if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous() and tuple(t.shape) == (H, S)):
            raise ValueError("lse parts must be contiguous CUDA float32 [H, S]")
    o = torch.empty_like(o_parts[0]) if out is None else out
    lse_t = lse if isinstance(lse, torch.Tensor) else (
        torch.empty((H, S), dtype=torch.float32, device=o.device) if lse else None)
    op = (_P * n)(*[t.data_ptr() for t in o_parts])
    lp = (_P * n)(*[t.data_ptr() for t in lse_parts])
    lw = None if log_w is None else (ctypes.c_float * n)(*[float(x) for x in log_w])
    _raise(lib().h3attn_merge(n, op, lp, lw, H, S, d, o.data_ptr(), _dptr(lse_t), _stream(stream)), "merge")
    return o, lse_t


def tail_workspace(p: Plan, device="cuda") -> torch.Tensor:
    n = lib().h3attn_tail_workspace_bytes(ctypes.byref(p))
    if n == 0:
        raise H3Error(EINVAL, "tail_workspace")
    return torch.empty(n, dtype=torch.uint8, device=device)


def tail_correct(p: Plan, v, kv_sel, o, lse, ws, tail_ws=None, stream=None) -> None:
    """Fold the routed-out video key blocks into (o, lse) as one pooled term per query block, in place.
    Call after route(p, q, k, ws, kv_sel) and forward(..., kv_sel, ws, out=o, lse=lse) with the same ws."""
    _check_qkv(v, o)
    tw = tail_workspace(p, v.device) if tail_ws is None else tail_ws
    _raise(lib().h3attn_tail_correct(ctypes.byref(p), v.data_ptr(), kv_sel.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                     ws.data_ptr(), ws.numel(), tw.data_ptr(), tw.numel(), _stream(stream)),
           "tail_correct")


# ------------------------------------------------------------- paged int8 cache


def _is(t, dtype, shape, dev: int) -> bool:
    """Contiguous, of this type, shape and device index (the checks of every call, cheapest form)."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _name(dev: int) -> str:
    return f"cuda:{dev}" if dev >= 0 else "cpu"


def _want(t, name: str, dtype, shape, dev: int):
    if not _is(t, dtype, shape, dev):
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on {_name(dev)}, not "
                         f"{t.dtype} {list(t.shape)} on {t.device}")
    return t


class Cache:
    """Paged int8 cache (h3attn_cache): k, v int8 [n_pages, H, 64, d]; k_scale, v_scale float32 [n_pages, H]; times
    float32 [n_pages, 64] or None.  ``empty`` allocates one; the tensors may also come from elsewhere."""

    __slots__ = ("_t", "_c")

    def __init__(self, k, v, k_scale, v_scale, times=None):
        if not (k.is_cuda and k.dtype == torch.int8 and k.dim() == 4 and k.shape[2] == 64 and k.is_contiguous()):
            raise ValueError("k must be contiguous CUDA int8 [n_pages, H, 64, d]")
        n, H, _, d = k.shape
        dev = k.get_device()
        _want(v, "v", torch.int8, k.shape, dev)
        _want(k_scale, "k_scale", torch.float32, (n, H), dev)
        _want(v_scale, "v_scale", torch.float32, (n, H), dev)
        if times is not None:
            _want(times, "times", torch.float32, (n, 64), dev)
        self._t = (k, v, k_scale, v_scale, times)
        self._c = _CacheStruct(n, H, d, 64, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                               _dptr(times))

    @classmethod
    def empty(cls, n_pages: int, H: int, d: int, times: bool = False, device="cuda") -> "Cache":
        k = torch.empty((n_pages, H, 64, d), dtype=torch.int8, device=device)
        s = torch.empty((2, n_pages, H), dtype=torch.float32, device=device)
        t = torch.full((n_pages, 64), float("nan"), device=device) if times else None
        return cls(k, torch.empty_like(k), s[0], s[1], t)

    k = property(lambda self: self._t[0])
    v = property(lambda self: self._t[1])
    k_scale = property(lambda self: self._t[2])
    v_scale = property(lambda self: self._t[3])
    times = property(lambda self: self._t[4])
    n_pages = property(lambda self: self._c.n_pages)
    H = property(lambda self: self._c.H)
    d = property(lambda self: self._c.d)
    device = property(lambda self: self._t[0].device)


class Rope:
    """Rotation table of appended keys (h3attn_rope): cos, sin float32 [n_pos, dim / 2]; index int32 [T], the table
    row of each appended row, or None for its position in the sequence."""

    __slots__ = ("_t", "_c")

    def __init__(self, cos, sin, index=None, interleaved: bool = False):
        if not (cos.dtype == torch.float32 and cos.dim() == 2 and cos.is_contiguous()):
            raise ValueError("cos must be contiguous float32 [n_pos, dim / 2]")
        _want(sin, "sin", torch.float32, cos.shape, cos.get_device())
        if index is not None:
            _want(index, "index", torch.int32, (index.numel(),), cos.get_device())
        self._t = (cos, sin, index)
        self._c = _RopeStruct(cos.data_ptr(), sin.data_ptr(), _dptr(index), cos.shape[0], 2 * cos.shape[1],
                              int(interleaved))


def cache_workspace(c: Cache, H: int, T: int, B: int) -> torch.Tensor:
    """Workspace of the cache calls for H query heads, T packed rows and B sequences."""
    n = lib().h3attn_cache_workspace_bytes(ctypes.byref(c._c), H, T, B)
    if n == 0:
        raise H3Error(EINVAL, "cache_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=c.device)


def _batch(dev: int, T: int, row_start, length, page_table) -> _BatchStruct:
    i32 = torch.int32
    if not (page_table.dim() == 2 and _is(page_table, i32, page_table.shape, dev)):
        raise ValueError(f"page_table must be contiguous int32 [B, max_pages] on cuda:{dev}")
    B, width = page_table.shape
    _want(row_start, "row_start", i32, (B + 1,), dev)
    _want(length, "length", i32, (B,), dev)
    return _BatchStruct(B, T, width, row_start.data_ptr(), length.data_ptr(), page_table.data_ptr())


def _rows(t, name: str, H, d: int, dev: int):
    """A bf16 [H, T, d] tensor of any head and row stride (rows themselves contiguous): T, head stride, row stride.
    The stride of an extent of one does not matter and may be anything."""
    shape = t.shape
    if not (t.dtype is torch.bfloat16 and len(shape) == 3 and shape[2] == d and (H is None or shape[0] == H)
            and t.get_device() == dev):
        raise ValueError(f"{name} must be bf16 [{'H' if H is None else H}, T, {d}] on cuda:{dev}")
    h, r, x = t.stride()
    if x != 1 and t.numel() != 0:
        raise ValueError(f"{name} must have contiguous rows")
    return shape[1], h if shape[0] > 1 else 0, r if shape[1] > 1 else 0


def _space(ws, dev: int):
    """The caller's workspace: its address goes to kernels on this device."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous on {_name(dev)}, not on {ws.device}")
    return ws


def _on(dev: int, stream):
    """Context in which the cache's device and the call's stream, one of that device, are current."""
    if stream is None and dev == torch._C._cuda_getDevice():
        return _HERE
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream must be one of {_name(dev)}, not of cuda:{stream.device_index}")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(dev))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return stack


_HERE = contextlib.nullcontext()
_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle without building a Stream object


def cache_append(c: Cache, k, v, row_start, length, page_table, rope: Optional[Rope] = None, row_times=None, ws=None,
                 stream=None) -> None:
    """Append rows to the cache (h3attn_cache_append): k, v bf16 [H, T, d] (any head and row strides that are multiples
    of 8), packed row row_start[b] + i becomes row length[b] + i of sequence b; keys rotated by ``rope``.
    Bad offsets, lengths, page ids and rotation indices are recorded in ``ws``, whose first 256 bytes the call uses:
    check(ws) tells, and without a ws nothing does."""
    cs = c._c
    dev = c._t[0].get_device()
    T, kh, kr = _rows(k, "k", cs.H, cs.d, dev)
    Tv, vh, vr = _rows(v, "v", cs.H, cs.d, dev)
    if Tv != T:
        raise ValueError("k and v must have the same rows")
    b = _batch(dev, T, row_start, length, page_table)
    if rope is not None and (rope._t[0].get_device() != dev or (rope._t[2] is not None and rope._t[2].shape[0] != T)):
        raise ValueError("rope must be on the cache's device, its index of T entries")
    if row_times is not None:
        _want(row_times, "row_times", torch.float32, (T,), dev)
    with _on(dev, stream):
        ws = torch.zeros(256, dtype=torch.uint8, device=c.device) if ws is None else _space(ws, dev)
        rc = lib().h3attn_cache_append(cs, b, k.data_ptr(), kh, kr, v.data_ptr(), vh, vr,
                                       rope._c if rope is not None else None, _dptr(row_times), ws.data_ptr(),
                                       ws.numel(), _raw_stream(dev))
    _raise(rc, "cache_append")


def cache_read(c: Cache, row_start, first, page_table, T: Optional[int] = None, k_out=None, v_out=None, ws=None,
               stream=None):
    """Cached rows as bf16 [H, T, d] (h3attn_cache_read): packed row row_start[b] + i gets row first[b] + i of sequence
    b.  T packed rows, or the buffers k_out and v_out (both, or one for K or V alone); returns (k, v).  Rows of new
    buffers that belong to no sequence are not written.  Bad device values are recorded in ``ws`` as by
    cache_append."""
    cs = c._c
    dev = c._t[0].get_device()
    with _on(dev, stream):
        if k_out is None and v_out is None:
            if T is None:
                raise ValueError("cache_read needs T or an output buffer")
            k_out = torch.empty((cs.H, T, cs.d), dtype=torch.bfloat16, device=c.device)
            v_out = torch.empty_like(k_out)
        rows = T if T is not None else (k_out if k_out is not None else v_out).shape[1]
        if k_out is not None:
            _want(k_out, "k_out", torch.bfloat16, (cs.H, rows, cs.d), dev)
        if v_out is not None:
            _want(v_out, "v_out", torch.bfloat16, (cs.H, rows, cs.d), dev)
        b = _batch(dev, rows, row_start, first, page_table)
        ws = torch.zeros(256, dtype=torch.uint8, device=c.device) if ws is None else _space(ws, dev)
        rc = lib().h3attn_cache_read(cs, b, _dptr(k_out), _dptr(v_out), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    _raise(rc, "cache_read")
    return k_out, v_out


def cache_forward(c: Cache, q, row_start, length, page_table, causal: bool = False, pen=None, q_times=None,
                  max_rows: Optional[int] = None, ws=None, out=None, lse: bool | torch.Tensor = False,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of packed query rows q bf16 [H, T, d] over the cached rows [0, length[b]) of their sequence
    (h3attn_cache_forward); (o, lse) is one partition for merge().  The penalty needs q_times (float32 [T], NaN for
    rows without one) and the cache's times.  Rows of a new ``out`` that belong to no sequence are not written.  q . k /
    sqrt(d) and each row's largest score, penalty included, must stay below 2^23 in magnitude; beyond, the result is
    undefined.  ``max_rows``, the most rows of a sequence in this call, is worth giving: without it the kernel is chosen
    as if all T rows were one sequence's.  Bad device values and waits that gave up are recorded in ``ws`` (check(ws));
    a call without one allocates and clears up to 39 MB and drops the record."""
    cs = c._c
    dev = c._t[0].get_device()
    T, qh, qr = _rows(q, "q", None, cs.d, dev)
    H, d = q.shape[0], cs.d
    b = _batch(dev, T, row_start, length, page_table)
    pn = _pen(pen)
    if q_times is not None:
        _want(q_times, "q_times", torch.float32, (T,), dev)
    if out is not None:
        _want(out, "out", torch.bfloat16, (H, T, d), dev)
    given = isinstance(lse, torch.Tensor)
    if given:
        _want(lse, "lse", torch.float32, (H, T), dev)
    with _on(dev, stream):
        o = torch.empty((H, T, d), dtype=torch.bfloat16, device=c.device) if out is None else out
        lse_t = lse if given else torch.empty((H, T), dtype=torch.float32, device=c.device) if lse else None
        ws = cache_workspace(c, H, T, b.B) if ws is None else _space(ws, dev)
        rc = lib().h3attn_cache_forward(cs, b, H, max_rows or 0, q.data_ptr(), qh, qr, int(causal), pn, _dptr(q_times),
                                        o.data_ptr(), _dptr(lse_t), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    _raise(rc, "cache_forward")
    return o, lse_t


def check(ws: torch.Tensor, stream=None) -> int:
    """Synchronise and return (and clear) the device status word."""
    return int(lib().h3attn_check(ws.data_ptr(), _stream(stream)))


def set_wait_polls(polls: int) -> None:
    """Test and diagnostics only: bound the attention kernels' waits of later calls to `polls` polls
    (0 = default, no poll bound)."""
    _raise(lib().h3attn_set_wait_polls(polls), "set_wait_polls")


def selftest_timeout(ws: torch.Tensor, polls: int, stream=None) -> None:
    _raise(lib().h3attn_selftest_timeout(ws.data_ptr(), polls, _stream(stream)), "selftest_timeout")
