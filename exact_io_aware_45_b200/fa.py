"""Thin Python binding of libfa.so (argument marshalling only).

The raw functions carry the C names of ``include/fa.h`` and take integer
device pointers; ``forward`` / ``backward`` / ``attention`` accept torch CUDA
tensors, allocate outputs and workspace with torch, pass the current stream
and raise ``FaError`` on a non-zero status. Every step of the computation runs
in the library's CUDA kernels. There is no fallback: if the library is missing
the first call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
# FA_LIBRARY may name another build of libfa.so (e.g. one compiled with
# different tile parameters); the default is the in-tree build.
LIB_PATH = os.environ.get("FA_LIBRARY") or os.path.join(PKG, "_lib", "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_CACHE = range(6)
FA_F32, FA_BF16 = 0, 1
PATH_AUTO, PATH_SIMT, PATH_TC = 0, 1, 2
FA_STALL_FWD, FA_STALL_BWD, FA_STALL_DQ = 1, 2, 4

# every symbol include/fa.h declares
EXPORTS = ("fa_status_string", "fa_version", "fa_fwd_workspace_size", "fa_bwd_workspace_size",
           "fa_fwd", "fa_fwd_ex", "fa_bwd", "fa_bwd_ex", "fa_bwd_preprocess", "fa_bwd_main",
           "fa_bwd_finalize", "fa_last_launch_count", "fa_get_device_error", "fa_exp2_fma",
           "fa_fwd_varlen", "fa_bwd_varlen", "fa_bwd_varlen_workspace_size",
           "fa_bwd_deterministic", "fa_fwd_window", "fa_bwd_window", "fa_bwd_noalloc",
           "fa_debug_set_stall", "fa_fwd_mod", "fa_bwd_mod", "fa_cache_workspace_size",
           "fa_cache_extend", "fa_cache_write", "fa_cache_fork", "fa_cache_free",
           "fa_cache_copy", "fa_cache_compact", "fa_fwd_paged", "fa_fwd_shared",
           "fa_paged_workspace_size")

_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_S = ctypes.c_size_t
_FWD_ARGS = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _I, _P, _P]
_BWD_ARGS = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _I, _I, _P, _S,
             _P]


class FaMods(ctypes.Structure):
    """fa_mods of include/fa.h: mask (and score) modifiers."""
    _fields_ = [("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
                ("prefix", ctypes.c_int), ("doc_ids", ctypes.c_void_p),
                ("softcap", ctypes.c_float)]


def mods(window_left: int = -1, window_right: int = -1, prefix: int = 0, doc_ids=None,
         softcap: float = 0.0) -> FaMods:
    """An fa_mods value; doc_ids is an int32 CUDA tensor [N] or None."""
    return FaMods(int(window_left), int(window_right), int(prefix),
                  None if doc_ids is None else doc_ids.data_ptr(), float(softcap))


class FaCache(ctypes.Structure):
    """fa_cache of include/fa.h: a paged key/value cache."""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("layer_stride", ctypes.c_longlong), ("page_stride", ctypes.c_longlong),
                ("layers", ctypes.c_int), ("pages", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("page_size", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int),
                ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("seqs", ctypes.c_int), ("seq_pages", ctypes.c_int), ("err", ctypes.c_void_p)]


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """Loads libfa.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfa.so not built ({LIB_PATH}); run "
                               "python -m exact_io_aware_45_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_status_string.argtypes = [_I]
        L.fa_version.restype = _I
        L.fa_fwd_workspace_size.restype = _S
        L.fa_bwd_workspace_size.restype = _S
        L.fa_bwd_workspace_size.argtypes = [_I, _I, _I, _I]
        L.fa_fwd.argtypes = _FWD_ARGS
        L.fa_fwd_ex.argtypes = _FWD_ARGS + [_I]
        L.fa_bwd.argtypes = _BWD_ARGS
        for n in ("fa_bwd_ex", "fa_bwd_preprocess", "fa_bwd_main", "fa_bwd_finalize",
                  "fa_bwd_deterministic"):
            getattr(L, n).argtypes = _BWD_ARGS + [_I]
        for n in ("fa_fwd", "fa_fwd_ex", "fa_bwd", "fa_bwd_ex", "fa_bwd_preprocess",
                  "fa_bwd_main", "fa_bwd_finalize", "fa_get_device_error", "fa_bwd_deterministic"):
            getattr(L, n).restype = _I
        L.fa_last_launch_count.restype = _I
        L.fa_get_device_error.argtypes = [_P, _P]
        L.fa_exp2_fma.argtypes = [_P, _P, ctypes.c_longlong, _P]
        L.fa_exp2_fma.restype = _I
        L.fa_fwd_varlen.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I,
                                    _P, _P]
        L.fa_fwd_varlen.restype = _I
        L.fa_bwd_varlen.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                    _I, _F, _I, _I, _I, _P, _S, _P]
        L.fa_bwd_varlen.restype = _I
        L.fa_fwd_window.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P,
                                    _I, _P, _P]
        L.fa_fwd_window.restype = _I
        L.fa_bwd_window.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F,
                                    _I, _I, _I, _P, _I, _I, _P, _S, _P]
        L.fa_bwd_window.restype = _I
        L.fa_fwd_mod.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P,
                                 ctypes.POINTER(FaMods), _I, _P, _P]
        L.fa_fwd_mod.restype = _I
        L.fa_bwd_mod.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I,
                                 _P, ctypes.POINTER(FaMods), _I, _I, _P, _S, _P]
        L.fa_bwd_mod.restype = _I
        L.fa_debug_set_stall.argtypes = [_I, ctypes.c_longlong]
        L.fa_debug_set_stall.restype = _I
        L.fa_bwd_varlen_workspace_size.argtypes = [_I, _I, _I, _I, _I]
        L.fa_bwd_varlen_workspace_size.restype = _S
        C = _P          # const fa_cache*: an address, or byref() of one
        for n, args in (("fa_cache_extend", [C, _P, _I, _P, _I, _P, _P, _S, _P]),
                        ("fa_cache_write", [C, _I, _P, _P, _P, _P, _I, _P, _I, _P]),
                        ("fa_cache_fork", [C, _P, _P, _I, _P, _S, _P]),
                        ("fa_cache_free", [C, _P, _I, _P, _S, _P]),
                        ("fa_cache_copy", [C, _P, _P, _I, _P, _S, _P]),
                        ("fa_cache_compact", [C, _P, _S, _P]),
                        ("fa_fwd_paged", [C, _I, _P, _P, _P, _P, _I, _I, _I, _F, _I, _I, _F, _P,
                                          _S, _P]),
                        ("fa_fwd_shared", [C, _I, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _I, _F,
                                           _P, _S, _P])):
            getattr(L, n).argtypes = args
            getattr(L, n).restype = _I
        L.fa_cache_workspace_size.argtypes = [C, _I]
        L.fa_cache_workspace_size.restype = _S
        L.fa_paged_workspace_size.argtypes = [C, _I, _I, _I, _I]
        L.fa_paged_workspace_size.restype = _S
        _lib = L
    return _lib


# ------------------------------------------------------------------ raw C functions

def status_string(s: int) -> str:
    return lib().fa_status_string(int(s)).decode()


def fa_version() -> int:
    return lib().fa_version()


def fa_fwd_workspace_size() -> int:
    return lib().fa_fwd_workspace_size()


def fa_bwd_workspace_size(B, Hq, N, d) -> int:
    return lib().fa_bwd_workspace_size(B, Hq, N, d)


def fa_fwd(*args) -> int:
    return lib().fa_fwd(*args)


def fa_fwd_ex(*args) -> int:
    return lib().fa_fwd_ex(*args)


def fa_bwd(*args) -> int:
    return lib().fa_bwd(*args)


def fa_bwd_ex(*args) -> int:
    return lib().fa_bwd_ex(*args)


def fa_bwd_preprocess(*args) -> int:
    return lib().fa_bwd_preprocess(*args)


def fa_bwd_main(*args) -> int:
    return lib().fa_bwd_main(*args)


def fa_bwd_finalize(*args) -> int:
    return lib().fa_bwd_finalize(*args)


def fa_last_launch_count() -> int:
    return lib().fa_last_launch_count()


def fa_get_device_error(workspace_ptr: int, stream_ptr: int) -> int:
    return lib().fa_get_device_error(workspace_ptr, stream_ptr)


def fa_exp2_fma(x_ptr: int, y_ptr: int, n: int, stream_ptr: int) -> int:
    return lib().fa_exp2_fma(x_ptr, y_ptr, n, stream_ptr)


def fa_bwd_deterministic(*args) -> int:
    return lib().fa_bwd_deterministic(*args)


def fa_fwd_window(*args) -> int:
    return lib().fa_fwd_window(*args)


def fa_bwd_window(*args) -> int:
    return lib().fa_bwd_window(*args)


def fa_fwd_varlen(*args) -> int:
    return lib().fa_fwd_varlen(*args)


def fa_bwd_varlen(*args) -> int:
    return lib().fa_bwd_varlen(*args)


def fa_fwd_mod(*args) -> int:
    return lib().fa_fwd_mod(*args)


def fa_bwd_mod(*args) -> int:
    return lib().fa_bwd_mod(*args)


def fa_debug_set_stall(kernels: int, wait_cycles: int) -> int:
    return lib().fa_debug_set_stall(int(kernels), int(wait_cycles))


def fa_bwd_varlen_workspace_size(B, Hq, max_seqlen, total, d) -> int:
    return lib().fa_bwd_varlen_workspace_size(B, Hq, max_seqlen, total, d)


def fa_cache_workspace_size(cache, n) -> int:
    return lib().fa_cache_workspace_size(cache, n)


def fa_cache_extend(*args) -> int:
    return lib().fa_cache_extend(*args)


def fa_cache_write(*args) -> int:
    return lib().fa_cache_write(*args)


def fa_cache_fork(*args) -> int:
    return lib().fa_cache_fork(*args)


def fa_cache_free(*args) -> int:
    return lib().fa_cache_free(*args)


def fa_cache_copy(*args) -> int:
    return lib().fa_cache_copy(*args)


def fa_cache_compact(*args) -> int:
    return lib().fa_cache_compact(*args)


def fa_fwd_paged(*args) -> int:
    return lib().fa_fwd_paged(*args)


def fa_fwd_shared(*args) -> int:
    return lib().fa_fwd_shared(*args)


def fa_paged_workspace_size(cache, B, T, Hq, shared) -> int:
    return lib().fa_paged_workspace_size(cache, B, T, Hq, shared)


# ------------------------------------------------------------------ torch helpers

def _dtype_code(t) -> int:
    import torch
    if t == torch.float32:
        return FA_F32
    if t == torch.bfloat16:
        return FA_BF16
    raise TypeError(f"unsupported dtype {t}")


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _check(status: int, what: str):
    if status != FA_OK:
        raise FaError(status, what)


def _stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def new_workspace(nbytes: int, device):
    """A workspace buffer whose 256-byte error-word block is zeroed."""
    import torch
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _dims(q, k):
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    return B, Hq, Hkv, N, d


def forward(q, k, v, scale: Optional[float] = None, causal: bool = False, block_mask=None,
            path: int = PATH_AUTO, out=None, lse=None, workspace=None):
    """O, LSE = attention(q, k, v). q [B,Hq,N,d], k/v [B,Hkv,N,d] contiguous CUDA
    tensors (bf16 or fp32); block_mask uint8 [nb, nb] CUDA tensor or None;
    scale defaults to 1/sqrt(d)."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if lse is None else lse
    ws = new_workspace(fa_fwd_workspace_size(), q.device) if workspace is None else workspace
    s = fa_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, Hq, Hkv, N, d, float(scale),
                  int(bool(causal)), _ptr(block_mask), _dtype_code(q.dtype), _ptr(ws), _stream(),
                  int(path))
    _check(s, "fa_fwd")
    return o, l


def backward(q, k, v, o, do, lse, scale: Optional[float] = None, causal: bool = False,
             block_mask=None, grad_dtype=None, path: int = PATH_AUTO, workspace=None,
             deterministic: bool = False):
    """dQ, dK, dV of sum(O * dO). grad_dtype defaults to float32 (the tensor
    cores accumulate in fp32; a bf16 gradient adds its own rounding).
    deterministic: run-to-run identical dQ (fa_bwd_deterministic)."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    gdt = torch.float32 if grad_dtype is None else grad_dtype
    dq = torch.empty(q.shape, dtype=gdt, device=q.device)
    dk = torch.empty(k.shape, dtype=gdt, device=q.device)
    dv = torch.empty(v.shape, dtype=gdt, device=q.device)
    nbytes = fa_bwd_workspace_size(B, Hq, N, d)
    ws = new_workspace(nbytes, q.device) if workspace is None else workspace
    fn = fa_bwd_deterministic if deterministic else fa_bwd_ex
    s = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
           _ptr(dv), B, Hq, Hkv, N, d, float(scale), int(bool(causal)), _ptr(block_mask),
           _dtype_code(q.dtype), _dtype_code(gdt), _ptr(ws), ws.numel(), _stream(), int(path))
    _check(s, "fa_bwd_deterministic" if deterministic else "fa_bwd")
    return dq, dk, dv


def forward_varlen(q, k, v, cu_seqlens, max_seqlen: int, scale: Optional[float] = None,
                   causal: bool = False, out=None, lse=None, workspace=None):
    """Variable-length batch: q [total, Hq, d], k/v [total, Hkv, d] (bf16,
    sequences packed back to back), cu_seqlens int32 CUDA tensor [B + 1].
    Returns O [total, Hq, d] and LSE [Hq, total]."""
    import torch
    total, Hq, d = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((Hq, total), dtype=torch.float32, device=q.device) if lse is None else lse
    ws = new_workspace(fa_fwd_workspace_size(), q.device) if workspace is None else workspace
    s = fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), _ptr(cu_seqlens), B,
                      int(max_seqlen), total, Hq, Hkv, d, float(scale), int(bool(causal)),
                      _dtype_code(q.dtype), _ptr(ws), _stream())
    _check(s, "fa_fwd_varlen")
    return o, l


def backward_varlen(q, k, v, o, do, lse, cu_seqlens, max_seqlen: int,
                    scale: Optional[float] = None, causal: bool = False, grad_dtype=None,
                    workspace=None):
    """dQ, dK, dV of a variable-length batch (layouts as forward_varlen)."""
    import torch
    total, Hq, d = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    gdt = torch.float32 if grad_dtype is None else grad_dtype
    dq = torch.empty(q.shape, dtype=gdt, device=q.device)
    dk = torch.empty(k.shape, dtype=gdt, device=q.device)
    dv = torch.empty(v.shape, dtype=gdt, device=q.device)
    nbytes = fa_bwd_varlen_workspace_size(B, Hq, int(max_seqlen), total, d)
    ws = new_workspace(nbytes, q.device) if workspace is None else workspace
    s = fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                      _ptr(dk), _ptr(dv), _ptr(cu_seqlens), B, int(max_seqlen), total, Hq, Hkv,
                      d, float(scale), int(bool(causal)), _dtype_code(q.dtype), _dtype_code(gdt),
                      _ptr(ws), ws.numel(), _stream())
    _check(s, "fa_bwd_varlen")
    return dq, dk, dv


def forward_window(q, k, v, window_left: int, window_right: int, scale: Optional[float] = None,
                   causal: bool = False, block_mask=None):
    """O, LSE of sliding-window attention (fa_fwd_window); layouts as forward."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q)
    l = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    ws = new_workspace(fa_fwd_workspace_size(), q.device)
    s = fa_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, Hq, Hkv, N, d, float(scale),
                      int(bool(causal)), int(window_left), int(window_right), _ptr(block_mask),
                      _dtype_code(q.dtype), _ptr(ws), _stream())
    _check(s, "fa_fwd_window")
    return o, l


def backward_window(q, k, v, o, do, lse, window_left: int, window_right: int,
                    scale: Optional[float] = None, causal: bool = False, block_mask=None,
                    grad_dtype=None):
    """dQ, dK, dV of sliding-window attention (fa_bwd_window)."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    gdt = torch.float32 if grad_dtype is None else grad_dtype
    dq = torch.empty(q.shape, dtype=gdt, device=q.device)
    dk = torch.empty(k.shape, dtype=gdt, device=q.device)
    dv = torch.empty(v.shape, dtype=gdt, device=q.device)
    ws = new_workspace(fa_bwd_workspace_size(B, Hq, N, d), q.device)
    s = fa_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                      _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, float(scale), int(bool(causal)),
                      int(window_left), int(window_right), _ptr(block_mask), _dtype_code(q.dtype),
                      _dtype_code(gdt), _ptr(ws), ws.numel(), _stream())
    _check(s, "fa_bwd_window")
    return dq, dk, dv


def forward_mod(q, k, v, m: FaMods, scale: Optional[float] = None, causal: bool = False,
                block_mask=None, workspace=None, out=None, lse=None):
    """O, LSE with mask modifiers (fa_fwd_mod); layouts and out / lse / workspace
    as forward."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if lse is None else lse
    ws = new_workspace(fa_fwd_workspace_size(), q.device) if workspace is None else workspace
    s = fa_fwd_mod(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, Hq, Hkv, N, d, float(scale),
                   int(bool(causal)), _ptr(block_mask), ctypes.byref(m), _dtype_code(q.dtype),
                   _ptr(ws), _stream())
    _check(s, "fa_fwd_mod")
    return o, l


def backward_mod(q, k, v, o, do, lse, m: FaMods, scale: Optional[float] = None,
                 causal: bool = False, block_mask=None, grad_dtype=None, workspace=None):
    """dQ, dK, dV with mask modifiers (fa_bwd_mod); the forward's modifiers."""
    import torch
    B, Hq, Hkv, N, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    gdt = torch.float32 if grad_dtype is None else grad_dtype
    dq = torch.empty(q.shape, dtype=gdt, device=q.device)
    dk = torch.empty(k.shape, dtype=gdt, device=q.device)
    dv = torch.empty(v.shape, dtype=gdt, device=q.device)
    ws = new_workspace(fa_bwd_workspace_size(B, Hq, N, d), q.device) if workspace is None \
        else workspace
    s = fa_bwd_mod(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                   _ptr(dv), B, Hq, Hkv, N, d, float(scale), int(bool(causal)), _ptr(block_mask),
                   ctypes.byref(m), _dtype_code(q.dtype), _dtype_code(gdt), _ptr(ws), ws.numel(),
                   _stream())
    _check(s, "fa_bwd_mod")
    return dq, dk, dv


def device_error(workspace) -> int:
    """Reads and clears the workspace's error word (synchronises the stream)."""
    return fa_get_device_error(_ptr(workspace), _stream())


def _autograd_fn():
    import torch

    class _Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, scale, causal, block_mask):
            o, lse = forward(q, k, v, scale, causal, block_mask)
            ctx.save_for_backward(q, k, v, o, lse)
            ctx.scale, ctx.causal, ctx.block_mask = scale, causal, block_mask
            return o

        @staticmethod
        def backward(ctx, do):
            q, k, v, o, lse = ctx.saved_tensors
            dq, dk, dv = backward(q, k, v, o, do.contiguous(), lse, ctx.scale, ctx.causal,
                                  ctx.block_mask, grad_dtype=q.dtype)
            return dq, dk, dv, None, None, None

    return _Attention


def attention(q, k, v, scale: Optional[float] = None, causal: bool = False, block_mask=None):
    """Differentiable attention (torch autograd), gradients in the input dtype."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _autograd_fn().apply(q, k, v, scale, causal, block_mask)


# ------------------------------------------------------------------ paged cache

_INT_MIN, _INT_MAX = -1 << 31, (1 << 31) - 1


def _c_int(x) -> int:
    """A number for an int argument of the library; ctypes would take it modulo 2^32."""
    if not _INT_MIN <= x <= _INT_MAX:
        raise ValueError(f"{x} does not fit an int")
    return x


class PagedCache:
    """Keys and values of many sequences in a pool of fixed-size pages (fa_cache
    of include/fa.h, which says what the calls do and when they are refused).

    k, v: [layers, pages, Hkv, page_size, d] CUDA tensors, bf16 or fp32, with
    equal strides and contiguous pages; table int32 [seqs, seq_pages], lens int32
    [seqs], refs int32 [pages], contiguous. The cache keeps and updates these
    tensors; ``new`` makes an empty one. Lists of slots and pages are int32 CUDA
    tensors. Calls are asynchronous on the current stream; what the device
    refuses is raised by ``check``."""

    def __init__(self, k, v, table, lens, refs):
        import torch
        if k.dim() != 5 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v are [layers, pages, Hkv, page_size, d] of one type and stride")
        L, P, Hkv, ps, d = k.shape
        # the stride of a dimension of one entry moves nothing: as in a contiguous tensor
        plain = (P * Hkv * ps * d, Hkv * ps * d, ps * d, d, 1)
        stride, v_stride = (tuple(p if n == 1 else s for n, s, p in zip(t.shape, t.stride(), plain))
                            for t in (k, v))
        if stride != v_stride:
            raise ValueError("k and v are [layers, pages, Hkv, page_size, d] of one type and stride")
        if min(k.shape) < 1 or stride[2:] != plain[2:]:
            raise ValueError("a page [Hkv, page_size, d] of k and v is contiguous and not empty")
        if table.dim() != 2 or lens.shape != table.shape[:1] or refs.shape != (P,):
            raise ValueError("table is [seqs, seq_pages], lens [seqs], refs [pages]")
        for t in (table, lens, refs):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError("table, lens and refs are contiguous int32 tensors")
        if not k.is_cuda or any(t.device != k.device for t in (v, table, lens, refs)):
            raise ValueError("the tensors of a cache are on one CUDA device")
        self.k, self.v, self.table, self.lens, self.refs = k, v, table, lens, refs
        self.device, self.dtype = k.device, k.dtype
        self.layers, self.pages, self.Hkv, self.page_size, self.d = k.shape
        self.err = torch.zeros(64, dtype=torch.int32, device=k.device)
        self._c = FaCache(_ptr(k), _ptr(v), stride[0], stride[1], L, P, Hkv, ps, d,
                          _dtype_code(k.dtype), _ptr(table), _ptr(lens), _ptr(refs),
                          table.shape[0], table.shape[1], _ptr(self.err))
        # a call costs the host as much as small ones cost the GPU: what every call needs is
        # looked up once (workspace sizes by the sizes they depend on)
        self._torch, self._index = torch, k.device.index
        self._ref = ctypes.addressof(self._c)
        self._current, self._raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self._int32, self._sizes = torch.int32, {}
        L = lib()
        self._extend, self._write, self._free = L.fa_cache_extend, L.fa_cache_write, L.fa_cache_free
        self._fork, self._copy, self._compact = L.fa_cache_fork, L.fa_cache_copy, L.fa_cache_compact
        self._paged, self._shared = L.fa_fwd_paged, L.fa_fwd_shared
        if fa_cache_workspace_size(self._ref, 0) == 0:
            raise ValueError("unsupported cache: page_size is 16, 32, 64 or 128, d 16, 32, 64 or "
                             "128, strides are multiples of 16 bytes")

    @classmethod
    def new(cls, layers: int, pages: int, Hkv: int, page_size: int, d: int, seqs: int,
            seq_pages: int, dtype=None, device="cuda"):
        """An empty cache (dtype defaults to bfloat16)."""
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        shape = (layers, pages, Hkv, page_size, d)
        k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        table = torch.full((seqs, seq_pages), -1, dtype=torch.int32, device=device)
        lens, refs = (torch.zeros(n, dtype=torch.int32, device=device) for n in (seqs, pages))
        return cls(k, v, table, lens, refs)

    def _list(self, t) -> int:
        """The length of a list of slots, pages, positions or offsets."""
        if t.dtype is not self._int32 or t.dim() != 1 or not t.is_contiguous() or \
                t.get_device() != self._index:
            raise ValueError("a list is a contiguous int32 tensor on the cache's device")
        n = t.numel()
        return n if n <= _INT_MAX else _c_int(n)

    def _call(self, fn, *args):
        """A library call on the cache's device and its current stream."""
        index = self._index
        if self._current() == index:
            s = fn(self._ref, *args, self._raw_stream(index))
        else:
            with self._torch.cuda.device(index):
                s = fn(self._ref, *args, self._raw_stream(index))
        if s:
            raise FaError(s, fn.__name__)

    def _workspace(self, *key):
        """A new workspace: for lists of (n,) entries, or attention of (B, T, Hq, shared)."""
        size = self._sizes.get(key)
        if size is None:
            fn = fa_cache_workspace_size if len(key) == 1 else fa_paged_workspace_size
            with self._torch.cuda.device(self._index):
                size = self._sizes[key] = fn(self._ref, *key)
        return self.err.new_empty(size, dtype=self._torch.uint8), size

    def extend(self, seqs, tokens):
        """Makes room for new tokens: `tokens` of each sequence, or cu_seqlens
        (int32 [n + 1]). Returns the positions of the first ones, int32 [n]."""
        n = self._list(seqs)
        if isinstance(tokens, self._torch.Tensor):     # (referenced until its use is enqueued)
            if self._list(tokens) != n + 1:
                raise ValueError("cu_seqlens has one entry more than the list of sequences")
            cu, each = tokens.data_ptr(), 0
        else:
            cu, each = 0, _c_int(int(tokens))
        pos = seqs.new_empty(n)
        ws, size = self._workspace(n)
        self._call(self._extend, seqs.data_ptr(), n, cu, each, pos.data_ptr(),
                   ws.data_ptr(), size)
        return pos

    def write(self, layer: int, k, v, seqs, pos, cu_seqlens=None):
        """Writes new keys and values [total, Hkv, d] of one layer from the
        positions that extend returned on; rows of equal shares, or cu_seqlens."""
        n = self._list(seqs)
        if self._list(pos) != n:
            raise ValueError("lists of different lengths")
        cu = 0
        if cu_seqlens is not None:
            if self._list(cu_seqlens) != n + 1:
                raise ValueError("cu_seqlens has one entry more than the list of sequences")
            cu = cu_seqlens.data_ptr()
        shape = k.shape
        for t in (k, v):
            if t.shape != shape or t.dtype != self.dtype or not t.is_contiguous() or \
                    t.get_device() != self._index:
                raise ValueError("k and v are contiguous [total, Hkv, d] of the cache's type")
        if len(shape) != 3 or shape[1] != self.Hkv or shape[2] != self.d:
            raise ValueError("k and v are contiguous [total, Hkv, d] of the cache's type")
        self._call(self._write, _c_int(layer), k.data_ptr(), v.data_ptr(), seqs.data_ptr(),
                   pos.data_ptr(), n, cu, _c_int(shape[0]))

    def _pairs(self, fn, src, dst):
        n = self._list(src)
        if self._list(dst) != n:
            raise ValueError("lists of different lengths")
        ws, size = self._workspace(n)
        self._call(fn, src.data_ptr(), dst.data_ptr(), n, ws.data_ptr(), size)

    def fork(self, src, dst):
        """Makes the empty sequences dst copies of src: full pages are shared."""
        self._pairs(self._fork, src, dst)

    def copy_pages(self, src, dst):
        """Copies pages src to pages dst in all layers."""
        self._pairs(self._copy, src, dst)

    def free(self, seqs):
        """Empties sequences and gives up their pages."""
        n = self._list(seqs)
        ws, size = self._workspace(n)
        self._call(self._free, seqs.data_ptr(), n, ws.data_ptr(), size)

    def compact(self):
        """Moves the pages in use to the front of the pool."""
        ws, size = self._workspace(0)
        self._call(self._compact, ws.data_ptr(), size)

    def check(self):
        """Raises FaError if the device refused a call or a wait ran out since the last
        check (synchronises the stream); if both, the refusal is left for the next check."""
        with self._torch.cuda.device(self._index):
            _check(fa_get_device_error(_ptr(self.err), self._raw_stream(self._index)),
                   "paged cache")


def _forward_cache(q, cache, layer, shared, seqs, scale, causal, window_left, softcap, out, lse,
                   workspace):
    index, shape = cache._index, q.shape
    if q.dtype != cache.dtype or q.get_device() != index or not q.is_contiguous() or \
            len(shape) != 4 or shape[3] != cache.d:
        raise ValueError("q is a contiguous [B, Hq, T, d] of the cache's type, on its device")
    B, Hq, T, d = shape
    if not (_INT_MIN <= layer <= _INT_MAX and _INT_MIN <= shared <= _INT_MAX and
            _INT_MIN <= window_left <= _INT_MAX):      # (in line: a call takes the host 15 us)
        raise ValueError("layer, shared and window_left are ints of 32 bits")
    if seqs is not None and cache._list(seqs) != B:
        raise ValueError("one sequence for each batch entry")
    torch = cache._torch
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != shape or out.dtype != q.dtype or out.get_device() != index or \
            not out.is_contiguous():
        raise ValueError("out is like q")
    if lse is None:
        lse = q.new_empty((B, Hq, T), dtype=torch.float32)
    elif lse.shape != shape[:3] or lse.dtype != torch.float32 or lse.get_device() != index or \
            not lse.is_contiguous():
        raise ValueError("lse is float32 [B, Hq, T]")
    if workspace is None:
        workspace, size = cache._workspace(B, T, Hq, shared)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace is contiguous, on the cache's device")
    else:
        size = workspace.numel() * workspace.element_size()
    if scale is None:
        scale = d ** -0.5
    slots = 0 if seqs is None else seqs.data_ptr()
    causal = 1 if causal else 0
    if shared:
        cache._call(cache._shared, layer, q.data_ptr(), out.data_ptr(), lse.data_ptr(), slots, B,
                    T, Hq, shared, scale, causal, window_left, softcap, workspace.data_ptr(), size)
    else:
        cache._call(cache._paged, layer, q.data_ptr(), out.data_ptr(), lse.data_ptr(), slots, B, T,
                    Hq, scale, causal, window_left, softcap, workspace.data_ptr(), size)
    return out, lse


def forward_paged(q, cache: PagedCache, layer: int, seqs=None, scale: Optional[float] = None,
                  causal: bool = True, window_left: int = -1, softcap: float = 0.0, out=None,
                  lse=None, workspace=None):
    """O, LSE of the last T tokens of each sequence over the cache (fa_fwd_paged;
    without gradients). q [B, Hq, T, d]; seqs int32 [B], or None for slots 0 .. B-1. A workspace
    (fa_paged_workspace_size bytes) serves one call at a time."""
    return _forward_cache(q, cache, layer, 0, seqs, scale, causal, window_left, softcap, out, lse,
                          workspace)


def forward_shared(q, cache: PagedCache, layer: int, shared: int, seqs=None,
                   scale: Optional[float] = None, causal: bool = True, window_left: int = -1,
                   softcap: float = 0.0, out=None, lse=None, workspace=None):
    """forward_paged for sequences that begin with the same `shared` tokens (a
    multiple of the page size), read once for the batch (fa_fwd_shared)."""
    return _forward_cache(q, cache, layer, int(shared), seqs, scale, causal, window_left, softcap,
                          out, lse, workspace)
