"""ctypes binding of libfa.so (C ABI in include/fa.h) -- argument marshalling only.

Every function here checks that the tensors live on a CUDA device with the expected
dtype and contiguity, passes their device pointers and the current CUDA stream to the
library, and raises ``FAError`` with the library's status and message on failure.  No
attention arithmetic happens in Python; if ``libfa.so`` has not been built, every call
raises instead of falling back to anything else.

Calls run on the current stream, or on ``stream``.  Tensors that a call on another stream makes
itself are that stream's memory; those that the caller passes are the caller's to keep until the
call has run.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# FA_LIBRARY selects another build of the library, e.g. the debug build libfa_debug.so
LIB_PATH = os.environ.get("FA_LIBRARY") or os.path.join(_HERE, "libfa.so")

FA_OK = 0
FA_ERR_INVALID = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_WORKSPACE = 3
FA_ERR_CUDA = 4
FA_ERR_TIMEOUT = 5
FA_ERR_DEVICE_ARG = 6
FA_ERR_DEBUG_CHECK = 7
FA_ERR_NO_PAGES = 8
FA_BF16 = 0
FA_F32 = 1

# Every symbol include/fa.h declares, with its ctypes signature.
_P, _I, _F, _Z, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
SIGNATURES = {
    "fa_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_fwd_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P]),
    "fa_fwd_window": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P]),
    "fa_fwd_bshd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P]),
    "fa_fwd_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _I, _P]),
    "fa_decode_workspace_size": (_Z, [_I, _I, _I, _I]),
    "fa_decode": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _Z, _P]),
    "fa_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "fa_decode_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _Z, _P]),
    "fa_decode_ex": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _Z, _P]),
    "fa_merge_lse": (_I, [_P, _P, _I, _I, _I, _P, _P, _I, _P]),
    "fa_decode_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _Z, _P]),
    "fa_decode_paged_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                                 _P, _Z, _P]),
    "fa_fwd_varlen_workspace_size": (_Z, [_I] * 4),
    "fa_fwd_varlen": (_I, [_P] * 7 + [_I] * 6 + [_L] * 3 + [_F, _I, _I, _I, _P, _Z, _P]),
    "fa_fwd_varlen_paged": (_I, [_P] * 8 + [_I] * 8 + [_L, _F, _I, _I, _I, _P, _Z, _P]),
    "fa_rope": (_I, [_P] * 7 + [_I] * 6 + [_L] * 4 + [_I] * 3 + [_P]),
    "fa_cache_append": (_I, [_P] * 9 + [_I] * 7 + [_L] * 2 + [_P]),
    "fa_cache_append_ex": (_I, [_P] * 10 + [_I] * 7 + [_L] * 2 + [_P]),
    "fa_rope_append": (_I, [_P] * 14 + [_I] * 10 + [_L] * 4 + [_I, _P]),
    "fa_rope_append_ex": (_I, [_P] * 15 + [_I] * 10 + [_L] * 4 + [_I, _P]),
    "fa_pages_reserve_workspace_size": (_Z, [_I, _I]),
    "fa_pages_reserve": (_I, [_P] * 5 + [_I] * 4 + [_P, _Z, _P]),
    "fa_pages_reserve_ex": (_I, [_P] * 6 + [_I] * 4 + [_P, _Z, _P]),
    "fa_pages_fork": (_I, [_P] * 6 + [_I] * 5 + [_P]),
    "fa_pages_free": (_I, [_P] * 5 + [_I] * 5 + [_P]),
    "fa_pages_compact_workspace_size": (_Z, [_I]),
    "fa_pages_compact": (_I, [_P] * 4 + [_I] * 4 + [_P, _Z, _P]),
    "fa_pages_copy": (_I, [_P] * 3 + [_I, _I, _L, _P]),
    "fa_get_error": (_I, [_P]),
    "fa_set_wait_limit_ns": (None, [ctypes.c_ulonglong]),
    "fa_fwd_selftest_timeout": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_decode_selftest_timeout": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _Z, _P]),
    "fa_build_flags": (_I, []),
    "fa_debug_selftest_bounds": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_status_str": (ctypes.c_char_p, [_I]),
    "fa_last_error_message": (ctypes.c_char_p, []),
    "fa_version": (_I, []),
}

_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{status_str(status)}: {message}")


def load(path: str = LIB_PATH):
    """Load libfa.so (once) and declare its signatures.  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise FAError(FA_ERR_UNSUPPORTED,
                          f"{path} is not built (run: python -m exact_io_aware_81_b200.build)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_str(status: int) -> str:
    try:
        return load().fa_status_str(int(status)).decode()
    except Exception:
        return str(status)


def _c_int(n) -> int:
    """An integer of the caller's for a C int.  ctypes keeps the low 32 bits of a longer one, which
    makes other numbers of them (a window of 2^32 + 5 one of 5); the nearest C int means the same
    here: a window of all keys, or a size that the library refuses."""
    return max(-2 ** 31, min(int(n), 2 ** 31 - 1))


def _check(rc: int):
    if rc != FA_OK:
        raise FAError(rc, load().fa_last_error_message().decode())


def _stream_handle(stream, device=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream)


@contextlib.contextmanager
def _on_device(*tensors):
    """Run a library call on the device of its tensors (the C ABI launches on the current
    device); every tensor passed must be on that one device."""
    dev = tensors[0].device
    for t in tensors[1:]:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors must be on {dev}; found one on {t.device}")
    with torch.cuda.device(dev):
        yield dev


def _require(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _new(shape, dtype, dev, stream, handed_back=True):
    """A tensor that a call makes: memory of the stream that the call runs on.  As memory of the
    current stream it could be handed out while other work of that stream still used it, and handed
    out again, once dropped, before the call had run.  One that is handed back to the caller may be
    used on the current stream too, so that stream is recorded as a user."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    current = torch.cuda.current_stream(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream), dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if handed_back:
        t.record_stream(current)
    return t


def _output(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape, device, stream) -> torch.Tensor:
    """A caller-provided output checked against its dtype and exact shape, or a new one."""
    shape = tuple(shape)
    if t is None:
        return _new(shape, dtype, device, stream)
    _require(t, name, dtype, len(shape))
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
        scale: Optional[float] = None, out_dtype: torch.dtype = torch.bfloat16,
        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
        stream=None, window: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention forward: q (B,Hq,Nq,d), k/v (B,Hkv,Nk,d) bf16 -> (o, lse).

    scale defaults to 1/sqrt(d) (as flash_attn_func's softmax_scale=None does on the
    toolsku.com page).  causal uses bottom-right alignment (row i sees keys up to
    i + Nk - Nq).  window = W >= 1 (causal only) restricts row i to its W most recent
    keys (fa_fwd_window); 0 means no window.  o has out_dtype (bf16 or fp32); lse is
    fp32 (B,Hq,Nq), natural log.
    """
    _require(q, "q", torch.bfloat16, 4)
    _require(k, "k", torch.bfloat16, 4)
    _require(v, "v", torch.bfloat16, 4)
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if (Bk, dk) != (B, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    out, lse = _fwd_outputs(q, (B, Hq, Nq, d), (B, Hq, Nq), out_dtype, out, lse, stream)
    odt = FA_F32 if out_dtype == torch.float32 else FA_BF16
    if window:
        if not causal:
            raise ValueError("a sliding window needs causal=True")
        with _on_device(q, k, v, out, lse) as dev:
            rc = load().fa_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                      lse.data_ptr(), B, Hq, Hkv, Nq, Nk, d, float(scale), _c_int(window),
                                      odt, _stream_handle(stream, dev))
    else:
        with _on_device(q, k, v, out, lse) as dev:
            rc = load().fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  lse.data_ptr(), B, Hq, Hkv, Nq, Nk, d, float(scale), int(bool(causal)),
                                  odt, _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def _fwd_outputs(q, o_shape, lse_shape, out_dtype, out, lse, stream):
    return (_output(out, "out", out_dtype, o_shape, q.device, stream),
            _output(lse, "lse", torch.float32, lse_shape, q.device, stream))


def fwd_bshd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
             scale: Optional[float] = None, out_dtype: torch.dtype = torch.bfloat16,
             out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
             stream=None, window: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention forward on (batch, sequence, heads, dim) tensors (fa_fwd_bshd), the layout
    flash_attn_func takes: q (B,Nq,Hq,d), k/v (B,Nk,Hkv,d) bf16 -> o (B,Nq,Hq,d) and lse
    fp32 (B,Hq,Nq).  causal, scale, window and out_dtype as fwd."""
    _require(q, "q", torch.bfloat16, 4)
    _require(k, "k", torch.bfloat16, 4)
    _require(v, "v", torch.bfloat16, 4)
    B, Nq, Hq, d = q.shape
    Bk, Nk, Hkv, dk = k.shape
    if (Bk, dk) != (B, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    if window and not causal:
        raise ValueError("a sliding window needs causal=True")
    out, lse = _fwd_outputs(q, (B, Nq, Hq, d), (B, Hq, Nq), out_dtype, out, lse, stream)
    odt = FA_F32 if out_dtype == torch.float32 else FA_BF16
    with _on_device(q, k, v, out, lse) as dev:
        rc = load().fa_fwd_bshd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                B, Hq, Hkv, Nq, Nk, d, float(scale), int(bool(causal)), _c_int(window), odt,
                                _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def fwd_window(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int,
               scale: Optional[float] = None, out_dtype: torch.dtype = torch.bfloat16,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Sliding-window causal attention (fa_fwd_window): row i sees keys j with
    i + Nk - Nq - window < j <= i + Nk - Nq.  Arguments as fwd."""
    if int(window) < 1:
        raise ValueError("window must be >= 1")
    return fwd(q, k, v, causal=True, scale=scale, out_dtype=out_dtype, out=out, lse=lse,
               stream=stream, window=int(window))


def fwd_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_scale: torch.Tensor,
            k_scale: torch.Tensor, v_scale: torch.Tensor, causal: bool = False,
            scale: Optional[float] = None, out_dtype: torch.dtype = torch.bfloat16,
            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
            stream=None, window: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention forward over FP8 E4M3 inputs: q (B,Hq,Nq,d), k/v (B,Hkv,Nk,d) uint8 bytes
    with fp32 per-head scales q_scale (Hq), k_scale/v_scale (Hkv) -> (o, lse).  The value
    of a q row of head h is q_scale[h] * e4m3(bytes); likewise K and V.  ``scale`` defaults
    to 1/sqrt(d); d must be 128."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, torch.uint8, 4)
    for t, n in ((q_scale, "q_scale"), (k_scale, "k_scale"), (v_scale, "v_scale")):
        _require(t, n, torch.float32, 1)
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if Bk != B or dk != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if q_scale.numel() != Hq or k_scale.numel() != Hkv or v_scale.numel() != Hkv:
        raise ValueError("q_scale must have Hq entries, k_scale and v_scale Hkv entries")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    out, lse = _fwd_outputs(q, (B, Hq, Nq, d), (B, Hq, Nq), out_dtype, out, lse, stream)
    odt = FA_F32 if out_dtype == torch.float32 else FA_BF16
    with _on_device(q, k, v, q_scale, k_scale, v_scale, out, lse) as dev:
        rc = load().fa_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_scale.data_ptr(),
                               k_scale.data_ptr(), v_scale.data_ptr(), out.data_ptr(), lse.data_ptr(),
                               B, Hq, Hkv, Nq, Nk, d, float(scale), int(bool(causal)), _c_int(window), odt,
                               _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def decode_workspace_size(B: int, Hq: int, Nmax: int, d: int) -> int:
    return int(load().fa_decode_workspace_size(B, Hq, Nmax, d))


def decode(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor, seqlens: torch.Tensor,
           scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
           want_lse: bool = True, stream=None):
    """Decode step: q (B,Hq,d) against caches (B,Hkv,Nmax,d) up to seqlens[b] (int32, device).

    Returns (o (B,Hq,d) bf16, lse (B,Hq) fp32 or None).  ``workspace`` is a uint8 CUDA
    tensor of at least decode_workspace_size(...) bytes; one is allocated if omitted.
    """
    _require(q, "q", torch.bfloat16, 3)
    _require(kcache, "kcache", torch.bfloat16, 4)
    _require(vcache, "vcache", torch.bfloat16, 4)
    _require(seqlens, "seqlens", torch.int32, 1)
    B, Hq, d = q.shape
    Bk, Hkv, Nmax, dk = kcache.shape
    if (Bk, dk) != (B, d) or tuple(vcache.shape) != tuple(kcache.shape) or seqlens.shape[0] != B:
        raise ValueError("shape mismatch between q, kcache, vcache and seqlens")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    workspace = _workspace(workspace, decode_workspace_size(B, Hq, Nmax, d), q.device, stream)
    out, lse = _decode_outputs(q, out, lse, want_lse, stream)
    with _on_device(q, kcache, vcache, seqlens, out, lse, workspace) as dev:
        rc = load().fa_decode(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(), seqlens.data_ptr(),
                              out.data_ptr(), lse.data_ptr() if lse is not None else None,
                              B, Hq, Hkv, Nmax, d, float(scale), workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def decode_paged(q: torch.Tensor, kpages: torch.Tensor, vpages: torch.Tensor,
                 block_table: torch.Tensor, seqlens: torch.Tensor, scale: Optional[float] = None,
                 workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Decode over a paged cache (fa_decode_paged): q (B,Hq,d); kpages/vpages
    (num_pages,Hkv,page_size,d) bf16; block_table int32 (B,max_pages) and seqlens int32[B]
    on the device.  Token t of sequence b is row t % page_size of page
    block_table[b, t // page_size].  Returns (o, lse) as decode does."""
    _require(q, "q", torch.bfloat16, 3)
    _require(kpages, "kpages", torch.bfloat16, 4)
    _require(vpages, "vpages", torch.bfloat16, 4)
    _require(block_table, "block_table", torch.int32, 2)
    _require(seqlens, "seqlens", torch.int32, 1)
    B, Hq, d = q.shape
    num_pages, Hkv, page_size, dk = kpages.shape
    max_pages = block_table.shape[1]
    if (dk != d or tuple(vpages.shape) != tuple(kpages.shape) or seqlens.shape[0] != B
            or block_table.shape[0] != B):
        raise ValueError("shape mismatch between q, kpages, vpages, block_table and seqlens")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    workspace = _workspace(workspace, decode_workspace_size(B, Hq, page_size * max_pages, d), q.device, stream)
    out, lse = _decode_outputs(q, out, lse, want_lse, stream)
    with _on_device(q, kpages, vpages, block_table, seqlens, out, lse, workspace) as dev:
        rc = load().fa_decode_paged(q.data_ptr(), kpages.data_ptr(), vpages.data_ptr(),
                                    block_table.data_ptr(), seqlens.data_ptr(), out.data_ptr(),
                                    lse.data_ptr() if lse is not None else None, B, Hq, Hkv,
                                    num_pages, page_size, max_pages, d, float(scale),
                                    workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def _decode_outputs(q, out, lse, want_lse, stream, out_dtype=torch.bfloat16):
    B, Hq, d = q.shape
    out = _output(out, "out", out_dtype, (B, Hq, d), q.device, stream)
    if lse is not None or want_lse:
        lse = _output(lse, "lse", torch.float32, (B, Hq), q.device, stream)
    return out, lse


def _workspace(workspace, need, device, stream):
    if workspace is None:
        return _new(max(need, 16), torch.uint8, device, stream, handed_back=False)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace


def decode_ex(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor, seqlens: torch.Tensor,
              scale: Optional[float] = None, out_dtype: torch.dtype = torch.bfloat16,
              workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """fa_decode_ex: decode with a bf16 or fp32 output (fp32 keeps a partial result exact
    enough to merge again with merge_lse)."""
    _require(q, "q", torch.bfloat16, 3)
    _require(kcache, "kcache", torch.bfloat16, 4)
    _require(vcache, "vcache", torch.bfloat16, 4)
    _require(seqlens, "seqlens", torch.int32, 1)
    B, Hq, d = q.shape
    Bk, Hkv, Nmax, dk = kcache.shape
    if (Bk, dk) != (B, d) or tuple(vcache.shape) != tuple(kcache.shape) or seqlens.shape[0] != B:
        raise ValueError("shape mismatch between q, kcache, vcache and seqlens")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    workspace = _workspace(workspace, decode_workspace_size(B, Hq, Nmax, d), q.device, stream)
    out, lse = _decode_outputs(q, out, lse, want_lse, stream, out_dtype)
    with _on_device(q, kcache, vcache, seqlens, out, lse, workspace) as dev:
        rc = load().fa_decode_ex(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(), seqlens.data_ptr(),
                                 out.data_ptr(), lse.data_ptr() if lse is not None else None,
                                 B, Hq, Hkv, Nmax, d, float(scale),
                                 FA_F32 if out_dtype == torch.float32 else FA_BF16, workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def merge_lse(o_parts: torch.Tensor, lse_parts: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None):
    """fa_merge_lse: o_parts (P, *rows, d) fp32 and lse_parts (P, *rows) fp32 (natural log,
    -inf = no keys) -> (o (*rows, d), lse (*rows))."""
    _require(o_parts, "o_parts", torch.float32, o_parts.dim())
    _require(lse_parts, "lse_parts", torch.float32, lse_parts.dim())
    if o_parts.dim() < 3 or tuple(o_parts.shape[:-1]) != tuple(lse_parts.shape):
        raise ValueError("o_parts must be (P, *rows, d) and lse_parts (P, *rows)")
    P, d = o_parts.shape[0], o_parts.shape[-1]
    row_shape = tuple(o_parts.shape[1:-1])
    rows = 1
    for x in row_shape:
        rows *= x
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    out = _output(out, "out", out_dtype, row_shape + (d,), o_parts.device, stream)
    lse = _output(lse, "lse", torch.float32, row_shape, o_parts.device, stream)
    with _on_device(o_parts, lse_parts, out, lse) as dev:
        rc = load().fa_merge_lse(o_parts.data_ptr(), lse_parts.data_ptr(), P, rows, d, out.data_ptr(),
                                 lse.data_ptr(), FA_F32 if out_dtype == torch.float32 else FA_BF16,
                                 _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def decode_fp8(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor, k_scale: torch.Tensor,
               v_scale: torch.Tensor, seqlens: torch.Tensor, scale: Optional[float] = None,
               workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Decode over an FP8 E4M3 cache (fa_decode_fp8): kcache/vcache uint8 (B,Hkv,Nmax,d)
    holding E4M3 bytes; k_scale/v_scale float32 (Hkv,) per-head dequantization scales."""
    _require(q, "q", torch.bfloat16, 3)
    _require(kcache, "kcache", torch.uint8, 4)
    _require(vcache, "vcache", torch.uint8, 4)
    _require(k_scale, "k_scale", torch.float32, 1)
    _require(v_scale, "v_scale", torch.float32, 1)
    _require(seqlens, "seqlens", torch.int32, 1)
    B, Hq, d = q.shape
    Bk, Hkv, Nmax, dk = kcache.shape
    if ((Bk, dk) != (B, d) or tuple(vcache.shape) != tuple(kcache.shape) or seqlens.shape[0] != B
            or k_scale.shape[0] != Hkv or v_scale.shape[0] != Hkv):
        raise ValueError("shape mismatch between q, the caches, the scales and seqlens")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    workspace = _workspace(workspace, decode_workspace_size(B, Hq, Nmax, d), q.device, stream)
    out, lse = _decode_outputs(q, out, lse, want_lse, stream)
    with _on_device(q, kcache, vcache, k_scale, v_scale, seqlens, out, lse, workspace) as dev:
        rc = load().fa_decode_fp8(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(), k_scale.data_ptr(),
                                  v_scale.data_ptr(), seqlens.data_ptr(), out.data_ptr(),
                                  lse.data_ptr() if lse is not None else None, B, Hq, Hkv, Nmax, d,
                                  float(scale), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def decode_paged_fp8(q: torch.Tensor, kpages: torch.Tensor, vpages: torch.Tensor,
                     k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor,
                     seqlens: torch.Tensor, scale: Optional[float] = None,
                     workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """FP8 decode over a paged cache (fa_decode_paged_fp8): pools uint8
    (num_pages,Hkv,page_size,d) of E4M3 bytes, per-head scales, block table as decode_paged."""
    _require(q, "q", torch.bfloat16, 3)
    _require(kpages, "kpages", torch.uint8, 4)
    _require(vpages, "vpages", torch.uint8, 4)
    _require(k_scale, "k_scale", torch.float32, 1)
    _require(v_scale, "v_scale", torch.float32, 1)
    _require(block_table, "block_table", torch.int32, 2)
    _require(seqlens, "seqlens", torch.int32, 1)
    B, Hq, d = q.shape
    num_pages, Hkv, page_size, dk = kpages.shape
    max_pages = block_table.shape[1]
    if (dk != d or tuple(vpages.shape) != tuple(kpages.shape) or seqlens.shape[0] != B
            or block_table.shape[0] != B or k_scale.shape[0] != Hkv or v_scale.shape[0] != Hkv):
        raise ValueError("shape mismatch between q, the pools, the scales, block_table and seqlens")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    workspace = _workspace(workspace, decode_workspace_size(B, Hq, page_size * max_pages, d), q.device, stream)
    out, lse = _decode_outputs(q, out, lse, want_lse, stream)
    with _on_device(q, kpages, vpages, k_scale, v_scale, block_table, seqlens, out, lse, workspace) as dev:
        rc = load().fa_decode_paged_fp8(q.data_ptr(), kpages.data_ptr(), vpages.data_ptr(),
                                        k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
                                        seqlens.data_ptr(), out.data_ptr(),
                                        lse.data_ptr() if lse is not None else None, B, Hq, Hkv,
                                        num_pages, page_size, max_pages, d, float(scale),
                                        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                        _stream_handle(stream, dev))
    _check(rc)
    return out, lse


# --------------- packed sequences, rotary positions, cache filling, page management
#
# These calls are short (a few microseconds on the device), so their checks come in two parts:
# one expression that a right argument passes (devices compared by index), and, when it does not,
# a function that finds out what is wrong.  The device is switched only when the tensors are not
# on the current one.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # current_stream without an object
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device_of(t, name) -> int:
    try:
        dev = t.get_device()
        if dev >= 0:
            return dev
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise ValueError(f"{name} must be a CUDA tensor")


def _other_device(t, name, dev):
    return ValueError(f"all tensors must be on cuda:{dev}; found {name} on {t.device}")


def _tensor(t, name, dtype, ndim, dev):
    """The pointer of a contiguous CUDA tensor of this type and rank on device number `dev`."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.dim() == ndim and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _require(t, name, dtype, ndim)
    raise _other_device(t, name, dev)


def _rows(t, name, dtypes, dev):
    """A (T, H, d) CUDA tensor whose heads are contiguous; tokens may be strided.  Returns
    (pointer, token stride in elements, T, H, d)."""
    try:
        T, H, d = t.shape
        st, sh, sd = t.stride()
        if sd == 1 and sh == d and st >= H * d and T > 1 and t.dtype in dtypes and t.get_device() == dev:
            return t.data_ptr(), st, T, H, d
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions (tokens, heads, d), got {t.dim()}")
    if t.get_device() != dev:
        raise _other_device(t, name, dev)
    T, H, d = t.shape
    st, sh, sd = t.stride()
    if T <= 1:  # the stride of a single token says nothing
        st = H * d
    if (sd != 1 and d > 1) or (sh != d and H > 1) or st < H * d:
        raise ValueError(f"{name} must have contiguous heads (strides (*, d, 1)), got {t.stride()}")
    return t.data_ptr(), st, T, H, d


def _launch(fn, dev, stream, *args):
    """Call the library with device number `dev` current, on `stream` or its current stream."""
    if stream is not None:
        handle = int(stream.cuda_stream)
    elif _raw_stream is not None:
        handle = _raw_stream(dev)
    else:
        handle = int(torch.cuda.current_stream(dev).cuda_stream)
    if dev == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != FA_OK:
        _check(rc)


def _scratch(workspace, size, sizes, dev, stream):
    """(pointer, bytes) of the caller's workspace, whose size the library checks, or of a new one of
    size(*sizes) bytes (kept alive by the third)."""
    if workspace is None:
        workspace = _new(max(size(*sizes), 16), torch.uint8, dev, stream, handed_back=False)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    elif workspace.get_device() != dev:
        raise _other_device(workspace, "workspace", dev)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _rotation(positions, inv_freq, axes, T, dev):
    """Pointers and sizes of the rotation's tables: positions (T,) or (A, T), inv_freq (F,)."""
    one = isinstance(positions, torch.Tensor) and positions.dim() == 1
    pp = _tensor(positions, "positions", torch.int32, 1 if one else 2, dev)
    pf = _tensor(inv_freq, "inv_freq", torch.float32, 1, dev)
    A, n = (1, positions.numel()) if one else positions.shape
    F = inv_freq.numel()
    if n != T:
        raise ValueError(f"positions must cover {T} tokens, got {tuple(positions.shape)}")
    pa = None
    if axes is not None:
        pa = _tensor(axes, "axes", torch.int32, 1, dev)
        if axes.numel() != F:
            raise ValueError("axes and inv_freq must have the same length")
    elif A != 1:
        raise ValueError("several position axes need `axes`, the axis of each frequency")
    return pp, pf, pa, F, A


_ROPE_TYPES = (torch.bfloat16, torch.float32)
_BF16 = (torch.bfloat16,)


def varlen_workspace_size(B: int, Tq: int, Hq: int, Hkv: int) -> int:
    return int(load().fa_fwd_varlen_workspace_size(B, Tq, Hq, Hkv))


def _varlen_outputs(q, dev, out_dtype, out, lse, stream):
    """Pointers of o (Tq,Hq,d) and lse (Hq,Tq), new ones unless given, and the output's code."""
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    Tq, Hq, d = q.shape
    if out is None:
        out = _new((Tq, Hq, d), out_dtype, dev, stream)
    if lse is None:
        lse = _new((Hq, Tq), torch.float32, dev, stream)
    po, pl = _tensor(out, "out", out_dtype, 3, dev), _tensor(lse, "lse", torch.float32, 2, dev)
    if out.shape != q.shape or tuple(lse.shape) != (Hq, Tq):
        raise ValueError(f"out must have shape {tuple(q.shape)} and lse {(Hq, Tq)}, "
                         f"got {tuple(out.shape)} and {tuple(lse.shape)}")
    return po, pl, out, lse, FA_F32 if out_dtype == torch.float32 else FA_BF16


def fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
               cu_seqlens_k: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None,
               window: int = 0, out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None):
    """Attention over packed sequences (fa_fwd_varlen): q (Tq,Hq,d), k/v (Tk,Hkv,d) bf16, tokens
    strided or not; cu_seqlens_q / cu_seqlens_k int32 (B+1,) on the device (the latter defaults to
    the former).  Returns (o (Tq,Hq,d), lse fp32 (Hq,Tq)); causal is bottom-right aligned in each
    sequence, a row that sees no key gives o = 0 and lse = -inf.  ``workspace`` is a uint8 CUDA
    tensor of varlen_workspace_size(B, Tq, Hq, Hkv) bytes; one is allocated if omitted."""
    dev = _device_of(q, "q")
    pq, sq, Tq, Hq, d = _rows(q, "q", _BF16, dev)
    pk, sk, Tk, Hkv, dk = _rows(k, "k", _BF16, dev)
    pv, sv, Tv, Hv, dv = _rows(v, "v", _BF16, dev)
    pcq = _tensor(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
    pck = pcq if cu_seqlens_k is None else _tensor(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1, dev)
    B = cu_seqlens_q.numel() - 1
    if (dk != d or (Tv, Hv, dv) != (Tk, Hkv, dk) or B < 1
            or (cu_seqlens_k is not None and cu_seqlens_k.numel() != B + 1)):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)} and the cu_seqlens")
    po, pl, out, lse, odt = _varlen_outputs(q, dev, out_dtype, out, lse, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if Tq == 0:
        return out, lse
    pw, nw, workspace = _scratch(workspace, varlen_workspace_size, (B, Tq, Hq, Hkv), dev, stream)
    _launch(load().fa_fwd_varlen, dev, stream, pq, pk, pv, po, pl, pcq, pck, B, Tq, Tk, Hq, Hkv, d, sq, sk, sv,
            float(scale), int(bool(causal)), _c_int(window), odt, pw, nw)
    return out, lse


def fwd_varlen_paged(q: torch.Tensor, kpages: torch.Tensor, vpages: torch.Tensor, block_table: torch.Tensor,
                     cu_seqlens_q: torch.Tensor, seqlens: torch.Tensor, causal: bool = True,
                     scale: Optional[float] = None, window: int = 0, out_dtype: torch.dtype = torch.bfloat16,
                     workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, stream=None):
    """fwd_varlen with the keys in a paged cache (fa_fwd_varlen_paged): q (Tq,Hq,d) bf16 packed by
    cu_seqlens_q int32 (B+1,); sequence b attends the first seqlens[b] tokens of its pages (pools
    (num_pages,Hkv,page_size,d) bf16, block_table int32 (B,max_pages)), of which its rows are the
    last: chunked prefill, or a prompt that continues a shared prefix."""
    dev = _device_of(q, "q")
    pq, sq, Tq, Hq, d = _rows(q, "q", _BF16, dev)
    pkp, pvp = _tensor(kpages, "kpages", torch.bfloat16, 4, dev), _tensor(vpages, "vpages", torch.bfloat16, 4, dev)
    pbt = _tensor(block_table, "block_table", torch.int32, 2, dev)
    pcq = _tensor(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
    psl = _tensor(seqlens, "seqlens", torch.int32, 1, dev)
    num_pages, Hkv, page_size, dk = kpages.shape
    B, max_pages = block_table.shape
    if dk != d or vpages.shape != kpages.shape or seqlens.shape[0] != B or cu_seqlens_q.shape[0] != B + 1:
        raise ValueError("shape mismatch between q, kpages, vpages, block_table, cu_seqlens_q and seqlens")
    po, pl, out, lse, odt = _varlen_outputs(q, dev, out_dtype, out, lse, stream)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if Tq == 0:
        return out, lse
    pw, nw, workspace = _scratch(workspace, varlen_workspace_size, (B, Tq, Hq, Hkv), dev, stream)
    _launch(load().fa_fwd_varlen_paged, dev, stream, pq, pkp, pvp, pbt, pcq, psl, po, pl, B, Tq, Hq, Hkv, num_pages,
            page_size, max_pages, d, sq, float(scale), int(bool(causal)), _c_int(window), odt, pw, nw)
    return out, lse


def rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor,
         axes: Optional[torch.Tensor] = None, interleaved: bool = False, inverse: bool = False,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions (fa_rope): q (T,Hq,d) and k (T,Hkv,d), bf16 or fp32, either may be None;
    positions int32 (T,) or (A,T); inv_freq fp32 (F,); axes int32 (F,), the axis of each
    frequency.  Returns (q_out, k_out), new tensors unless given (q_out=q works in place).
    Tokens may be strided (slices of a fused projection).  inverse=True is the transposed
    rotation: with the gradients of the outputs as q and k it returns those of the inputs."""
    if q is None and k is None:
        raise ValueError("q and k cannot both be None")
    first = q if q is not None else k
    dev = _device_of(first, "q" if q is not None else "k")
    types = (first.dtype,) if first.dtype in _ROPE_TYPES else _ROPE_TYPES
    pq, sq, pqo, sqo, Tq, Hq, dq = _turned(q, q_out, "q", types, dev) if q is not None else _NOTHING
    pk, sk, pko, sko, Tk, Hk, dk = _turned(k, k_out, "k", types, dev) if k is not None else _NOTHING
    if q is not None and k is not None and (Tq, dq) != (Tk, dk):
        raise ValueError("q and k must have the same tokens and head dim")
    T, d = (Tq, dq) if q is not None else (Tk, dk)
    if q is not None and q_out is None:
        q_out = _new(q.shape, q.dtype, dev, stream)
        pqo, sqo = q_out.data_ptr(), Hq * dq
    if k is not None and k_out is None:
        k_out = _new(k.shape, k.dtype, dev, stream)
        pko, sko = k_out.data_ptr(), Hk * dk
    if q is None:
        q_out = None
    if k is None:
        k_out = None
    pp, pf, pa, F, A = _rotation(positions, inv_freq, axes, T, dev)
    if T > 0:
        _launch(load().fa_rope, dev, stream, pq, pk, pqo, pko, pp, pf, pa, T, Hq, Hk, d, F, A, sq, sk, sqo, sko,
                FA_F32 if first.dtype is torch.float32 else FA_BF16, 1 if interleaved else 0, 1 if inverse else 0)
    return q_out, k_out


_NOTHING = (None, 0, None, 0, 0, 0, 0)


def _turned(x, out, name, types, dev):
    """Pointers, strides and sizes of one of rope's tensors and its output (if given)."""
    p, st, T, H, d = _rows(x, name, types, dev)
    if out is None:
        return p, st, None, 0, T, H, d
    po, so, To, Ho, do = _rows(out, name + "_out", types, dev)
    if (To, Ho, do) != (T, H, d):
        raise ValueError(f"{name}_out must have shape {(T, H, d)}, got {tuple(out.shape)}")
    return p, st, po, so, T, H, d


def _status(status, dev):
    """The pointer of a reservation's status word, if there is one."""
    if status is None:
        return None
    p = _tensor(status, "status", torch.int32, 1, dev)
    if status.numel() != 1:
        raise ValueError(f"status must have 1 entry, got {status.numel()}")
    return p


def _destination(k, v, kpages, vpages, block_table, cu_seqlens, seqlens, k_scale, v_scale, status, dev):
    """The checks fa_cache_append and fa_rope_append share: (k, v) rows and the pages' arguments."""
    pk, sk, T, Hkv, d = _rows(k, "k", _BF16, dev)
    pv, sv, Tv, Hv, dv = _rows(v, "v", _BF16, dev)
    fp8 = k_scale is not None or v_scale is not None
    pool = torch.uint8 if fp8 else torch.bfloat16
    pkp, pvp = _tensor(kpages, "kpages", pool, 4, dev), _tensor(vpages, "vpages", pool, 4, dev)
    pks = pvs = None
    if fp8:
        pks, pvs = _tensor(k_scale, "k_scale", torch.float32, 1, dev), _tensor(v_scale, "v_scale", torch.float32, 1, dev)
        if k_scale.numel() != Hkv or v_scale.numel() != Hkv:
            raise ValueError("k_scale and v_scale must have Hkv entries")
    pbt = _tensor(block_table, "block_table", torch.int32, 2, dev)
    pcu, psl = _tensor(cu_seqlens, "cu_seqlens", torch.int32, 1, dev), _tensor(seqlens, "seqlens", torch.int32, 1, dev)
    num_pages, H, page_size, dk = kpages.shape
    B, max_pages = block_table.shape
    if ((Tv, Hv, dv) != (T, Hkv, d) or (H, dk) != (Hkv, d) or vpages.shape != kpages.shape or seqlens.numel() != B
            or cu_seqlens.numel() != B + 1):
        raise ValueError("shape mismatch between k, v, the pools, block_table, cu_seqlens and seqlens")
    return (pk, sk), (pv, sv), (pkp, pvp, pks, pvs, pbt, pcu, psl, _status(status, dev)), (T, B, Hkv, num_pages, page_size, max_pages, d)


def cache_append(k: torch.Tensor, v: torch.Tensor, kpages: torch.Tensor, vpages: torch.Tensor,
                 block_table: torch.Tensor, cu_seqlens: torch.Tensor, seqlens: torch.Tensor,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None, stream=None,
                 status: Optional[torch.Tensor] = None):
    """Put new tokens' k and v (T,Hkv,d), packed by cu_seqlens int32 (B+1,), into the pages
    (fa_cache_append): the last positions of sequences of length seqlens (which include them).
    Pools (num_pages,Hkv,page_size,d) bf16, or uint8 E4M3 with k_scale / v_scale fp32 (Hkv,).
    ``status`` is what pages_reserve wrote for these tokens: if it refused, nothing is written."""
    dev = _device_of(kpages, "kpages")
    (pk, sk), (pv, sv), ptrs, (T, B, Hkv, num_pages, page_size, max_pages, d) = _destination(
        k, v, kpages, vpages, block_table, cu_seqlens, seqlens, k_scale, v_scale, status, dev)
    if T == 0:
        return
    _launch(load().fa_cache_append_ex, dev, stream, pk, pv, *ptrs, T, B, Hkv, num_pages, page_size, max_pages, d, sk, sv)


def rope_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                inv_freq: torch.Tensor, kpages: torch.Tensor, vpages: torch.Tensor, block_table: torch.Tensor,
                cu_seqlens: torch.Tensor, seqlens: torch.Tensor, axes: Optional[torch.Tensor] = None,
                interleaved: bool = False, k_scale: Optional[torch.Tensor] = None,
                v_scale: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None, stream=None,
                status: Optional[torch.Tensor] = None):
    """rope of q and k and cache_append of the rotated k and of v in one launch
    (fa_rope_append).  Returns q_out (None if q is None).  ``status`` as in cache_append; if the
    reservation was refused, q_out is not written either."""
    dev = _device_of(kpages, "kpages")
    (pk, sk), (pv, sv), ptrs, (T, B, Hkv, num_pages, page_size, max_pages, d) = _destination(
        k, v, kpages, vpages, block_table, cu_seqlens, seqlens, k_scale, v_scale, status, dev)
    pq = po = None
    sq = so = Hq = 0
    if q is not None:
        if q_out is None:
            q_out = _new(q.shape, torch.bfloat16, dev, stream)
        pq, sq, po, so, Tq, Hq, dq = _turned(q, q_out, "q", _BF16, dev)
        if (Tq, dq) != (T, d):
            raise ValueError("q and k must have the same tokens and head dim")
    pp, pf, pa, F, A = _rotation(positions, inv_freq, axes, T, dev)
    if T == 0:
        return q_out
    _launch(load().fa_rope_append_ex, dev, stream, pq, pk, pv, po, pp, pf, pa, *ptrs, T, B, Hq, Hkv, num_pages,
            page_size, max_pages, d, F, A, sq, sk, sv, so, 1 if interleaved else 0)
    return q_out


def _page_state(block_table, seqlens, refcount):
    dev = _device_of(block_table, "block_table")
    ptrs = (_tensor(block_table, "block_table", torch.int32, 2, dev), _tensor(seqlens, "seqlens", torch.int32, 1, dev),
            _tensor(refcount, "refcount", torch.int32, 1, dev))
    S, max_pages = block_table.shape
    if seqlens.numel() != S:
        raise ValueError("block_table and seqlens must have the same number of slots")
    return dev, ptrs, (S, max_pages, refcount.numel())


def _list(t, name, n, dev):
    p = _tensor(t, name, torch.int32, 1, dev)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} entries, got {t.numel()}")
    return p


def _copies(copies, n, dev, stream):
    if copies is None:
        copies = _new((n, 2), torch.int32, dev, stream)
    p = _tensor(copies, "copies", torch.int32, 2, dev)
    if tuple(copies.shape) != (n, 2):
        raise ValueError(f"copies must have shape {(n, 2)}, got {tuple(copies.shape)}")
    return p, copies


def pages_reserve_workspace_size(S: int, num_pages: int) -> int:
    return int(load().fa_pages_reserve_workspace_size(S, num_pages))


def pages_compact_workspace_size(num_pages: int) -> int:
    return int(load().fa_pages_compact_workspace_size(num_pages))


def pages_reserve(block_table: torch.Tensor, seqlens: torch.Tensor, refcount: torch.Tensor, add: torch.Tensor,
                  page_size: int, copies: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Lengthen every slot s by add[s] tokens (fa_pages_reserve).  Returns copies int32 (S,2):
    {old, new} for each shared last page that was split, else -1; pass it to pages_copy for
    every layer's pools.  Too few free pages: nothing changes; ``status`` int32 (1,) becomes
    FA_ERR_NO_PAGES (FA_OK after a call that took place), or without it get_error() says so.
    Tokens must not be appended after a refusal: pass the same ``status`` to rope_append or
    cache_append, which then write nothing, or look first."""
    dev, state, (S, max_pages, num_pages) = _page_state(block_table, seqlens, refcount)
    pa = _list(add, "add", S, dev)
    pc, copies = _copies(copies, S, dev, stream)
    pw, nw, workspace = _scratch(workspace, pages_reserve_workspace_size, (S, num_pages), dev, stream)
    _launch(load().fa_pages_reserve_ex, dev, stream, *state, pa, pc, _status(status, dev), S, max_pages, num_pages, _c_int(page_size), pw, nw)
    return copies


def pages_fork(block_table: torch.Tensor, seqlens: torch.Tensor, refcount: torch.Tensor, src: torch.Tensor,
               dst: torch.Tensor, page_size: int, lengths: Optional[torch.Tensor] = None, stream=None):
    """Empty slots dst become the first lengths[i] tokens (None: all) of slots src, sharing
    their pages (fa_pages_fork)."""
    dev, state, (S, max_pages, num_pages) = _page_state(block_table, seqlens, refcount)
    ps = _tensor(src, "src", torch.int32, 1, dev)
    n = src.numel()
    pd = _list(dst, "dst", n, dev)
    pl = _list(lengths, "lengths", n, dev) if lengths is not None else None
    if n == 0:
        return
    _launch(load().fa_pages_fork, dev, stream, *state, ps, pd, pl, n, S, max_pages, num_pages, _c_int(page_size))


def pages_free(block_table: torch.Tensor, seqlens: torch.Tensor, refcount: torch.Tensor, slots: torch.Tensor,
               page_size: int, keep: Optional[torch.Tensor] = None, stream=None):
    """Cut the listed slots to their first keep[i] tokens (None: none) and give back the pages
    behind them (fa_pages_free)."""
    dev, state, (S, max_pages, num_pages) = _page_state(block_table, seqlens, refcount)
    ps = _tensor(slots, "slots", torch.int32, 1, dev)
    n = slots.numel()
    pk = _list(keep, "keep", n, dev) if keep is not None else None
    if n == 0:
        return
    _launch(load().fa_pages_free, dev, stream, *state, ps, pk, n, S, max_pages, num_pages, _c_int(page_size))


def pages_compact(block_table: torch.Tensor, seqlens: torch.Tensor, refcount: torch.Tensor, page_size: int,
                  copies: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Move the live pages to the front of the pool (fa_pages_compact).  Returns copies int32
    (num_pages // 2, 2), {from, to} and -1 behind the last move, for pages_copy."""
    dev, state, (S, max_pages, num_pages) = _page_state(block_table, seqlens, refcount)
    pc, copies = _copies(copies, num_pages // 2, dev, stream)
    pw, nw, workspace = _scratch(workspace, pages_compact_workspace_size, (num_pages,), dev, stream)
    _launch(load().fa_pages_compact, dev, stream, *state, pc, S, max_pages, num_pages, _c_int(page_size), pw, nw)
    return copies


def pages_copy(kpages: torch.Tensor, vpages: Optional[torch.Tensor], copies: torch.Tensor, stream=None):
    """Copy page copies[i,0] to page copies[i,1] in both pools (fa_pages_copy); -1 is skipped.
    Pools (num_pages,Hkv,page_size,d), bf16 or uint8."""
    dev, dtype = _device_of(kpages, "kpages"), kpages.dtype
    if dtype not in (torch.bfloat16, torch.uint8):
        raise ValueError(f"kpages must be bfloat16 or uint8, got {dtype}")
    pk = _tensor(kpages, "kpages", dtype, 4, dev)
    pv = None
    if vpages is not None:
        pv = _tensor(vpages, "vpages", dtype, 4, dev)
        if vpages.shape != kpages.shape:
            raise ValueError("kpages and vpages must have the same shape")
    pc = _tensor(copies, "copies", torch.int32, 2, dev)
    if copies.shape[1] != 2:
        raise ValueError(f"copies must have shape (n, 2), got {tuple(copies.shape)}")
    num_pages, Hkv, page_size, d = kpages.shape
    if copies.shape[0] == 0:
        return
    _launch(load().fa_pages_copy, dev, stream, pk, pv, pc, copies.shape[0], num_pages,
            Hkv * page_size * d * kpages.element_size())


def get_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device-side status; where several were
    recorded, the next call returns the next."""
    return int(load().fa_get_error(_stream_handle(stream)))


def set_wait_limit_ns(ns: int):
    load().fa_set_wait_limit_ns(int(ns))


def fwd_selftest_timeout(q, k, v, causal=False, scale=None, stream=None):
    """Run the prefill kernel with its score-ready signal withheld (time-limit self-test)."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _fwd_outputs(q, (B, Hq, Nq, d), (B, Hq, Nq), torch.bfloat16, None, None, stream)
    with _on_device(q, k, v, out, lse) as dev:
        rc = load().fa_fwd_selftest_timeout(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                            lse.data_ptr(), B, Hq, Hkv, Nq, Nk, d, float(scale),
                                            int(bool(causal)), _stream_handle(stream, dev))
    _check(rc)
    return out, lse


def decode_selftest_timeout(q, kcache, vcache, seqlens, k_scale=None, v_scale=None, scale=None, stream=None):
    """Run a decode (bf16 caches, or E4M3 caches when both scales are given) with the split
    kernel's first copy withheld in every CTA (time-limit self-test)."""
    B, Hq, d = q.shape
    Hkv, Nmax = kcache.shape[1], kcache.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _decode_outputs(q, None, None, True, stream)
    ws = _workspace(None, decode_workspace_size(B, Hq, Nmax, d), q.device, stream)
    with _on_device(q, kcache, vcache, seqlens, out, lse, ws, k_scale, v_scale) as dev:
        rc = load().fa_decode_selftest_timeout(
            q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(),
            k_scale.data_ptr() if k_scale is not None else None,
            v_scale.data_ptr() if v_scale is not None else None, seqlens.data_ptr(), out.data_ptr(),
            lse.data_ptr(), B, Hq, Hkv, Nmax, d, float(scale), ws.data_ptr(), ws.numel(),
            _stream_handle(stream, dev))
    _check(rc)
    return out, lse


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def decode_noalloc(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                   seqlens: torch.Tensor, scale: Optional[float] = None,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   stream=None):
    """Decode step through fa_decode_noalloc: same result as ``decode`` but the library
    uses its own fixed 32 MiB scratch instead of a workspace, for callers that cannot
    allocate device memory.  ``out`` and ``lse`` must then be passed in by the caller;
    calls that overlap on the GPU share the scratch and must be ordered."""
    _require(q, "q", torch.bfloat16, 3)
    _require(kcache, "kcache", torch.bfloat16, 4)
    _require(vcache, "vcache", torch.bfloat16, 4)
    _require(seqlens, "seqlens", torch.int32, 1)
    B, Hq, d = q.shape
    Bk, Hkv, Nmax, dk = kcache.shape
    if (Bk, dk) != (B, d) or tuple(vcache.shape) != tuple(kcache.shape) or seqlens.shape[0] != B:
        raise ValueError("shape mismatch between q, kcache, vcache and seqlens")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        raise ValueError("decode_noalloc writes into a caller-provided `out`")
    out, lse = _decode_outputs(q, out, lse, False, stream)
    with _on_device(q, kcache, vcache, seqlens, out, lse) as dev:
        rc = load().fa_decode_noalloc(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(),
                                      seqlens.data_ptr(), out.data_ptr(),
                                      lse.data_ptr() if lse is not None else None,
                                      B, Hq, Hkv, Nmax, d, float(scale), _stream_handle(stream, dev))
    _check(rc)
    return out, lse
