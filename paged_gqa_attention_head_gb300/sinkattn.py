"""Thin ctypes binding of libsinkattn (include/sinkattn.h).

Argument marshalling only: tensors are checked (device, dtype, contiguity,
shape), their device pointers and the current CUDA stream are passed to the C
ABI, and error codes become exceptions.  Every step of the attention runs in
the library's CUDA kernels; there is no fallback.  Workspaces are torch
allocations owned by this module (one per device and size, zero-initialised).
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
import warnings
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsinkattn.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE_TOO_SMALL, ERR_CUDA = range(5)
STATUS_BAD_PAGE, STATUS_BAD_LENGTH, STATUS_BAD_CU_SEQLENS, STATUS_WAIT_TIMEOUT = 1, 2, 4, 8
STATUS_VALUE_RANGE, STATUS_NO_PAGES = 16, 32
FLAG_LAUNCH_NEXT_EARLY, FLAG_START_EARLY = 1, 2
PAGE_SIZE = 16

# every symbol the header declares, with (restype, argtypes)
_P, _I32, _F, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_I64 = ctypes.c_int64


class PagedDesc(ctypes.Structure):
    _fields_ = [("num_seqs", _I32), ("num_qo_heads", _I32), ("num_kv_heads", _I32),
                ("head_dim", _I32), ("page_size", _I32), ("num_pages", _I32),
                ("max_pages_per_seq", _I32), ("window", _I32), ("max_sms", _I32),
                ("wait_limit_us", _I32), ("flags", _I32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_context", _I32), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("factor", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("original_context", _I32), ("scaling", _I32),
                ("rotary_dim", _I32), ("interleaved", _I32)]


_DP = ctypes.POINTER(PagedDesc)
SIGNATURES = {
    "sinkattn_error_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sinkattn_version": (ctypes.c_int, []),
    "sinkattn_last_cuda_error": (ctypes.c_char_p, []),
    "sinkattn_decode_workspace_size": (ctypes.c_int, [_DP, ctypes.POINTER(_SZ)]),
    "sinkattn_workspace_init": (ctypes.c_int, [_P, _SZ, _P]),
    "sinkattn_decode": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_decode_splitkv": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_decode_merge": (ctypes.c_int, [_P, _P, _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_decode_append": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _SZ,
                                              _P]),
    "sinkattn_decode_append_rope": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _F,
                                                   ctypes.POINTER(RopeDesc), _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_decode_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _P]),
    "sinkattn_prefill_workspace_size": (ctypes.c_int, [_DP, ctypes.POINTER(_SZ)]),
    "sinkattn_prefill": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _F, _P, _P, _DP,
                                        _P, _SZ, _P]),
    "sinkattn_prefill_noncausal": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _F, _P, _P, _DP, _P, _SZ,
                                                  _P]),
    "sinkattn_prefill_fp8": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _F, _P,
                                            _P, _DP, _P, _SZ, _P]),
    "sinkattn_append_kv": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_decode_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _SZ,
                                           _P]),
    "sinkattn_decode_fp8_splitkv": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _DP,
                                                   _P, _SZ, _P]),
    "sinkattn_append_kv_fp8": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _DP, _P, _SZ,
                                              _P]),
    "sinkattn_append_kv_int8": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _I32, _P, _P, _P, _P, _P, _DP, _P,
                                               _SZ, _P]),
    "sinkattn_decode_int8_workspace_size": (ctypes.c_int, [_DP, ctypes.POINTER(_SZ)]),
    "sinkattn_decode_int8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_decode_int8_report": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _SZ, _P, _P]),
    "sinkattn_prefill_int8_workspace_size": (ctypes.c_int, [_DP, _I32, ctypes.POINTER(_SZ)]),
    "sinkattn_prefill_int8": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _F, _P, _P, _DP,
                                             _P, _SZ, _P]),
    "sinkattn_prefill_int8_report": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _F, _P, _P, _DP,
                                                    _P, _SZ, _P, _P]),
    "sinkattn_append_kv_int4": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _I32, _P, _DP, _P, _SZ, _P]),
    "sinkattn_unpack_kv_int4": (ctypes.c_int, [_P, _P, _I32, _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_decode_int4_workspace_size": (ctypes.c_int, [_DP, ctypes.POINTER(_SZ)]),
    "sinkattn_decode_int4": (ctypes.c_int, [_P, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _SZ, _P, _P]),
    "sinkattn_prefill_int4_workspace_size": (ctypes.c_int, [_DP, _I32, ctypes.POINTER(_SZ)]),
    "sinkattn_prefill_int4": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _F, _P, _P, _DP, _P, _SZ, _P, _P]),
    "sinkattn_plan_step": (ctypes.c_int, [_P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_release_pages": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_qk_norm_rope": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _P, _F, _P, _I32,
                                             ctypes.POINTER(RotaryDesc), _P, _P, _DP, _P, _SZ, _P]),
    "sinkattn_get_status": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_uint32), _P]),
}

_lib = None


class SinkAttnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        detail = ""
        if code == ERR_CUDA:
            detail = f" [{load().sinkattn_last_cuda_error().decode()}]"
        super().__init__(f"{what}: {error_string(code)} ({code}){detail}")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libsinkattn.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m "
                               "paged_gqa_attention_head_gb300.build` (needs nvcc)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def error_string(code: int) -> str:
    return load().sinkattn_error_string(code).decode()


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise SinkAttnError(rc, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device, ndim: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_workspaces: dict = {}


def workspace(nbytes: int, device: torch.device, tag: str = "default") -> torch.Tensor:
    """A zero-initialised uint8 device buffer of at least nbytes, cached per (device, tag)."""
    key = (device, tag)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def paged_desc(num_seqs, num_qo_heads, num_kv_heads, head_dim, num_pages, max_pages_per_seq,
               page_size=PAGE_SIZE, window=0, max_sms=0, wait_limit_us=0, flags=0) -> PagedDesc:
    """window > 0: sliding window (each query sees the keys at its last `window`
    positions); 0: full attention.  max_sms > 0: the persistent decode and prefill grids
    use at most that many SMs (the rest stay free for concurrent work on other streams);
    0: all SMs.  wait_limit_us > 0: give-up time of the kernels' pipeline waits (0: 2 s).
    flags: FLAG_LAUNCH_NEXT_EARLY (prefill) / FLAG_START_EARLY (split-KV decode), the
    overlap of a prefill and the decode after it on one stream."""
    return PagedDesc(num_seqs, num_qo_heads, num_kv_heads, head_dim, page_size, num_pages,
                     max_pages_per_seq, int(window), int(max_sms), int(wait_limit_us), int(flags))


_ws_sizes: dict = {}


def decode_workspace_size(desc: PagedDesc) -> int:
    """Bytes of decode workspace for desc on the current device (memoised)."""
    key = (torch.cuda.current_device() if torch.cuda.is_available() else -1,
           tuple(getattr(desc, f) for f, _ in desc._fields_))
    n = _ws_sizes.get(key)
    if n is None:
        c = _SZ()
        _check(load().sinkattn_decode_workspace_size(ctypes.byref(desc), ctypes.byref(c)),
               "decode_workspace_size")
        n = _ws_sizes[key] = c.value
    return n


def prefill_workspace_size(desc: PagedDesc) -> int:
    n = _SZ()
    _check(load().sinkattn_prefill_workspace_size(ctypes.byref(desc), ctypes.byref(n)),
           "prefill_workspace_size")
    return n.value


def get_status(ws: torch.Tensor) -> int:
    """Read and clear the device status word of a workspace (synchronous)."""
    v = ctypes.c_uint32()
    _check(load().sinkattn_get_status(_ptr(ws), ctypes.byref(v), _stream(ws.device)), "get_status")
    return v.value


def _codes(t: torch.Tensor) -> torch.Tensor:
    """An FP8 E4M3 cache tensor as its uint8 codes (float8_e4m3fn tensors are viewed)."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _decode_prep(q, k_pages, v_pages, block_table, seq_lens, sinks, scale, out, lse, ws,
                 want_lse, window=0, kv_dtype=torch.bfloat16, max_sms=0, wait_limit_us=0, flags=0):
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(k_pages, "k_pages", kv_dtype, dev, 4)
    _need(v_pages, "v_pages", kv_dtype, dev, 4)
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(seq_lens, "seq_lens", torch.int32, dev, 1)
    B, Hq, D = q.shape
    num_pages, Hkv, P, D2 = k_pages.shape
    if D2 != D or tuple(v_pages.shape) != tuple(k_pages.shape) or P != PAGE_SIZE:
        raise ValueError("k_pages / v_pages must be [num_pages, Hkv, 16, D] matching q")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens rows must equal the batch")
    if sinks is not None:
        _need(sinks, "sinks", torch.float32, dev, 1)
        if sinks.shape[0] != Hq:
            raise ValueError("sinks must have one entry per query head")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", torch.bfloat16, dev, 3)
    if lse is None and want_lse:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=dev)
    elif lse is not None:
        _need(lse, "lse", torch.float32, dev, 2)
    desc = paged_desc(B, Hq, Hkv, D, num_pages, block_table.shape[1], window=window,
                      max_sms=max_sms, wait_limit_us=wait_limit_us, flags=flags)
    nbytes = decode_workspace_size(desc)
    if ws is None:
        ws = workspace(nbytes, dev)
    elif ws.numel() < nbytes:
        raise ValueError(f"workspace needs {nbytes} bytes")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    return desc, out, lse, ws, scale


def decode(q, k_pages, v_pages, block_table, seq_lens, sinks=None, scale=None, out=None, lse=None,
           workspace_buf=None, return_lse=True, window=0, max_sms=0, wait_limit_us=0, flags=0):
    """Split-KV paged decode with sinks (sinkattn_decode).  window > 0: sliding window;
    max_sms > 0: the split-KV grid on at most that many SMs.  Returns (out, lse)."""
    desc, out, lse, ws, scale = _decode_prep(q, k_pages, v_pages, block_table, seq_lens, sinks,
                                             scale, out, lse, workspace_buf, return_lse, window,
                                             max_sms=max_sms, wait_limit_us=wait_limit_us, flags=flags)
    _check(load().sinkattn_decode(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                                  _ptr(seq_lens), _ptr(sinks), scale, _ptr(out), _ptr(lse),
                                  ctypes.byref(desc), _ptr(ws), ws.numel(), _stream(q.device)),
           "sinkattn_decode")
    return out, lse


def decode_splitkv(q, k_pages, v_pages, block_table, seq_lens, sinks=None, scale=None, out=None,
                   lse=None, workspace_buf=None, return_lse=True, window=0, max_sms=0, wait_limit_us=0):
    """First decode kernel only (sinkattn_decode_splitkv); follow with decode_merge."""
    desc, out, lse, ws, scale = _decode_prep(q, k_pages, v_pages, block_table, seq_lens, sinks,
                                             scale, out, lse, workspace_buf, return_lse, window,
                                             max_sms=max_sms, wait_limit_us=wait_limit_us)
    _check(load().sinkattn_decode_splitkv(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                                          _ptr(seq_lens), _ptr(sinks), scale, _ptr(out), _ptr(lse),
                                          ctypes.byref(desc), _ptr(ws), ws.numel(),
                                          _stream(q.device)), "sinkattn_decode_splitkv")
    return out, lse, ws, desc


def decode_merge(seq_lens, sinks, out, lse, desc, ws):
    """Second decode kernel (sinkattn_decode_merge) on the split-KV kernel's workspace."""
    _check(load().sinkattn_decode_merge(_ptr(seq_lens), _ptr(sinks), _ptr(out), _ptr(lse),
                                        ctypes.byref(desc), _ptr(ws), ws.numel(),
                                        _stream(out.device)), "sinkattn_decode_merge")
    return out, lse


def prefill(q, k, v, cu_seqlens, sinks=None, scale=None, k_pages=None, v_pages=None,
            prefix_block_table=None, prefix_lens=None, out=None, lse=None, workspace_buf=None,
            return_lse=True, window=0, max_sms=0, wait_limit_us=0, flags=0):
    """Causal ragged prefill, optionally over a paged prefix (sinkattn_prefill).  window > 0:
    sliding window; max_sms > 0: the persistent grid on at most that many SMs.  Returns
    (out, lse)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(k, "k", torch.bfloat16, dev, 3)
    _need(v, "v", torch.bfloat16, dev, 3)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (T, Hkv, D) or tuple(v.shape) != (T, Hkv, D):
        raise ValueError("k / v must be [T, Hkv, D] matching q")
    n = cu_seqlens.shape[0] - 1
    if sinks is not None:
        _need(sinks, "sinks", torch.float32, dev, 1)
    num_pages = maxp = 0
    if k_pages is not None:
        _need(k_pages, "k_pages", torch.bfloat16, dev, 4)
        _need(v_pages, "v_pages", torch.bfloat16, dev, 4)
        _need(prefix_block_table, "prefix_block_table", torch.int32, dev, 2)
        _need(prefix_lens, "prefix_lens", torch.int32, dev, 1)
        num_pages, maxp = k_pages.shape[0], prefix_block_table.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(T, Hq, dtype=torch.float32, device=dev)
    desc = paged_desc(n, Hq, Hkv, D, num_pages, maxp, window=window, max_sms=max_sms,
                      wait_limit_us=wait_limit_us, flags=flags)
    nbytes = prefill_workspace_size(desc)
    ws = workspace_buf if workspace_buf is not None else workspace(nbytes, dev, "prefill")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check(load().sinkattn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), T, _ptr(k_pages),
                                   _ptr(v_pages), _ptr(prefix_block_table), _ptr(prefix_lens),
                                   _ptr(sinks), scale, _ptr(out), _ptr(lse), ctypes.byref(desc),
                                   _ptr(ws), ws.numel(), _stream(dev)), "sinkattn_prefill")
    return out, lse


def prefill_noncausal(q, k, v, cu_seqlens, sinks=None, scale=None, out=None, lse=None,
                      workspace_buf=None, return_lse=True, max_sms=0, wait_limit_us=0):
    """Non-causal ragged prefill without a KV cache (sinkattn_prefill_noncausal): query t of
    request i attends every token of request i.  Returns (out, lse)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(k, "k", torch.bfloat16, dev, 3)
    _need(v, "v", torch.bfloat16, dev, 3)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (T, Hkv, D) or tuple(v.shape) != (T, Hkv, D):
        raise ValueError("k / v must be [T, Hkv, D] matching q")
    n = cu_seqlens.shape[0] - 1
    if sinks is not None:
        _need(sinks, "sinks", torch.float32, dev, 1)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(T, Hq, dtype=torch.float32, device=dev)
    desc = paged_desc(n, Hq, Hkv, D, 0, 0, max_sms=max_sms, wait_limit_us=wait_limit_us)
    nbytes = prefill_workspace_size(desc)
    ws = workspace_buf if workspace_buf is not None else workspace(nbytes, dev, "prefill")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check(load().sinkattn_prefill_noncausal(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), T, _ptr(sinks),
                                             scale, _ptr(out), _ptr(lse), ctypes.byref(desc), _ptr(ws),
                                             ws.numel(), _stream(dev)), "sinkattn_prefill_noncausal")
    return out, lse


def prefill_fp8(q, k, v, cu_seqlens, sinks=None, scale=None, k_pages=None, v_pages=None,
                k_scale=None, v_scale=None, prefix_block_table=None, prefix_lens=None, out=None,
                lse=None, workspace_buf=None, return_lse=True, window=0, max_sms=0, wait_limit_us=0):
    """Chunked prefill over an FP8 E4M3 paged prefix (sinkattn_prefill_fp8): k_pages / v_pages
    uint8 (or float8_e4m3fn) [num_pages, Hkv, 16, D] codes, k_scale / v_scale float32 [Hkv] or
    None (1); the new tokens' q, k, v bf16.  Returns (out, lse)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(k, "k", torch.bfloat16, dev, 3)
    _need(v, "v", torch.bfloat16, dev, 3)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (T, Hkv, D) or tuple(v.shape) != (T, Hkv, D):
        raise ValueError("k / v must be [T, Hkv, D] matching q")
    if k_pages is None or v_pages is None or prefix_block_table is None or prefix_lens is None:
        raise ValueError("prefill_fp8 needs the FP8 prefix pages, block table and lengths")
    k_pages, v_pages = _codes(k_pages), _codes(v_pages)
    _need(k_pages, "k_pages", torch.uint8, dev, 4)
    _need(v_pages, "v_pages", torch.uint8, dev, 4)
    _need(prefix_block_table, "prefix_block_table", torch.int32, dev, 2)
    _need(prefix_lens, "prefix_lens", torch.int32, dev, 1)
    _scales(k_scale, v_scale, Hkv, dev)
    if sinks is not None:
        _need(sinks, "sinks", torch.float32, dev, 1)
    n = cu_seqlens.shape[0] - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(T, Hq, dtype=torch.float32, device=dev)
    desc = paged_desc(n, Hq, Hkv, D, k_pages.shape[0], prefix_block_table.shape[1], window=window,
                      max_sms=max_sms, wait_limit_us=wait_limit_us)
    ws = workspace_buf if workspace_buf is not None else workspace(prefill_workspace_size(desc), dev,
                                                                   "prefill")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check(load().sinkattn_prefill_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), T, _ptr(k_pages),
                                       _ptr(v_pages), _ptr(k_scale), _ptr(v_scale),
                                       _ptr(prefix_block_table), _ptr(prefix_lens), _ptr(sinks), scale,
                                       _ptr(out), _ptr(lse), ctypes.byref(desc), _ptr(ws), ws.numel(),
                                       _stream(dev)), "sinkattn_prefill_fp8")
    return out, lse


def append_kv(k, v, cu_seqlens, block_table, start_pos, k_pages, v_pages, workspace_buf=None):
    """Scatter new K/V rows into the paged cache in place (sinkattn_append_kv)."""
    dev = k.device
    _need(k, "k", torch.bfloat16, dev, 3)
    _need(v, "v", torch.bfloat16, dev, 3)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(start_pos, "start_pos", torch.int32, dev, 1)
    _need(k_pages, "k_pages", torch.bfloat16, dev, 4)
    _need(v_pages, "v_pages", torch.bfloat16, dev, 4)
    T, Hkv, D = k.shape
    n = cu_seqlens.shape[0] - 1
    desc = paged_desc(n, Hkv, Hkv, D, k_pages.shape[0], block_table.shape[1])
    ws = workspace_buf if workspace_buf is not None else workspace(256, dev, "append")
    _check(load().sinkattn_append_kv(_ptr(k), _ptr(v), _ptr(cu_seqlens), T, _ptr(block_table),
                                     _ptr(start_pos), _ptr(k_pages), _ptr(v_pages),
                                     ctypes.byref(desc), _ptr(ws), ws.numel(), _stream(dev)),
           "sinkattn_append_kv")
    return k_pages, v_pages


def _scales(k_scale, v_scale, Hkv, dev):
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is not None:
            _need(t, name, torch.float32, dev, 1)
            if t.shape[0] != Hkv:
                raise ValueError(f"{name} must have one entry per KV head")


def decode_append(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, sinks=None, scale=None,
                  out=None, lse=None, workspace_buf=None, return_lse=True, window=0, max_sms=0,
                  wait_limit_us=0):
    """Decode step with its K/V append (sinkattn_decode_append): the new rows k_new / v_new
    [B, Hkv, D] go into the cache at position seq_lens - 1 (seq_lens counts them) and are
    attended in the same pass.  k_pages / v_pages are written in place.  Returns (out, lse)."""
    desc, out, lse, ws, scale = _decode_prep(q, k_pages, v_pages, block_table, seq_lens, sinks,
                                             scale, out, lse, workspace_buf, return_lse, window,
                                             max_sms=max_sms, wait_limit_us=wait_limit_us)
    B, Hkv, D = q.shape[0], k_pages.shape[1], q.shape[2]
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _need(t, name, torch.bfloat16, q.device, 3)
        if tuple(t.shape) != (B, Hkv, D):
            raise ValueError(f"{name} must be [B, Hkv, D] = {(B, Hkv, D)}")
    _check(load().sinkattn_decode_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages),
                                         _ptr(v_pages), _ptr(block_table), _ptr(seq_lens),
                                         _ptr(sinks), scale, _ptr(out), _ptr(lse), ctypes.byref(desc),
                                         _ptr(ws), ws.numel(), _stream(q.device)),
           "sinkattn_decode_append")
    return out, lse


def rope_desc(base: float, factor: float = 1.0, original_context: int = 4096,
              beta_fast: float = 32.0, beta_slow: float = 1.0) -> RopeDesc:
    """Rotary-embedding parameters (NeoX layout, YaRN scaling; factor 1 = plain RoPE)."""
    return RopeDesc(float(base), float(factor), int(original_context), float(beta_fast),
                    float(beta_slow))


def decode_append_rope(q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, sinks=None,
                       scale=None, rope: Optional[RopeDesc] = None, out=None, lse=None,
                       workspace_buf=None, return_lse=True, window=0, max_sms=0,
                       wait_limit_us=0):
    """Decode step with rotary embedding and K/V append (sinkattn_decode_append_rope): q and
    k_new (not yet rotated) are rotated at position seq_lens - 1, the rotated key and v_new go
    into the cache there, and the rotated query attends.  rope: a RopeDesc (rope_desc(...)).
    k_pages / v_pages are written in place.  Returns (out, lse)."""
    if not isinstance(rope, RopeDesc):
        raise TypeError("rope must be a RopeDesc (see rope_desc)")
    desc, out, lse, ws, scale = _decode_prep(q, k_pages, v_pages, block_table, seq_lens, sinks,
                                             scale, out, lse, workspace_buf, return_lse, window,
                                             max_sms=max_sms, wait_limit_us=wait_limit_us)
    B, Hkv, D = q.shape[0], k_pages.shape[1], q.shape[2]
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        _need(t, name, torch.bfloat16, q.device, 3)
        if tuple(t.shape) != (B, Hkv, D):
            raise ValueError(f"{name} must be [B, Hkv, D] = {(B, Hkv, D)}")
    _check(load().sinkattn_decode_append_rope(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pages),
                                              _ptr(v_pages), _ptr(block_table), _ptr(seq_lens),
                                              _ptr(sinks), scale, ctypes.byref(rope), _ptr(out),
                                              _ptr(lse), ctypes.byref(desc), _ptr(ws), ws.numel(),
                                              _stream(q.device)), "sinkattn_decode_append_rope")
    return out, lse


def decode_fp8(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, sinks=None, scale=None,
               out=None, lse=None, workspace_buf=None, return_lse=True, window=0, max_sms=0,
               wait_limit_us=0):
    """Split-KV paged decode over an FP8 E4M3 cache (sinkattn_decode_fp8).  k_pages / v_pages:
    uint8 (or float8_e4m3fn) [num_pages, Hkv, 16, D] codes; k_scale / v_scale: float32 [Hkv]
    per-KV-head scales or None (1).  Returns (out, lse)."""
    k_pages, v_pages = _codes(k_pages), _codes(v_pages)
    desc, out, lse, ws, scale = _decode_prep(q, k_pages, v_pages, block_table, seq_lens, sinks,
                                             scale, out, lse, workspace_buf, return_lse, window,
                                             kv_dtype=torch.uint8, max_sms=max_sms,
                                             wait_limit_us=wait_limit_us)
    _scales(k_scale, v_scale, k_pages.shape[1], q.device)
    _check(load().sinkattn_decode_fp8(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale),
                                      _ptr(v_scale), _ptr(block_table), _ptr(seq_lens), _ptr(sinks),
                                      scale, _ptr(out), _ptr(lse), ctypes.byref(desc), _ptr(ws),
                                      ws.numel(), _stream(q.device)), "sinkattn_decode_fp8")
    return out, lse


def decode_fp8_splitkv(q, k_pages, v_pages, k_scale, v_scale, block_table, seq_lens, sinks=None,
                       scale=None, out=None, lse=None, workspace_buf=None, return_lse=True, window=0,
                       max_sms=0, wait_limit_us=0):
    """First kernel of decode_fp8 only (sinkattn_decode_fp8_splitkv); follow with decode_merge."""
    k_pages, v_pages = _codes(k_pages), _codes(v_pages)
    desc, out, lse, ws, scale = _decode_prep(q, k_pages, v_pages, block_table, seq_lens, sinks,
                                             scale, out, lse, workspace_buf, return_lse, window,
                                             kv_dtype=torch.uint8, max_sms=max_sms,
                                             wait_limit_us=wait_limit_us)
    _scales(k_scale, v_scale, k_pages.shape[1], q.device)
    _check(load().sinkattn_decode_fp8_splitkv(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale),
                                              _ptr(v_scale), _ptr(block_table), _ptr(seq_lens),
                                              _ptr(sinks), scale, _ptr(out), _ptr(lse),
                                              ctypes.byref(desc), _ptr(ws), ws.numel(),
                                              _stream(q.device)), "sinkattn_decode_fp8_splitkv")
    return out, lse, ws, desc


def append_kv_fp8(k, v, k_scale, v_scale, cu_seqlens, block_table, start_pos, k_pages, v_pages,
                  workspace_buf=None):
    """Quantise new bf16 K/V rows to E4M3 codes (x / scale[g], nearest, saturating) and scatter
    them into an FP8 cache in place (sinkattn_append_kv_fp8)."""
    dev = k.device
    k_pages, v_pages = _codes(k_pages), _codes(v_pages)
    _need(k, "k", torch.bfloat16, dev, 3)
    _need(v, "v", torch.bfloat16, dev, 3)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(start_pos, "start_pos", torch.int32, dev, 1)
    _need(k_pages, "k_pages", torch.uint8, dev, 4)
    _need(v_pages, "v_pages", torch.uint8, dev, 4)
    T, Hkv, D = k.shape
    _scales(k_scale, v_scale, Hkv, dev)
    n = cu_seqlens.shape[0] - 1
    desc = paged_desc(n, Hkv, Hkv, D, k_pages.shape[0], block_table.shape[1])
    ws = workspace_buf if workspace_buf is not None else workspace(256, dev, "append")
    _check(load().sinkattn_append_kv_fp8(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale),
                                         _ptr(cu_seqlens), T, _ptr(block_table), _ptr(start_pos),
                                         _ptr(k_pages), _ptr(v_pages), ctypes.byref(desc), _ptr(ws),
                                         ws.numel(), _stream(dev)), "sinkattn_append_kv_fp8")
    return k_pages, v_pages


def decode_noalloc(q, k_pages, v_pages, block_table, seq_lens, sinks=None, scale=None, out=None,
                   lse=None, status=None, window=0):
    """sinkattn_decode_noalloc: the same decode with the library's fixed scratch array
    instead of a workspace, for callers that cannot allocate device memory.  Calls on
    one device must not overlap on the GPU.  status: optional int32/uint32 device
    tensor of one element receiving this call's status bits."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    _need(k_pages, "k_pages", torch.bfloat16, dev, 4)
    B, Hq, D = q.shape
    num_pages, Hkv = k_pages.shape[:2]
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=dev)
    desc = paged_desc(B, Hq, Hkv, D, num_pages, block_table.shape[1], window=window)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check(load().sinkattn_decode_noalloc(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                                          _ptr(seq_lens), _ptr(sinks), scale, _ptr(out), _ptr(lse),
                                          ctypes.byref(desc), _ptr(status), _stream(dev)),
           "sinkattn_decode_noalloc")
    return out, lse


# ---------------------------------------------------------------- INT8 cache, queries and keys
# The calls below run in steps of a few microseconds on the GPU, so what they cost on the host shows:
# descriptors and sizes are kept by their values, and a tensor is checked in one expression, its
# fault named only when there is one.
_Tensor = torch.Tensor
_functions: dict = {}  # the library's entry points by name
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_capturing = torch.cuda.is_current_stream_capturing


def _need_cuda(t: torch.Tensor, name: str) -> int:
    """The index of the tensor's CUDA device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, is on {t.device}")
    return t.get_device()


def _need_dense(t: torch.Tensor, name: str, dtype: torch.dtype, index: int, ndim: int) -> None:
    if not (type(t) is _Tensor and t.dtype is dtype and t.dim() == ndim and t.get_device() == index
            and t.is_contiguous()):
        _need(t, name, dtype, torch.device("cuda", index), ndim)


def _need_rows(t: torch.Tensor, name: str, index: int) -> tuple:
    """Checks bf16 rows [T, H, D], each row's [H, D] dense (a part of wider rows will do), and
    returns T, H, D and the row stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {torch.bfloat16}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims, got {tuple(t.shape)}")
    T, H, D = t.shape
    row, head, elem = t.stride()
    if (D > 1 and elem != 1) or (H > 1 and head != D):
        raise ValueError(f"{name}: the heads of a token must be dense")
    return T, H, D, row if T > 1 else H * D


_descs: dict = {}


def _desc_ref(*key):
    """A reference to the descriptor of these values (num_seqs, num_qo_heads, num_kv_heads, head_dim,
    num_pages, max_pages_per_seq, window, max_sms, wait_limit_us); descriptors are only read."""
    ref = _descs.get(key)
    if ref is None:
        if len(_descs) > 4096:
            _descs.clear()
        B, Hq, Hkv, D, pages, columns, window, max_sms, wait = key
        ref = _descs[key] = ctypes.byref(paged_desc(B, Hq, Hkv, D, pages, columns, window=window, max_sms=max_sms,
                                                    wait_limit_us=wait))
    return ref


def _call(index: int, what: str, *args) -> None:
    """The library call on the device `index`."""
    fn = _functions.get(what)
    if fn is None:
        fn = _functions[what] = getattr(load(), what)
    if _current_device() == index:
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc:
        raise SinkAttnError(rc, what)


def _captures(index: int) -> bool:
    """Whether the current stream of the device `index` is being captured."""
    if _current_device() == index:
        return _capturing()
    with torch.cuda.device(index):
        return _capturing()


def _status_buffer(index: int) -> Optional[torch.Tensor]:
    """The status word that the calls below share when they are given no workspace_buf (bits are OR-ed
    in, so streams and graphs may share it): workspace(256, device, "append"), read by
    default_status.  None while a capture runs before the word exists."""
    key = _append_keys.get(index)
    if key is None:
        key = _append_keys[index] = (torch.device("cuda", index), "append")
    ws = _workspaces.get(key)
    if ws is None:
        if _captures(index):
            warnings.warn("a captured call will not report its status: call default_status() once before the capture",
                          RuntimeWarning, stacklevel=3)
            return None
        with _status_lock:
            ws = _workspaces.get(key)
            if ws is None:  # zero before a call on another stream can set a bit
                ws = torch.zeros(256, dtype=torch.uint8, device=key[0])
                torch.cuda.current_stream(index).synchronize()
                _workspaces[key] = ws
    return ws


def _status_args(index: int) -> tuple:
    """Address and bytes of the shared status word; (None, 0) without one."""
    ws = _status_buffer(index)
    return (None, 0) if ws is None else (ws.data_ptr(), 256)


def default_status(device=None) -> int:
    """Read and clear the status bits (STATUS_*) of the calls on a CUDA device (default: the current
    one) that were given no workspace_buf: append_kv, append_kv_fp8, append_kv_int8, qk_norm_rope,
    decode_int8, prefill_int8, the 4-bit cache's calls and the page plan, from any thread or stream,
    eager or replayed from a graph.  It waits for the current stream; work on others counts once it has
    run.  Call it once before a first capture, so that the captured calls have a word to report to."""
    index = torch.device("cuda" if device is None else device).index
    return get_status(_status_buffer(_current_device() if index is None else index))


_append_keys: dict = {}
_status_lock = threading.Lock()


class _Scratch(threading.local):
    def __init__(self):
        self.buffers = {}


_scratch = _Scratch()


def _stream_workspace(nbytes: int, index: int, stream: int, tag: str, header: bool = True) -> torch.Tensor:
    """Default scratch of a call on the current stream: one buffer per (host thread, device, stream,
    tag).  So calls on two streams never share one, and neither do two threads that call on one
    stream: a call is a split kernel and its merge, and another thread's split kernel may come
    between them.  While the stream is captured the call gets a buffer of its own in the graph's
    memory, whose header, if the call reads it, the graph clears at each replay; so no two graphs, and
    no graph and an eager call, share one."""
    if _captures(index):
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=torch.device("cuda", index))
        if header:
            _call(index, "sinkattn_workspace_init", ws.data_ptr(), ws.numel(), stream)
        return ws
    key = (index, stream, tag)
    ws = _scratch.buffers.get(key)
    if ws is None or ws.numel() < nbytes:
        if ws is not None:  # used on this stream alone, so its memory may go back to the allocator
            nbytes = max(nbytes, 2 * ws.numel())
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=torch.device("cuda", index))
        _scratch.buffers[key] = ws
    return ws


def _workspace_args(ws: torch.Tensor, index: int) -> tuple:
    """Address and bytes of a workspace that the caller gave."""
    if not isinstance(ws, _Tensor):
        raise TypeError("workspace_buf must be a tensor")
    if ws.get_device() != index:
        raise ValueError(f"workspace_buf is on {ws.device}, expected cuda:{index}")
    if not ws.is_contiguous():
        raise ValueError("workspace_buf must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _need_int8_cache(k_pages, v_pages, kv_scales, index: int) -> tuple:
    _need_dense(k_pages, "k_pages", torch.int8, index, 4)
    _need_dense(v_pages, "v_pages", torch.int8, index, 4)
    _need_dense(kv_scales, "kv_scales", torch.float32, index, 3)
    shape = k_pages.shape
    if v_pages.shape != shape or shape[2] != PAGE_SIZE:
        raise ValueError("k_pages / v_pages must both be [num_pages, Hkv, 16, D]")
    if kv_scales.shape != (shape[0], shape[1], 2):
        raise ValueError("kv_scales must be [num_pages, Hkv, 2] (of K and of V)")
    return shape


def append_kv_int8(k, v, cu_seqlens, block_table, start_pos, k_pages, v_pages, kv_scales,
                   workspace_buf=None):
    """Quantise new bf16 K/V rows into an INT8 cache in place (sinkattn_append_kv_int8): k_pages /
    v_pages int8 [num_pages, Hkv, 16, D], kv_scales float32 [num_pages, Hkv, 2], all three updated;
    k, v [T, Hkv, D], each token's heads dense (parts of a fused projection's rows will do)."""
    dev = _need_cuda(k, "k")
    T, Hkv, D, ks = _need_rows(k, "k", dev)
    Tv, Hv, Dv, vs = _need_rows(v, "v", dev)
    _need_dense(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    _need_dense(block_table, "block_table", torch.int32, dev, 2)
    _need_dense(start_pos, "start_pos", torch.int32, dev, 1)
    pages, Hp, _, Dp = _need_int8_cache(k_pages, v_pages, kv_scales, dev)
    if (Tv, Hv, Dv) != (T, Hkv, D) or (Hp, Dp) != (Hkv, D):
        raise ValueError("k, v must be [T, Hkv, D] matching the pages")
    n, columns = block_table.shape
    if cu_seqlens.shape[0] != n + 1 or start_pos.shape[0] != n:
        raise ValueError("block_table / start_pos rows must equal the sequences of cu_seqlens")
    ws, nbytes = _status_args(dev) if workspace_buf is None else _workspace_args(workspace_buf, dev)
    _call(dev, "sinkattn_append_kv_int8", k.data_ptr(), ks, v.data_ptr(), vs, cu_seqlens.data_ptr(), T,
          block_table.data_ptr(), start_pos.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), kv_scales.data_ptr(),
          _desc_ref(n, Hkv, Hkv, D, pages, columns, 0, 0, 0), ws, nbytes, _raw_stream(dev))
    return k_pages, v_pages, kv_scales


def decode_int8_workspace_size(desc: PagedDesc) -> int:
    """Bytes of workspace that decode_int8 needs for desc on the current device."""
    c = _SZ()
    _check(load().sinkattn_decode_int8_workspace_size(ctypes.byref(desc), ctypes.byref(c)),
           "decode_int8_workspace_size")
    return c.value


def prefill_int8_workspace_size(desc: PagedDesc, total_tokens: int) -> int:
    """Bytes of workspace with which prefill_int8 works fastest for desc on the current device (256
    are enough for it to work)."""
    c = _SZ()
    _check(load().sinkattn_prefill_int8_workspace_size(ctypes.byref(desc), total_tokens, ctypes.byref(c)),
           "prefill_int8_workspace_size")
    return c.value


_int8_sizes: dict = {}


def _int8_size(what: str, index: int, ref, key, *more) -> int:
    n = _int8_sizes.get((what, index, key, *more))
    if n is None:
        if len(_int8_sizes) > 4096:
            _int8_sizes.clear()
        c = _SZ()
        _call(index, what, ref, *more, ctypes.byref(c))
        n = _int8_sizes[(what, index, key, *more)] = c.value
    return n


def _attention_outputs(q, out, lse, return_lse, index):
    """The out and lse of q [T, Hq, D], given or made."""
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_dense(out, "out", torch.bfloat16, index, 3)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is not None:
        _need_dense(lse, "lse", torch.float32, index, 2)
        if lse.shape != q.shape[:2]:
            raise ValueError("lse must have one entry per row and head of q")
    elif return_lse:
        lse = torch.empty((q.shape[0], q.shape[1]), dtype=torch.float32, device=q.device)
    return out, lse


def _need_sinks(sinks, heads: int, index: int) -> Optional[int]:
    if sinks is None:
        return None
    _need_dense(sinks, "sinks", torch.float32, index, 1)
    if sinks.shape[0] != heads:
        raise ValueError("sinks must have one entry per query head")
    return sinks.data_ptr()


def decode_int8(q, k_pages, v_pages, kv_scales, block_table, seq_lens, sinks=None, scale=None, out=None,
                lse=None, workspace_buf=None, return_lse=True, window=0, max_sms=0, wait_limit_us=0):
    """Split-KV paged decode over an INT8 cache with a scale per page and KV head
    (sinkattn_decode_int8).  Status bits go to workspace_buf's header, without one to
    default_status.  Returns (out, lse)."""
    dev = _need_cuda(q, "q")
    _need_dense(q, "q", torch.bfloat16, dev, 3)
    _need_dense(block_table, "block_table", torch.int32, dev, 2)
    _need_dense(seq_lens, "seq_lens", torch.int32, dev, 1)
    B, Hq, D = q.shape
    pages, Hkv, _, Dp = _need_int8_cache(k_pages, v_pages, kv_scales, dev)
    n, columns = block_table.shape
    if Dp != D:
        raise ValueError("k_pages / v_pages must be [num_pages, Hkv, 16, D] matching q")
    if n != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens rows must equal the batch")
    sk = _need_sinks(sinks, Hq, dev)
    out, lse = _attention_outputs(q, out, lse, return_lse, dev)
    key = (B, Hq, Hkv, D, pages, columns, window, max_sms, wait_limit_us)
    desc, stream = _desc_ref(*key), _raw_stream(dev)
    if workspace_buf is None:
        ws = _stream_workspace(_int8_size("sinkattn_decode_int8_workspace_size", dev, desc, key), dev, stream, "decode",
                               header=False)
        at, nbytes, (status, _) = ws.data_ptr(), ws.numel(), _status_args(dev)
    else:
        (at, nbytes), status = _workspace_args(workspace_buf, dev), None
    _call(dev, "sinkattn_decode_int8_report", q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), kv_scales.data_ptr(),
          block_table.data_ptr(), seq_lens.data_ptr(), sk, D ** -0.5 if scale is None else float(scale), out.data_ptr(),
          None if lse is None else lse.data_ptr(), desc, at, nbytes, status, stream)
    return out, lse


def prefill_int8(q, k, v, cu_seqlens, k_pages, v_pages, kv_scales, prefix_block_table, prefix_lens, sinks=None,
                 scale=None, out=None, lse=None, workspace_buf=None, return_lse=True, window=0, max_sms=0,
                 wait_limit_us=0):
    """Chunked prefill over an INT8 paged prefix with a scale per page and KV head
    (sinkattn_prefill_int8); the new tokens' q, k, v bf16.  Status bits go to workspace_buf's header,
    without one to default_status.  Returns (out, lse)."""
    dev = _need_cuda(q, "q")
    _need_dense(q, "q", torch.bfloat16, dev, 3)
    _need_dense(k, "k", torch.bfloat16, dev, 3)
    _need_dense(v, "v", torch.bfloat16, dev, 3)
    _need_dense(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    _need_dense(prefix_block_table, "prefix_block_table", torch.int32, dev, 2)
    _need_dense(prefix_lens, "prefix_lens", torch.int32, dev, 1)
    T, Hq, D = q.shape
    pages, Hkv, _, Dp = _need_int8_cache(k_pages, v_pages, kv_scales, dev)
    n, columns = prefix_block_table.shape
    if k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D) or Dp != D:
        raise ValueError("k / v must be [T, Hkv, D] matching q and the pages")
    if cu_seqlens.shape[0] != n + 1 or prefix_lens.shape[0] != n:
        raise ValueError("prefix_block_table / prefix_lens rows must equal the requests of cu_seqlens")
    sk = _need_sinks(sinks, Hq, dev)
    out, lse = _attention_outputs(q, out, lse, return_lse, dev)
    key = (n, Hq, Hkv, D, pages, columns, window, max_sms, wait_limit_us)
    desc, stream = _desc_ref(*key), _raw_stream(dev)
    if workspace_buf is None:
        ws = _stream_workspace(_int8_size("sinkattn_prefill_int8_workspace_size", dev, desc, key, T), dev, stream,
                               "prefill")
        at, nbytes, (status, _) = ws.data_ptr(), ws.numel(), _status_args(dev)
    else:
        (at, nbytes), status = _workspace_args(workspace_buf, dev), None
    _call(dev, "sinkattn_prefill_int8_report", q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), T,
          k_pages.data_ptr(), v_pages.data_ptr(), kv_scales.data_ptr(), prefix_block_table.data_ptr(),
          prefix_lens.data_ptr(), sk, D ** -0.5 if scale is None else float(scale), out.data_ptr(),
          None if lse is None else lse.data_ptr(), desc, at, nbytes, status, stream)
    return out, lse


# ---------------------------------------------------------------- 4-bit cache, page plan
def _need_int4_cache(kv_pages, index: int) -> tuple:
    """Pages, KV heads and head_dim of a 4-bit cache."""
    _need_dense(kv_pages, "kv_pages", torch.uint8, index, 5)
    pages, heads, two, rows, dim = kv_pages.shape
    if two != 2 or rows != 9:
        raise ValueError("kv_pages must be [num_pages, Hkv, 2, 9, D]")
    return pages, heads, dim


def append_kv_int4(k, v, slots, kv_pages, workspace_buf=None):
    """Quantise new bf16 K/V rows into the slots of a 4-bit cache, in place (sinkattn_append_kv_int4):
    kv_pages uint8 [num_pages, Hkv, 2, 9, D]; slots int64 [T] (page * 16 + place; negative: padding), for
    example a StepPlan's; k, v [T, Hkv, D], each token's heads dense (parts of a fused projection's rows
    will do)."""
    dev = _need_cuda(k, "k")
    T, Hkv, D, ks = _need_rows(k, "k", dev)
    Tv, Hv, Dv, vs = _need_rows(v, "v", dev)
    _need_dense(slots, "slots", torch.int64, dev, 1)
    pages, Hp, Dp = _need_int4_cache(kv_pages, dev)
    if (Tv, Hv, Dv) != (T, Hkv, D) or (Hp, Dp) != (Hkv, D):
        raise ValueError("k, v must be [T, Hkv, D] matching the pages")
    if slots.shape[0] != T:
        raise ValueError("slots must have one entry per token")
    ws, nbytes = _status_args(dev) if workspace_buf is None else _workspace_args(workspace_buf, dev)
    _call(dev, "sinkattn_append_kv_int4", k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(), T, kv_pages.data_ptr(),
          _desc_ref(0, Hkv, Hkv, D, pages, 0, 0, 0, 0), ws, nbytes, _raw_stream(dev))
    return kv_pages


def unpack_kv_int4(kv_pages, pages=None, k_out=None, v_out=None, workspace_buf=None):
    """Pages of a 4-bit cache as bf16 pages [n, Hkv, 16, D], exactly (sinkattn_unpack_kv_int4): those
    that pages (int32 [n]) names, or all.  Returns (k_pages, v_pages)."""
    dev = _need_cuda(kv_pages, "kv_pages")
    num_pages, Hkv, D = _need_int4_cache(kv_pages, dev)
    n, wanted = num_pages, None
    if pages is not None:
        _need_dense(pages, "pages", torch.int32, dev, 1)
        n, wanted = pages.shape[0], pages.data_ptr()
    shape = (n, Hkv, PAGE_SIZE, D)
    for name, o in (("k_out", k_out), ("v_out", v_out)):
        if o is not None:
            _need_dense(o, name, torch.bfloat16, dev, 4)
            if o.shape != shape:
                raise ValueError(f"{name} must be [n, Hkv, 16, D] = {shape}")
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=kv_pages.device)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    ws, nbytes = _status_args(dev) if workspace_buf is None else _workspace_args(workspace_buf, dev)
    _call(dev, "sinkattn_unpack_kv_int4", kv_pages.data_ptr(), wanted, n, k_out.data_ptr(), v_out.data_ptr(),
          _desc_ref(0, Hkv, Hkv, D, num_pages, 0, 0, 0, 0), ws, nbytes, _raw_stream(dev))
    return k_out, v_out


def decode_int4_workspace_size(desc: PagedDesc) -> int:
    """Bytes of workspace that decode_int4 needs for desc on the current device."""
    c = _SZ()
    _check(load().sinkattn_decode_int4_workspace_size(ctypes.byref(desc), ctypes.byref(c)),
           "decode_int4_workspace_size")
    return c.value


def prefill_int4_workspace_size(desc: PagedDesc, total_tokens: int) -> int:
    """Bytes of workspace with which prefill_int4 works fastest for desc on the current device (256
    are enough for it to work)."""
    c = _SZ()
    _check(load().sinkattn_prefill_int4_workspace_size(ctypes.byref(desc), total_tokens, ctypes.byref(c)),
           "prefill_int4_workspace_size")
    return c.value


def decode_int4(q, kv_pages, block_table, seq_lens, sinks=None, scale=None, out=None, lse=None, workspace_buf=None,
                return_lse=True, window=0, max_sms=0, wait_limit_us=0):
    """Split-KV paged decode over a 4-bit cache, uint8 [num_pages, Hkv, 2, 9, D] (sinkattn_decode_int4).
    Status bits go to workspace_buf's header, without one to default_status.  Returns (out, lse)."""
    dev = _need_cuda(q, "q")
    _need_dense(q, "q", torch.bfloat16, dev, 3)
    _need_dense(block_table, "block_table", torch.int32, dev, 2)
    _need_dense(seq_lens, "seq_lens", torch.int32, dev, 1)
    B, Hq, D = q.shape
    pages, Hkv, Dp = _need_int4_cache(kv_pages, dev)
    n, columns = block_table.shape
    if Dp != D:
        raise ValueError("kv_pages must be [num_pages, Hkv, 2, 9, D] matching q")
    if n != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens rows must equal the batch")
    sk = _need_sinks(sinks, Hq, dev)
    out, lse = _attention_outputs(q, out, lse, return_lse, dev)
    key = (B, Hq, Hkv, D, pages, columns, window, max_sms, wait_limit_us)
    desc, stream = _desc_ref(*key), _raw_stream(dev)
    if workspace_buf is None:
        ws = _stream_workspace(_int8_size("sinkattn_decode_int4_workspace_size", dev, desc, key), dev, stream, "decode",
                               header=False)
        at, nbytes, (status, _) = ws.data_ptr(), ws.numel(), _status_args(dev)
    else:
        (at, nbytes), status = _workspace_args(workspace_buf, dev), None
    _call(dev, "sinkattn_decode_int4", q.data_ptr(), kv_pages.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), sk,
          D ** -0.5 if scale is None else float(scale), out.data_ptr(), None if lse is None else lse.data_ptr(), desc, at,
          nbytes, status, stream)
    return out, lse


def prefill_int4(q, k, v, cu_seqlens, kv_pages, prefix_block_table, prefix_lens, sinks=None, scale=None, out=None,
                 lse=None, workspace_buf=None, return_lse=True, window=0, max_sms=0, wait_limit_us=0):
    """Chunked prefill over a 4-bit paged prefix (sinkattn_prefill_int4); the new tokens' q, k, v bf16.
    Status bits go to workspace_buf's header, without one to default_status.  Returns (out, lse)."""
    dev = _need_cuda(q, "q")
    _need_dense(q, "q", torch.bfloat16, dev, 3)
    _need_dense(k, "k", torch.bfloat16, dev, 3)
    _need_dense(v, "v", torch.bfloat16, dev, 3)
    _need_dense(cu_seqlens, "cu_seqlens", torch.int32, dev, 1)
    _need_dense(prefix_block_table, "prefix_block_table", torch.int32, dev, 2)
    _need_dense(prefix_lens, "prefix_lens", torch.int32, dev, 1)
    T, Hq, D = q.shape
    pages, Hkv, Dp = _need_int4_cache(kv_pages, dev)
    n, columns = prefix_block_table.shape
    if k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D) or Dp != D:
        raise ValueError("k / v must be [T, Hkv, D] matching q and the pages")
    if cu_seqlens.shape[0] != n + 1 or prefix_lens.shape[0] != n:
        raise ValueError("prefix_block_table / prefix_lens rows must equal the requests of cu_seqlens")
    sk = _need_sinks(sinks, Hq, dev)
    out, lse = _attention_outputs(q, out, lse, return_lse, dev)
    key = (n, Hq, Hkv, D, pages, columns, window, max_sms, wait_limit_us)
    desc, stream = _desc_ref(*key), _raw_stream(dev)
    if workspace_buf is None:
        ws = _stream_workspace(_int8_size("sinkattn_prefill_int4_workspace_size", dev, desc, key, T), dev, stream,
                               "prefill")
        at, nbytes, (status, _) = ws.data_ptr(), ws.numel(), _status_args(dev)
    else:
        (at, nbytes), status = _workspace_args(workspace_buf, dev), None
    _call(dev, "sinkattn_prefill_int4", q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), T,
          kv_pages.data_ptr(), prefix_block_table.data_ptr(), prefix_lens.data_ptr(), sk,
          D ** -0.5 if scale is None else float(scale), out.data_ptr(), None if lse is None else lse.data_ptr(), desc, at,
          nbytes, status, stream)
    return out, lse


class StepPlan(NamedTuple):
    """What a serving step's calls take (plan_step), all on the device."""
    cu_seqlens: torch.Tensor  # int32 [B + 1]
    start_pos: torch.Tensor   # int32 [B] tokens held before the step (prefix lengths, append positions)
    seq_lens: torch.Tensor    # int32 [B] and after it (what a decode attends)
    positions: torch.Tensor   # int32 [max_tokens] of the packed rows; -1: padding, or a request not served
    slots: torch.Tensor       # int64 [max_tokens] in the cache; -1 likewise
    num_free: torch.Tensor    # int32 [1] pages left


def _need_page_list(seq_lens, block_table, free_pages, num_free, index: int) -> tuple:
    """Requests, columns of the table and pages of the pool."""
    _need_dense(seq_lens, "seq_lens", torch.int32, index, 1)
    _need_dense(block_table, "block_table", torch.int32, index, 2)
    _need_dense(free_pages, "free_pages", torch.int32, index, 1)
    _need_dense(num_free, "num_free", torch.int32, index, 1)
    B, columns = block_table.shape
    if seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens rows must equal the batch")
    if num_free.shape[0] != 1:
        raise ValueError("num_free must have one entry")
    return B, columns, free_pages.shape[0]


def plan_step(new_lens, seq_lens, block_table, free_pages, num_free, max_tokens, update=False,
              workspace_buf=None) -> StepPlan:
    """Block-table entries, slots, positions and lengths of a serving step, on the device
    (sinkattn_plan_step).  new_lens, seq_lens int32 [B]: tokens that each request brings and holds;
    block_table int32 [B, columns] is updated in place; free_pages int32 [num_pages] (as long as the
    pool, however few are free), num_free int32 [1]: the free pages, a stack; max_tokens: rows of the
    packed step (those behind the last request are padding).  update: seq_lens and num_free take their
    new values in place, as a captured step needs; else they stay, and the plan holds the new ones.
    STATUS_NO_PAGES in workspace_buf's header, without one in default_status, tells that some request was
    not served."""
    dev = _need_cuda(new_lens, "new_lens")
    _need_dense(new_lens, "new_lens", torch.int32, dev, 1)
    B, columns, pages = _need_page_list(seq_lens, block_table, free_pages, num_free, dev)
    if new_lens.shape[0] != B:
        raise ValueError("new_lens must have one entry per request")
    at = new_lens.device
    cu = torch.empty(B + 1, dtype=torch.int32, device=at)
    positions = torch.empty(max_tokens, dtype=torch.int32, device=at)
    slots = torch.empty(max_tokens, dtype=torch.int64, device=at)
    if update:
        start, lens, left = torch.empty_like(seq_lens), seq_lens, num_free
    else:
        start, lens, left = seq_lens, torch.empty_like(seq_lens), torch.empty_like(num_free)
    ws, nbytes = _status_args(dev) if workspace_buf is None else _workspace_args(workspace_buf, dev)
    _call(dev, "sinkattn_plan_step", new_lens.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(),
          num_free.data_ptr(), max_tokens, cu.data_ptr(), start.data_ptr() if update else None, lens.data_ptr(),
          left.data_ptr(), positions.data_ptr(), slots.data_ptr(), _desc_ref(B, 1, 1, 64, pages, columns, 0, 0, 0), ws,
          nbytes, _raw_stream(dev))
    return StepPlan(cu, start, lens, positions, slots, left)


def release_pages(done, seq_lens, block_table, free_pages, num_free, update=False, workspace_buf=None):
    """The pages of the requests with done (bool [B]) back to the list of free pages, which is updated in
    place, and their lengths to 0 (sinkattn_release_pages).  A page must be its request's alone and not in
    the list yet: one that rows of the table share would come to two requests.  update as for plan_step.
    Returns (seq_lens, num_free)."""
    dev = _need_cuda(done, "done")
    _need_dense(done, "done", torch.bool, dev, 1)
    B, columns, pages = _need_page_list(seq_lens, block_table, free_pages, num_free, dev)
    if done.shape[0] != B:
        raise ValueError("done must have one entry per request")
    lens, left = (seq_lens, num_free) if update else (torch.empty_like(seq_lens), torch.empty_like(num_free))
    ws, nbytes = _status_args(dev) if workspace_buf is None else _workspace_args(workspace_buf, dev)
    _call(dev, "sinkattn_release_pages", done.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(),
          num_free.data_ptr(), lens.data_ptr(), left.data_ptr(), _desc_ref(B, 1, 1, 64, pages, columns, 0, 0, 0), ws, nbytes,
          _raw_stream(dev))
    return lens, left


ROTARY_SCALING = {"none": 0, "linear": 1, "yarn": 2, "wavelength": 3}


def rotary_desc(base: float, rotary_dim: int, factor: float = 1.0, scaling: str = "none",
                original_context: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                interleaved: bool = False) -> RotaryDesc:
    """Rotation of the first rotary_dim elements of each head (a multiple of 16): pairs (i, i +
    rotary_dim / 2), or (2i, 2i + 1) if interleaved; scaling "none", "linear", "yarn" or
    "wavelength" (SINKATTN_ROTARY_* in include/sinkattn.h)."""
    if scaling not in ROTARY_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALING)}, got {scaling!r}")
    return RotaryDesc(float(base), float(factor), float(beta_fast), float(beta_slow), int(original_context),
                      ROTARY_SCALING[scaling], int(rotary_dim), int(bool(interleaved)))


def _need_weight(w, name: str, D: int, index: int) -> Optional[int]:
    if w is None:
        return None
    _need_dense(w, name, torch.float32, index, 1)
    if w.shape[0] != D:
        raise ValueError(f"{name} must have head_dim entries")
    return w.data_ptr()


def _rows_output(x, o, name: str, index: int):
    if o is None:
        return torch.empty_like(x) if x.is_contiguous() else torch.empty_like(x, memory_format=torch.contiguous_format)
    _need_dense(o, name, torch.bfloat16, index, 3)
    if o.shape != x.shape:
        raise ValueError(f"{name} must have its input's shape")
    return o


def qk_norm_rope(q, k, positions=None, rotary: Optional[RotaryDesc] = None, q_weight=None, k_weight=None,
                 eps: float = 1e-6, q_out=None, k_out=None, workspace_buf=None):
    """Per-head RMS norm and rotary embedding of a step's queries and keys in one pass
    (sinkattn_qk_norm_rope).  q [T, Hq, D], k [T, Hkv, D] bf16, each token's heads dense (parts of a
    fused projection's rows will do); k may be None.  positions int32 [T] (negative: padding, the
    rows are left as they were); q_weight / k_weight float32 [D] or None (no norm); rotary None: no
    rotation.  q_out / k_out dense, or q / k themselves if dense.  Returns (q_out, k_out)."""
    dev = _need_cuda(q, "q")
    T, Hq, D, qs = _need_rows(q, "q", dev)
    ks, Hkv = 0, Hq
    if k is not None:
        Tk, Hkv, Dk, ks = _need_rows(k, "k", dev)
        if (Tk, Dk) != (T, D):
            raise ValueError("k must be [T, Hkv, D] matching q")
    elif k_out is not None:
        raise ValueError("k_out given without its input")
    pos = rot = None
    if rotary is not None:
        if not isinstance(rotary, RotaryDesc):
            raise TypeError("rotary must be a RotaryDesc (see rotary_desc)")
        _need_dense(positions, "positions", torch.int32, dev, 1)
        if positions.shape[0] != T:
            raise ValueError("positions must have one entry per token")
        pos, rot = positions.data_ptr(), ctypes.byref(rotary)
    wq, wk = _need_weight(q_weight, "q_weight", D, dev), _need_weight(k_weight, "k_weight", D, dev)
    q_out = _rows_output(q, q_out, "q_out", dev)
    if k is not None:
        k_out = _rows_output(k, k_out, "k_out", dev)
    ws, nbytes = _status_args(dev) if workspace_buf is None else _workspace_args(workspace_buf, dev)
    _call(dev, "sinkattn_qk_norm_rope", q.data_ptr(), qs, None if k is None else k.data_ptr(), ks, wq, wk, float(eps), pos, T,
          rot, q_out.data_ptr(), None if k is None else k_out.data_ptr(), _desc_ref(0, Hq, Hkv, D, 0, 0, 0, 0, 0),
          ws, nbytes, _raw_stream(dev))
    return q_out, k_out
