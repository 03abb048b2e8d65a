"""Python binding of libpa.so (the C ABI declared in include/pa.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  torch provides device memory and the current
stream.  There is no fallback: if libpa.so is missing or cannot be loaded,
every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re
import threading
from typing import Optional, Tuple

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "pa.h")

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA = range(5)
PA_FP16, PA_BF16 = 0, 1
PA_DEVERR_WAIT_TIMEOUT, PA_DEVERR_BAD_CONTEXT, PA_DEVERR_BAD_SLOT, PA_DEVERR_BAD_INDEX = 1, 2, 4, 8
TREE_NODES = 128             # PA_TREE_NODES
DEFAULT_PARTITION = 512

_DTYPE_CODES = {torch.float16: PA_FP16, torch.bfloat16: PA_BF16}


class PaShape(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_blocks", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class PaError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status}){detail}")


_lock = threading.Lock()
_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpa.so (raises if it is absent: build it with
    ``python -m paged_kv_cache_226_gb300.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"libpa.so not found at {p}; build it with "
                              "`python -m paged_kv_cache_226_gb300.build`")
        lib = ctypes.CDLL(p)
        V, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        S = ctypes.POINTER(PaShape)
        lib.pa_reshape_and_cache.argtypes = [V, V, V, V, V, I64, S, V]
        lib.pa_decode.argtypes = [V, V, V, V, V, F, V, S, V]
        lib.pa_split_workspace_size.argtypes = [S, I32, I32]
        lib.pa_split_workspace_size.restype = ctypes.c_size_t
        lib.pa_decode_split.argtypes = [V, V, V, V, V, F, I32, I32, V, V, V, S, V]
        lib.pa_reduce.argtypes = [V, V, V, V, I32, I32, V, S, V]
        lib.pa_reshape_and_cache_fp8.argtypes = [V, V, V, V, V, I64, F, F, S, V]
        lib.pa_decode_fp8.argtypes = [V, V, V, V, V, F, F, F, V, S, V]
        lib.pa_decode_split_fp8.argtypes = [V, V, V, V, V, F, F, F, I32, I32, V, V, V, S, V]
        lib.pa_decode_step_fp8.argtypes = [V, V, V, V, V, V, V, V, F, F, F, I32, I32, V, V, V, V,
                                           V, S, V]
        for fn in ("pa_reshape_and_cache_fp8", "pa_decode_fp8", "pa_decode_split_fp8",
                   "pa_decode_step_fp8"):
            getattr(lib, fn).restype = ctypes.c_int
        lib.pa_balanced_workspace_size.argtypes = [S]
        lib.pa_balanced_workspace_size.restype = ctypes.c_size_t
        lib.pa_decode_step_balanced.argtypes = [V, V, V, V, V, V, V, V, F, V, ctypes.c_size_t, V,
                                                S, V]
        lib.pa_decode_step_balanced_fp8.argtypes = [V, V, V, V, V, V, V, V, F, F, F, V,
                                                    ctypes.c_size_t, V, S, V]
        lib.pa_decode_step_balanced.restype = ctypes.c_int
        lib.pa_decode_step_balanced_fp8.restype = ctypes.c_int
        lib.pa_copy_async.argtypes = [V, V, ctypes.c_size_t, V]
        lib.pa_copy_async.restype = ctypes.c_int
        for fn in (lib.pa_prefill, lib.pa_prefill_mma):
            fn.argtypes = [V, V, V, V, V, V, F, I32, V, S, V]
            fn.restype = ctypes.c_int
        lib.pa_prefill_workspace_size.argtypes = [S, I32]
        lib.pa_prefill_workspace_size.restype = ctypes.c_size_t
        lib.pa_prefill_ws.argtypes = [V, V, V, V, V, V, F, I32, V, ctypes.c_size_t, V, S, V]
        lib.pa_prefill_ws.restype = ctypes.c_int
        lib.pa_copy_blocks.argtypes = [V, V, I64, V, V, I64, V, I64, S, V]
        lib.pa_copy_blocks.restype = ctypes.c_int
        lib.pa_decode_step.argtypes = [V, V, V, V, V, V, V, V, F, I32, I32, V, V, V, V, V, S, V]
        lib.pa_decode_step.restype = ctypes.c_int
        lib.pa_decode_static_workspace.argtypes = [V, V, V, V, V, F, I32, I32, V, S, V]
        lib.pa_decode_static_workspace.restype = ctypes.c_int
        Z = ctypes.c_size_t
        rope = [V, I64, V, I64, V, I64, V, V, V, I32, I32, F, V, I64, V, V, I64]
        lib.pa_rope_and_cache.argtypes = [*rope, S, V]
        lib.pa_rope_and_cache_fp8.argtypes = [*rope, F, F, S, V]
        lib.pa_decode_weights_workspace_size.argtypes = [S, I32, I32]
        lib.pa_decode_weights.argtypes = [V, V, V, V, V, F, I32, I32, V, V, I64, V, Z, V, S, V]
        lib.pa_decode_weights_fp8.argtypes = [V, V, V, V, V, F, F, F, I32, I32, V, V, I64, V, Z, V,
                                              S, V]
        lib.pa_prefill_weights_workspace_size.argtypes = [S, I32, I32, I32]
        lib.pa_prefill_weights.argtypes = [V, V, V, V, V, F, I64, I32, I32, I32, V, V, I64, V, Z, S,
                                           V]
        lib.pa_evict_workspace_size.argtypes = [S, I32]
        for fn in (lib.pa_evict, lib.pa_evict_fp8):
            fn.argtypes = [V, V, V, V, V, V, V, V, I64, I32, I32, I32, I32, V, V, V, V, Z, S, V]
        norm = [V, I64, V, I64, V, I64, V, V, F, V, I32, V, V, V, I32, I32, F, V, I64, V, V, I64]
        lib.pa_norm_rope_and_cache.argtypes = [*norm, S, V]
        lib.pa_norm_rope_and_cache_fp8.argtypes = [*norm, F, F, S, V]
        lib.pa_tree_attention_workspace_size.argtypes = [S, I32, I32]
        lib.pa_tree_attention.argtypes = [V, V, V, V, V, V, V, F, I64, I32, I32, V, Z, V, S, V]
        lib.pa_tree_attention_fp8.argtypes = [V, V, V, V, V, V, V, F, F, F, I64, I32, I32, V, Z, V,
                                              S, V]
        lib.pa_accept_tree.argtypes = [V, V, V, V, I32, I64, I32, V, V, V, V]
        for fn in (lib.pa_commit_path, lib.pa_commit_path_fp8):
            fn.argtypes = [V, V, I32, V, V, V, V, I32, V, V, S, V]
        for fn in ("pa_decode_weights_workspace_size", "pa_prefill_weights_workspace_size",
                   "pa_evict_workspace_size", "pa_tree_attention_workspace_size"):
            getattr(lib, fn).restype = Z
        lib.pa_status_string.argtypes = [ctypes.c_int]
        lib.pa_status_string.restype = ctypes.c_char_p
        lib.pa_last_cuda_error.argtypes = []
        lib.pa_read_device_errors.argtypes = [ctypes.POINTER(I32), V]
        for fn in ("pa_reshape_and_cache", "pa_decode", "pa_decode_split", "pa_reduce",
                   "pa_last_cuda_error", "pa_read_device_errors"):
            getattr(lib, fn).restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def header_symbols(header: str = HEADER_PATH):
    """Names of the functions include/pa.h declares."""
    with open(header) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(pa_[a-z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != PA_OK:
        detail = ""
        if status == PA_ERR_CUDA:
            detail = f", cudaError {load().pa_last_cuda_error()}"
        raise PaError(fn, status, detail)


def _stream_handle(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype=None, device=None, host_ok: bool = False):
    """Checks a tensor argument; with ``host_ok`` a pinned host tensor is
    accepted too (the kernel reaches it through unified addressing)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    pinned_host = host_ok and not t.is_cuda and t.is_pinned()
    if not t.is_cuda and not pinned_host:
        raise ValueError(f"{name} must be a CUDA tensor" + (" or pinned host memory" if host_ok else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.is_cuda and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def make_shape(num_seqs: int, num_q_heads: int, k_cache: torch.Tensor,
               max_blocks_per_seq: int) -> PaShape:
    nb, bs, hkv, d = k_cache.shape
    if k_cache.dtype not in _DTYPE_CODES:
        raise TypeError(f"cache dtype must be float16 or bfloat16, got {k_cache.dtype}")
    return PaShape(num_seqs=num_seqs, num_q_heads=num_q_heads, num_kv_heads=hkv, head_dim=d,
                   block_size=bs, max_blocks_per_seq=max_blocks_per_seq, num_blocks=nb,
                   dtype=_DTYPE_CODES[k_cache.dtype], reserved=0)


def reshape_and_cache(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                      k_cache: torch.Tensor, v_cache: torch.Tensor) -> None:
    """Write each new token's K/V ([T][Hkv][D]) into slot_mapping's cache slots."""
    lib = load()
    dev = k_cache.device
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, k_cache.dtype, dev)
    for t, n in ((k, "k"), (v, "v")):
        _need(t, n, k_cache.dtype, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    T = slot_mapping.shape[0]
    if k.shape != (T, k_cache.shape[2], k_cache.shape[3]) or v.shape != k.shape:
        raise ValueError("k and v must be [num_tokens][num_kv_heads][head_dim]")
    shp = make_shape(0, k_cache.shape[2], k_cache, 1)
    _check("pa_reshape_and_cache",
           lib.pa_reshape_and_cache(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache),
                                    _ptr(v_cache), T, ctypes.byref(shp), _stream_handle(dev)))


def _decode_common(q, k_cache, v_cache, block_tables, context_lens, host_ok: bool = False):
    dev = k_cache.device
    _need(q, "q", k_cache.dtype, dev, host_ok)
    _need(k_cache, "k_cache", None, dev)
    _need(v_cache, "v_cache", k_cache.dtype, dev)
    _need(block_tables, "block_tables", torch.int32, dev, host_ok)
    _need(context_lens, "context_lens", torch.int32, dev, host_ok)
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [num_blocks][block_size][num_kv_heads][head_dim]")
    B, hq, d = q.shape
    if d != k_cache.shape[3] or block_tables.dim() != 2 or block_tables.shape[0] != B \
            or context_lens.shape != (B,):
        raise ValueError("inconsistent q / block_tables / context_lens shapes")
    return make_shape(B, hq, k_cache, block_tables.shape[1]), dev


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Single-pass paged decode attention (one CTA per sequence and KV head)."""
    lib = load()
    shp, dev = _decode_common(q, k_cache, v_cache, block_tables, context_lens)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype, dev)
    _check("pa_decode", lib.pa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                      _ptr(context_lens), float(scale), _ptr(out),
                                      ctypes.byref(shp), _stream_handle(dev)))
    return out


def num_partitions(max_context_len: int, partition_size: int = DEFAULT_PARTITION) -> int:
    return max(1, -(-int(max_context_len) // int(partition_size)))


def split_workspace(q: torch.Tensor, max_num_partitions: int, device=None
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Allocate (tmp_out, max_logits, exp_sums) for the split path (on
    ``device``, default q's)."""
    B, hq, d = q.shape
    device = q.device if device is None else device
    tmp = torch.empty((B, hq, max_num_partitions, d), dtype=torch.float32, device=device)
    ml = torch.empty((B, hq, max_num_partitions), dtype=torch.float32, device=device)
    es = torch.empty((B, hq, max_num_partitions), dtype=torch.float32, device=device)
    return tmp, ml, es


def workspace_size(num_seqs, num_q_heads, k_cache, max_blocks_per_seq, max_context_len,
                   partition_size=DEFAULT_PARTITION) -> int:
    shp = make_shape(num_seqs, num_q_heads, k_cache, max_blocks_per_seq)
    return int(load().pa_split_workspace_size(ctypes.byref(shp), int(max_context_len),
                                              int(partition_size)))


def decode_split(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                 partition_size: int, max_num_partitions: int, tmp_out=None, max_logits=None,
                 exp_sums=None):
    """Per-partition outputs (tmp_out, max_logits, exp_sums) of the context split."""
    lib = load()
    shp, dev = _decode_common(q, k_cache, v_cache, block_tables, context_lens)
    if tmp_out is None:
        tmp_out, max_logits, exp_sums = split_workspace(q, max_num_partitions)
    for t, n in ((tmp_out, "tmp_out"), (max_logits, "max_logits"), (exp_sums, "exp_sums")):
        _need(t, n, torch.float32, dev)
    B, hq, d = q.shape
    if tmp_out.numel() < B * hq * max_num_partitions * d or \
            max_logits.numel() < B * hq * max_num_partitions or \
            exp_sums.numel() < B * hq * max_num_partitions:
        raise PaError("pa_decode_split", PA_ERR_WORKSPACE)
    _check("pa_decode_split",
           lib.pa_decode_split(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               _ptr(context_lens), float(scale), int(partition_size),
                               int(max_num_partitions), _ptr(tmp_out), _ptr(max_logits),
                               _ptr(exp_sums), ctypes.byref(shp), _stream_handle(dev)))
    return tmp_out, max_logits, exp_sums


def reduce(tmp_out, max_logits, exp_sums, context_lens, partition_size: int,
           k_cache: torch.Tensor, max_blocks_per_seq: int, out: torch.Tensor) -> torch.Tensor:
    """Log-sum-exp merge of decode_split's partitions into out [B][Hq][D]."""
    lib = load()
    dev = out.device
    _need(out, "out", out.dtype, dev)
    for t, n in ((tmp_out, "tmp_out"), (max_logits, "max_logits"), (exp_sums, "exp_sums")):
        _need(t, n, torch.float32, dev)
    _need(context_lens, "context_lens", torch.int32, dev)
    B, hq, d = out.shape
    S = tmp_out.shape[2]
    if k_cache.dtype == torch.uint8:                     # FP8 cache: out keeps its own type
        shp = _fp8_shape(B, hq, k_cache, max_blocks_per_seq, out.dtype)
    else:
        if out.dtype != k_cache.dtype:
            raise TypeError("out must have the cache's dtype")
        shp = make_shape(B, hq, k_cache, max_blocks_per_seq)
    _check("pa_reduce", lib.pa_reduce(_ptr(tmp_out), _ptr(max_logits), _ptr(exp_sums),
                                      _ptr(context_lens), int(partition_size), int(S), _ptr(out),
                                      ctypes.byref(shp), _stream_handle(dev)))
    return out


def paged_attention(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                    max_context_len: int, out: Optional[torch.Tensor] = None,
                    mode: str = "auto", partition_size: int = DEFAULT_PARTITION,
                    workspace=None) -> torch.Tensor:
    """Decode attention through the single-pass or the split + merge path.

    ``mode="auto"`` splits when there are too few (sequence, KV head) pairs to
    fill the GPU evenly or when contexts are long; ``max_context_len`` is the
    host-known bound on ``context_lens`` (it sizes the split grid).
    """
    if out is None:
        out = torch.empty_like(q)
    if mode == "auto":
        mode = choose_mode(q.shape[0], k_cache.shape[2], max_context_len, partition_size,
                           q.device)
    if mode == "single":
        return decode(q, k_cache, v_cache, block_tables, context_lens, scale, out)
    if mode != "split":
        raise ValueError(f"unknown mode {mode!r}")
    S = num_partitions(max_context_len, partition_size)
    if workspace is None:
        workspace = split_workspace(q, S)
    tmp, ml, es = workspace
    decode_split(q, k_cache, v_cache, block_tables, context_lens, scale, partition_size, S,
                 tmp, ml, es)
    return reduce(tmp, ml, es, context_lens, partition_size, k_cache, block_tables.shape[1], out)


def copy_blocks(k_src: torch.Tensor, v_src: torch.Tensor, k_dst: torch.Tensor,
                v_dst: torch.Tensor, block_mapping: torch.Tensor,
                device: Optional[torch.device] = None) -> None:
    """Copy whole blocks ``(src, dst)`` of ``block_mapping`` (int64 [P][2], on
    the device) from the src pools to the dst pools (pa_copy_blocks): the same
    pool for copy-on-write, a pinned host pool on one side for swapping."""
    lib = load()
    dev = device or block_mapping.device
    _need(block_mapping, "block_mapping", torch.int64, dev)
    for t, n in ((k_src, "k_src"), (v_src, "v_src"), (k_dst, "k_dst"), (v_dst, "v_dst")):
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{n} must be a CUDA tensor or pinned host memory")
        if not t.is_contiguous() or t.dtype != k_src.dtype or t.dim() != 4:
            raise ValueError(f"{n} must be a contiguous 4-D pool of {k_src.dtype}")
        if t.shape[1:] != k_src.shape[1:]:
            raise ValueError("pools differ in block shape")
    if v_src.shape != k_src.shape or v_dst.shape != k_dst.shape:
        raise ValueError("K and V pools differ in shape")
    mp = block_mapping.reshape(-1, 2)
    shp = make_shape(0, k_src.shape[2], k_src, 1)
    with torch.cuda.device(dev):
        _check("pa_copy_blocks",
               lib.pa_copy_blocks(_ptr(k_src), _ptr(v_src), k_src.shape[0], _ptr(k_dst),
                                  _ptr(v_dst), k_dst.shape[0], _ptr(mp), mp.shape[0],
                                  ctypes.byref(shp), _stream_handle(dev)))


# ---- FP8 (E4M3) KV cache ---------------------------------------------------
#
# The cache tensors are torch.uint8 [num_blocks][block_size][Hkv][D] holding
# E4M3 codes; element value = e4m3(code) * scale, one scale for K and one for V.
# q, the new tokens and the output keep their fp16 / bf16 type.

def _fp8_shape(num_seqs, num_q_heads, k_cache: torch.Tensor, max_blocks_per_seq, dtype):
    nb, bs, hkv, d = k_cache.shape
    if k_cache.dtype != torch.uint8:
        raise TypeError("an FP8 cache is a torch.uint8 tensor of E4M3 codes")
    return PaShape(num_seqs=num_seqs, num_q_heads=num_q_heads, num_kv_heads=hkv, head_dim=d,
                   block_size=bs, max_blocks_per_seq=max_blocks_per_seq, num_blocks=nb,
                   dtype=_DTYPE_CODES[dtype], reserved=0)


def reshape_and_cache_fp8(k, v, slot_mapping, k_cache, v_cache, k_scale: float,
                          v_scale: float) -> None:
    """Quantise each new token's K/V to E4M3 (x / scale) into its cache slot."""
    lib = load()
    dev = k_cache.device
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.uint8, dev)
    for t, n in ((k, "k"), (v, "v")):
        _need(t, n, k.dtype, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    T = slot_mapping.shape[0]
    if k.shape != (T, k_cache.shape[2], k_cache.shape[3]) or v.shape != k.shape:
        raise ValueError("k and v must be [num_tokens][num_kv_heads][head_dim]")
    shp = _fp8_shape(0, k_cache.shape[2], k_cache, 1, k.dtype)
    _check("pa_reshape_and_cache_fp8",
           lib.pa_reshape_and_cache_fp8(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache),
                                        _ptr(v_cache), T, float(k_scale), float(v_scale),
                                        ctypes.byref(shp), _stream_handle(dev)))


def _fp8_common(q, k_cache, v_cache, block_tables, context_lens, host_ok: bool = False):
    dev = k_cache.device
    _need(q, "q", q.dtype, dev, host_ok)
    _need(k_cache, "k_cache", torch.uint8, dev)
    _need(v_cache, "v_cache", torch.uint8, dev)
    _need(block_tables, "block_tables", torch.int32, dev, host_ok)
    _need(context_lens, "context_lens", torch.int32, dev, host_ok)
    if q.dtype not in _DTYPE_CODES:
        raise TypeError("q must be float16 or bfloat16")
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [num_blocks][block_size][num_kv_heads][head_dim]")
    B, hq, d = q.shape
    if d != k_cache.shape[3] or block_tables.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("inconsistent q / block_tables / context_lens shapes")
    return _fp8_shape(B, hq, k_cache, block_tables.shape[1], q.dtype), dev


def decode_fp8(q, k_cache, v_cache, block_tables, context_lens, scale: float, k_scale: float,
               v_scale: float, out=None) -> torch.Tensor:
    """Single-pass paged decode over an E4M3 cache."""
    lib = load()
    shp, dev = _fp8_common(q, k_cache, v_cache, block_tables, context_lens)
    out = torch.empty_like(q) if out is None else out
    _need(out, "out", q.dtype, dev)
    _check("pa_decode_fp8",
           lib.pa_decode_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                             _ptr(context_lens), float(scale), float(k_scale), float(v_scale),
                             _ptr(out), ctypes.byref(shp), _stream_handle(dev)))
    return out


def decode_split_fp8(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                     k_scale: float, v_scale: float, partition_size: int,
                     max_num_partitions: int, workspace=None):
    """Per-partition outputs over an E4M3 cache (merge them with ``reduce``)."""
    lib = load()
    shp, dev = _fp8_common(q, k_cache, v_cache, block_tables, context_lens)
    tmp, ml, es = workspace if workspace is not None else split_workspace(q, max_num_partitions)
    _check("pa_decode_split_fp8",
           lib.pa_decode_split_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                   _ptr(context_lens), float(scale), float(k_scale),
                                   float(v_scale), int(partition_size), int(max_num_partitions),
                                   _ptr(tmp), _ptr(ml), _ptr(es), ctypes.byref(shp),
                                   _stream_handle(dev)))
    return tmp, ml, es


def decode_step_fp8(q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables,
                    context_lens, scale: float, k_scale: float, v_scale: float,
                    max_context_len: int, out=None, partition_size: int = DEFAULT_PARTITION,
                    workspace=None) -> torch.Tensor:
    """Fused decode layer-step over an E4M3 cache (pa_decode_step_fp8)."""
    lib = load()
    shp, dev = _fp8_common(q, k_cache, v_cache, block_tables, context_lens)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, n, q.dtype, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    out = torch.empty_like(q) if out is None else out
    S = num_partitions(max_context_len, partition_size)
    if workspace is None:
        workspace = step_workspace(q, k_cache.shape[2], S)
    tmp, ml, es, counters = workspace
    _check("pa_decode_step_fp8",
           lib.pa_decode_step_fp8(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                                  _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                  _ptr(context_lens), float(scale), float(k_scale),
                                  float(v_scale), int(partition_size), int(S), _ptr(tmp),
                                  _ptr(ml), _ptr(es), _ptr(counters), _ptr(out),
                                  ctypes.byref(shp), _stream_handle(dev)))
    return out


def step_workspace(q: torch.Tensor, num_kv_heads: int, max_num_partitions: int, device=None):
    """(tmp_out, max_logits, exp_sums, counters) for ``decode_step`` (on
    ``device``, default q's); the counters start at zero and every step leaves
    them at zero."""
    device = q.device if device is None else device
    tmp, ml, es = split_workspace(q, max_num_partitions, device)
    counters = torch.zeros((q.shape[0], num_kv_heads), dtype=torch.int32, device=device)
    return tmp, ml, es, counters


def decode_step(q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables, context_lens,
                scale: float, max_context_len: int, out: Optional[torch.Tensor] = None,
                partition_size: int = DEFAULT_PARTITION, workspace=None) -> torch.Tensor:
    """One fused decode layer-step (pa_decode_step): write each sequence's new
    token into the cache and attend, merging partitions in the same launch."""
    lib = load()
    shp, dev = _decode_common(q, k_cache, v_cache, block_tables, context_lens)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, n, k_cache.dtype, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    if k_new.shape != (q.shape[0], k_cache.shape[2], k_cache.shape[3]) or \
            v_new.shape != k_new.shape or slot_mapping.shape != (q.shape[0],):
        raise ValueError("k_new / v_new must be [num_seqs][num_kv_heads][head_dim], "
                         "slot_mapping [num_seqs]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype, dev)
    S = num_partitions(max_context_len, partition_size)
    if workspace is None:
        workspace = step_workspace(q, k_cache.shape[2], S)
    tmp, ml, es, counters = workspace
    _need(counters, "counters", torch.int32, dev)
    _check("pa_decode_step",
           lib.pa_decode_step(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                              _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                              _ptr(context_lens), float(scale), int(partition_size), int(S),
                              _ptr(tmp), _ptr(ml), _ptr(es), _ptr(counters), _ptr(out),
                              ctypes.byref(shp), _stream_handle(dev)))
    return out


def balanced_workspace(q: torch.Tensor, k_cache: torch.Tensor,
                       block_tables: torch.Tensor) -> torch.Tensor:
    """Zeroed workspace for ``decode_step_balanced`` (reusable across steps)."""
    if k_cache.dtype == torch.uint8:
        shp = _fp8_shape(q.shape[0], q.shape[1], k_cache, block_tables.shape[1], q.dtype)
    else:
        shp = make_shape(q.shape[0], q.shape[1], k_cache, block_tables.shape[1])
    with torch.cuda.device(q.device):
        n = int(load().pa_balanced_workspace_size(ctypes.byref(shp)))
    if n == 0:
        raise PaError("pa_balanced_workspace_size", PA_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device=q.device)


def decode_step_balanced(q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables,
                         context_lens, scale: float, out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, k_scale: float = None,
                         v_scale: float = None) -> torch.Tensor:
    """Fused decode layer-step with the work balanced over one wave of CTAs
    (pa_decode_step_balanced; pa_decode_step_balanced_fp8 for a uint8 E4M3
    cache with k_scale / v_scale)."""
    lib = load()
    fp8 = k_cache.dtype == torch.uint8
    if fp8:
        shp, dev = _fp8_common(q, k_cache, v_cache, block_tables, context_lens)
    else:
        shp, dev = _decode_common(q, k_cache, v_cache, block_tables, context_lens)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, n, q.dtype, dev)
    _need(slot_mapping, "slot_mapping", torch.int64, dev)
    if k_new.shape != (q.shape[0], k_cache.shape[2], k_cache.shape[3]) or \
            v_new.shape != k_new.shape or slot_mapping.shape != (q.shape[0],):
        raise ValueError("k_new / v_new must be [num_seqs][num_kv_heads][head_dim], "
                         "slot_mapping [num_seqs]")
    out = torch.empty_like(q) if out is None else out
    _need(out, "out", q.dtype, dev)
    if workspace is None:
        workspace = balanced_workspace(q, k_cache, block_tables)
    _need(workspace, "workspace", torch.uint8, dev)
    args = [_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
            _ptr(block_tables), _ptr(context_lens), ctypes.c_float(scale)]
    if fp8:
        args += [ctypes.c_float(k_scale), ctypes.c_float(v_scale)]
    args += [_ptr(workspace), ctypes.c_size_t(workspace.numel()), _ptr(out), ctypes.byref(shp),
             _stream_handle(dev)]
    fn = lib.pa_decode_step_balanced_fp8 if fp8 else lib.pa_decode_step_balanced
    _check("pa_decode_step_balanced" + ("_fp8" if fp8 else ""), fn(*args))
    return out


def prefill(q, k_cache, v_cache, block_tables, context_lens, query_start, scale: float,
            max_query_len: int, out: Optional[torch.Tensor] = None,
            kernel: str = "auto", schedule: bool = True,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Chunked-prefill attention (pa_prefill): the last C_b tokens of each
    sequence attend causally over its cache; q, out [total_tokens][Hq][D].
    kernel "mma" forces the mma.sync kernel (pa_prefill_mma).  schedule: order
    the tcgen05 kernel's work longest first (pa_prefill_ws, with ``workspace``
    or a fresh one of pa_prefill_workspace_size bytes); False: pa_prefill."""
    lib = load()
    dev = k_cache.device
    _need(q, "q", k_cache.dtype, dev)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, k_cache.dtype, dev)
    _need(block_tables, "block_tables", torch.int32, dev)
    _need(context_lens, "context_lens", torch.int32, dev)
    _need(query_start, "query_start", torch.int32, dev)
    B = context_lens.shape[0]
    if query_start.shape != (B + 1,) or block_tables.shape[0] != B or q.dim() != 3:
        raise ValueError("query_start must be [num_seqs + 1], q [total_tokens][Hq][D]")
    out = torch.empty_like(q) if out is None else out
    _need(out, "out", q.dtype, dev)
    shp = make_shape(B, q.shape[1], k_cache, block_tables.shape[1])
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
            _ptr(query_start), float(scale), int(max_query_len))
    if kernel == "mma" or not schedule:
        fn = lib.pa_prefill_mma if kernel == "mma" else lib.pa_prefill
        _check("pa_prefill", fn(*args, _ptr(out), ctypes.byref(shp), _stream_handle(dev)))
        return out
    if workspace is None:
        n = prefill_workspace_size(shp, max_query_len)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    _check("pa_prefill_ws", lib.pa_prefill_ws(*args, _ptr(workspace), workspace.numel(), _ptr(out),
                                              ctypes.byref(shp), _stream_handle(dev)))
    return out


def prefill_workspace_size(shp, max_query_len: int) -> int:
    """Bytes of the work-ordering workspace pa_prefill_ws needs (0: none)."""
    return int(load().pa_prefill_workspace_size(ctypes.byref(shp), int(max_query_len)))


# ---- a cache within a budget of tokens --------------------------------------
#
# State of a batch: weights (fp32) and positions (int32), [B][Hkv][W] with W at
# least the tokens a block table holds; entry i belongs to cache index i.

def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original_len: int = 0, slow: float = 1.0,
                     fast: float = 32.0, device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq, factor) for ``rope_and_cache``: inv_freq[i] = base^(-2i/R),
    stretched for contexts ``factor`` times the ``original_len`` trained on.

    scaling: ``"none"``; ``"linear"`` (every angle divided by factor);
    ``"ntk"`` (the base raised so that the slowest angle is divided by factor
    and the fastest stays); ``"bands"`` (pairs that turn fewer than ``slow``
    times over original_len are divided by factor, those that turn more than
    ``fast`` times stay, a linear ramp in turns between); ``"yarn"`` (the
    ramp linear in the pair's index, and cos / sin scaled by
    0.1 ln(factor) + 1)."""
    if rotary_dim <= 0 or rotary_dim % 2 or base <= 0:
        raise ValueError("rotary_dim must be even and positive, base positive")
    if factor < 1.0:
        raise ValueError("factor must be at least 1")
    half = rotary_dim // 2
    i = torch.arange(half, dtype=torch.float64)
    mult = 1.0
    if scaling == "ntk" and half > 1:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    inv = float(base) ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        inv = inv / factor
    elif scaling in ("bands", "yarn"):
        if original_len <= 0 or not 0 < slow < fast:
            raise ValueError("bands and yarn need original_len > 0 and 0 < slow < fast")
        turns = original_len * inv / (2 * np.pi)
        if scaling == "bands":
            keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        else:
            def pair_of(n):             # the pair that turns n times over original_len
                return rotary_dim * np.log(original_len / (n * 2 * np.pi)) / (2 * np.log(base))
            lo = max(np.floor(pair_of(fast)), 0.0)
            hi = min(np.ceil(pair_of(slow)), rotary_dim - 1.0)
            keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
            mult = 0.1 * float(np.log(factor)) + 1.0
        inv = inv * keep + inv / factor * (1.0 - keep)
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return inv.to(torch.float32).to(device or "cpu"), mult


_native = None
_bound = object()        # the library that _native calls


def _load_native():
    """The binding of the bounded-cache and tree calls (csrc/binding.cpp), set to call
    the loaded library: their checks and allocations in native code, since a
    layer makes three of them per step."""
    global _native, _bound
    lib = load()
    try:
        from . import _native as native
    except ImportError as e:
        raise ImportError(f"_native.so cannot be loaded ({e}); build it with "
                          "`python -m paged_kv_cache_226_gb300.build`") from e
    native.bind(lib._handle)
    _native, _bound = native, lib
    return native


def _refused(name: str, k_cache: torch.Tensor, status: int) -> None:
    _check(name + "_fp8" if k_cache.dtype is torch.uint8 else name, status)


def _must(t: torch.Tensor, name: str, dtype, device: torch.device, index: int) -> None:
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index
            and t.is_contiguous()):
        _need(t, name, dtype, device)
        raise ValueError(f"{name} must be contiguous, {dtype}, on {device}")


def _state(t: torch.Tensor, name: str, shape, dtype, device, index: int) -> None:
    """A [B][Hkv][W] state tensor; ``shape``: (B, Hkv, at least W)."""
    _must(t, name, dtype, device, index)
    got = t.shape
    if len(got) != 3 or got[0] != shape[0] or got[1] != shape[1] or got[2] < shape[2]:
        raise ValueError(f"{name} must be [{shape[0]}][{shape[1]}][>= {shape[2]}]")


def _weights_pair(weights, weights_out, shape, device, index: int) -> torch.Tensor:
    """weights_out, by default weights themselves or fresh zeros; both checked."""
    if weights_out is None:
        weights_out = weights if weights is not None else \
            torch.zeros(shape, dtype=torch.float32, device=device)
    _state(weights_out, "weights_out", shape, torch.float32, device, index)
    if weights is not None and weights is not weights_out:
        _state(weights, "weights", shape, torch.float32, device, index)
        if weights.shape != weights_out.shape:
            raise ValueError("weights and weights_out must have the same shape")
    return weights_out


def _workspace(workspace: Optional[torch.Tensor], nbytes: int, fn: str, device):
    """(tensor, bytes) of a workspace of at least nbytes."""
    if nbytes == 0:
        raise PaError(fn, PA_ERR_INVALID_ARG)
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes
    _need(workspace, "workspace", None, device)
    return workspace, workspace.numel() * workspace.element_size()


def rope_and_cache(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                   positions: torch.Tensor, slot_mapping: torch.Tensor, inv_freq: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor,
                   q_out: Optional[torch.Tensor] = None, interleaved: bool = False,
                   factor: float = 1.0, k_scale: Optional[float] = None,
                   v_scale: Optional[float] = None) -> Optional[torch.Tensor]:
    """Rotary positions on the new tokens' q and k, and the cache write of k
    and v (pa_rope_and_cache, or its E4M3 form for a uint8 cache); returns the
    turned q.

    q, k, v: [T][heads][D], a token's heads contiguous (slices of one
    projection's output will do); ``q=None`` writes the cache only.
    positions, slot_mapping: int64 [T]; inv_freq: fp32 [R/2], the first R dims
    of a head turn (``rope_frequencies``).  ``q_out=q`` turns q in place."""
    r = (_native if _bound is _lib else _load_native()).rope_and_cache(
        q, k, v, positions, slot_mapping, inv_freq, k_cache, v_cache, q_out, interleaved, factor,
        k_scale, v_scale)
    if r.__class__ is int:
        _refused("pa_rope_and_cache", k_cache, r)
    return r


@functools.lru_cache(maxsize=1024)
def weights_partition(num_seqs: int, num_kv_heads: int, max_context_len: int, fp8: bool,
                      index: int) -> int:
    """Partition size of ``decode_weights`` on device ``index``.

    A CTA costs its start and its record, and an SM holds 6 at a time.  Where
    a slot's share of the batch's tokens (every context taken at
    ``max_context_len``) is at most 1024, the contexts are cut into as many
    even pieces as the slots hold at once, but not below 1.5
    sqrt(max_context_len) tokens, 4 where all slots are in use: there the
    merge of the records takes over.  That is for three pieces or more, since
    lengths differ, else a piece is the next power of two to the share.  Above
    1024 the grid's waves count: as many pieces as 5.2 CTAs per SM allow if
    those are three or more, at most 1536 tokens over an E4M3 cache; else
    1024, or about 2.75 waves where that would start a second wave that stays
    almost empty.  Measured (us, this rule's size against others): 8 pairs of
    4096 tokens 8.7 at 128 (512: 13.1); 8 of 50,000 44.8 at 512 (1024: 45.2);
    32 of 4000 11.5 at 256 (160: 12.6); 128 of up to 1000 11.3 at 160 (256:
    12.4, 512: 15.4); 256 of 2048 51.1 at 704 (1024: 52.7); 512 of 2048 97.5
    at 416 (1024: 111.6); 320 of up to 4096 64.4 at 1024 (2048: 77.1); E4M3:
    64 of up to 8000 29.0 at 576 (1024: 40.3), 256 of 4096 70.0 at 1408
    (1024: 79.7)."""
    sms = torch.cuda.get_device_properties(index).multi_processor_count
    pairs, slots = max(1, num_seqs * num_kv_heads), sms * CTAS_PER_SM
    share = pairs * max_context_len / slots
    if share > 1024:
        pieces = (26 * sms) // (5 * pairs)
        if pieces >= 3:
            size = 128 * -(-max_context_len // (128 * pieces))
            return min(size, 1536) if fp8 else size
        waves = pairs * -(-max_context_len // 1024) / slots
        if 1 < waves < 1.3:
            pieces = -(-11 * slots // (4 * pairs))
            return 32 * -(-max_context_len // (32 * pieces))
        return 1024
    size = 64
    while size * size < 2.25 * max_context_len:
        size *= 2
    pieces = slots // pairs
    if pieces >= 3:
        even = 32 * -(-max_context_len // (32 * pieces))
        if even <= size:
            return size
        return min(1024, max(even, 64 * math.ceil(max_context_len ** 0.5 / 16)))
    while size < share:
        size *= 2
    return min(size, 1024)


def decode_weights(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                   max_context_len: int, weights: Optional[torch.Tensor] = None,
                   weights_out: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, partition_size: Optional[int] = None,
                   workspace: Optional[torch.Tensor] = None, k_scale: Optional[float] = None,
                   v_scale: Optional[float] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Decode attention that adds each cached token's attention weight to
    ``weights`` [B][Hkv][W] (pa_decode_weights, or its E4M3 form for a uint8
    cache); returns (out, weights_out).  The newest token's entry is set, not
    added to; ``weights=None`` starts at zero.  ``weights_out`` defaults to
    ``weights`` (in place), or a new tensor of zeros."""
    r = (_native if _bound is _lib else _load_native()).decode_weights(
        q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, weights,
        weights_out, out, weights_partition if partition_size is None else partition_size,
        workspace, k_scale, v_scale)
    if r.__class__ is int:
        _refused("pa_decode_weights", k_cache, r)
    return r


def prefill_weights(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
                    context_lens: torch.Tensor, query_start: torch.Tensor, scale: float,
                    max_query_len: int, max_context_len: int, window: int = 0,
                    weights: Optional[torch.Tensor] = None,
                    weights_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention weights that a chunk's queries (all, or the last ``window``)
    give to the cached tokens, added to ``weights`` [B][Hkv][W]
    (pa_prefill_weights; ``prefill`` gives the attention itself).  The chunk's
    own tokens are set, not added to.  ``weights_out`` defaults to ``weights``
    (in place), or a new tensor of zeros; returned."""
    r = (_native if _bound is _lib else _load_native()).prefill_weights(
        q, k_cache, block_tables, context_lens, query_start, scale, max_query_len,
        max_context_len, window, weights, weights_out, workspace)
    if r.__class__ is int:
        _refused("pa_prefill_weights", k_cache, r)
    return r


def evict(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
          context_lens: torch.Tensor, seen_lens: torch.Tensor, budget: int,
          weights: torch.Tensor, positions: torch.Tensor,
          known_lens: Optional[torch.Tensor] = None, trigger: Optional[int] = None,
          sinks: int = 0, recent: int = 0, weights_out: Optional[torch.Tensor] = None,
          positions_out: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
          workspace: Optional[torch.Tensor] = None
          ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Cut every sequence of more than ``trigger`` (default: budget) tokens to
    ``budget`` per KV head: the first ``sinks`` positions, the ``recent``
    newest and the largest weights stay, and the gaps are closed in the caches
    (pa_evict; pa_evict_fp8 for a uint8 cache).  Returns (new_lens, weights,
    positions); the state tensors are updated in place unless ``weights_out``
    / ``positions_out`` are given.  seen_lens: int32 [B], tokens the sequence
    has had in all; known_lens: int32 [B], the new_lens of the previous call
    (entries of ``positions`` that are set; None: none).  Blocks past
    ceil(new_len / block_size) are free afterwards
    (``PagedKVAllocator.truncate``)."""
    r = (_native if _bound is _lib else _load_native()).evict(
        k_cache, v_cache, block_tables, context_lens, seen_lens, budget, weights, positions,
        known_lens, trigger, sinks, recent, weights_out, positions_out, new_lens, workspace)
    if r.__class__ is int:
        _refused("pa_evict", k_cache, r)
    return (r, weights if weights_out is None else weights_out,
            positions if positions_out is None else positions_out)


# ---- speculative decoding: a tree of drafted tokens per sequence --------------
#
# Node i of sequence b is row query_start[b] + i of the batch and the cached
# token L_b - C_b + i; parents name a node's predecessor within its tree.

def norm_rope_and_cache(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                        positions: torch.Tensor, slot_mapping: torch.Tensor,
                        inv_freq: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        axes: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                        interleaved: bool = False, factor: float = 1.0,
                        k_scale: Optional[float] = None,
                        v_scale: Optional[float] = None) -> Optional[torch.Tensor]:
    """``rope_and_cache`` behind a norm of every head of q and k
    (pa_norm_rope_and_cache, or its E4M3 form for a uint8 cache): x becomes
    weight * x / sqrt(mean(x^2) + eps), then turns; returns the turned q.

    q_weight, k_weight: [D] of q's dtype (None: ones).  positions: int64 [T], or
    [A][T] with ``axes``, int32 [R/2]: the axis whose positions turn pair i
    (time, height and width of an image's patches, for instance)."""
    r = (_native if _bound is _lib else _load_native()).norm_rope_and_cache(
        q, k, v, positions, slot_mapping, inv_freq, k_cache, v_cache, q_weight, k_weight, eps, axes,
        q_out, interleaved, factor, k_scale, v_scale)
    if r.__class__ is int:
        _refused("pa_norm_rope_and_cache", k_cache, r)
    return r


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_tables: torch.Tensor, context_lens: torch.Tensor,
                   query_start: torch.Tensor, parents: Optional[torch.Tensor], scale: float,
                   max_query_len: int, max_context_len: int, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, k_scale: Optional[float] = None,
                   v_scale: Optional[float] = None) -> torch.Tensor:
    """Attention of trees of drafted tokens over the cache, which holds their
    keys and values (pa_tree_attention, or its E4M3 form for a uint8 cache):
    each node sees the context, its ancestors and itself.

    q, out: [total_tokens][Hq][D]; query_start: int32 [B + 1]; parents: int32
    [total_tokens], the node of the same tree that a node follows (below its
    own index; negative: the context), None: every tree is a line.  Trees have
    at most 128 nodes; context_lens counts them."""
    r = (_native if _bound is _lib else _load_native()).tree_attention(
        q, k_cache, v_cache, block_tables, context_lens, query_start, parents, scale, max_query_len,
        max_context_len, out, workspace, k_scale, v_scale)
    if r.__class__ is int:
        _refused("pa_tree_attention", k_cache, r)
    return r


def accept_tree(draft_tokens: torch.Tensor, target_tokens: torch.Tensor,
                parents: Optional[torch.Tensor], query_start: torch.Tensor, max_query_len: int
                ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The longest path of drafted tokens that the model agrees with
    (pa_accept_tree): (path, path_lens, next_tokens).

    draft_tokens: int64 [total_tokens], each node's token (node 0: the newest
    one, always kept); target_tokens: int64 [total_tokens], what the model gives
    after each node; parents, query_start: as for ``tree_attention``.  path:
    int32 [B][max_query_len], node indexes from node 0 on, -1 behind them;
    next_tokens: int64 [B], the model's token after the path's end."""
    r = (_native if _bound is _lib else _load_native()).accept_tree(
        draft_tokens, target_tokens, parents, query_start, max_query_len)
    if r.__class__ is int:
        _check("pa_accept_tree", r)
    return r


def commit_path(k_caches, v_caches, block_tables: torch.Tensor, context_lens: torch.Tensor,
                query_start: torch.Tensor, path: torch.Tensor, path_lens: torch.Tensor,
                new_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Keep of each tree the path's nodes: their rows close up behind the
    context in the caches of all layers (pa_commit_path; pa_commit_path_fp8 for
    uint8 caches), in place; returns the new context lengths, int32 [B].

    k_caches, v_caches: a cache each, or sequences of one per layer; path,
    path_lens: as ``accept_tree`` gives them.  Blocks past ceil(new_len /
    block_size) are free afterwards (``PagedKVAllocator.truncate``)."""
    if not isinstance(k_caches, torch.Tensor):
        k_caches = tuple(k_caches)
    if not isinstance(v_caches, torch.Tensor):
        v_caches = tuple(v_caches)
    r = (_native if _bound is _lib else _load_native()).commit_path(
        k_caches, v_caches, block_tables, context_lens, query_start, path, path_lens, new_lens)
    if r.__class__ is int:
        _refused("pa_commit_path", k_caches if isinstance(k_caches, torch.Tensor) else k_caches[0], r)
    return r


STATIC_WORKSPACE_BYTES = 32 << 20


def decode_static_workspace(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                            max_context_len: int, out: Optional[torch.Tensor] = None,
                            partition_size: int = DEFAULT_PARTITION) -> torch.Tensor:
    """Split decode + merge using the library's own fixed device buffer for
    the partition workspace (pa_decode_static_workspace): for callers that
    must not allocate device memory, e.g. inside a framework that owns the
    device memory pool.  ``out`` must be given by such callers (allocating it
    here is a convenience for tests).  Calls that overlap on the GPU share
    the buffer and race; keep them ordered."""
    lib = load()
    shp, dev = _decode_common(q, k_cache, v_cache, block_tables, context_lens)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", q.dtype, dev)
    S = num_partitions(max_context_len, partition_size)
    _check("pa_decode_static_workspace",
           lib.pa_decode_static_workspace(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(block_tables), _ptr(context_lens), float(scale),
                                          int(partition_size), int(S), _ptr(out),
                                          ctypes.byref(shp), _stream_handle(dev)))
    return out


CTAS_PER_SM = 6          # resident decode CTAs per SM in the shipped build


def choose_partition(num_seqs: int, num_kv_heads: int, max_context_len: int,
                     block_size: int = 16, device=None, context_lens=None) -> int:
    """Partition size for the split / fused paths.

    With at least half as many (sequence, KV head) pairs as resident CTA
    slots, the pairs alone give every slot work: 1024-token partitions then
    leave most contexts of a ragged batch in one partition (no merge) and
    the rest in few (measured on the fused step: shared-prefix batch 119 us
    against 133 us at 512 tokens, Llama-3-8B-shaped batch 60 us against 62).

    Fewer pairs (long contexts, small batches): the smallest multiple of 512
    that cuts the batch into at most 4.8 CTAs per SM, counting every
    context's ragged last piece (``context_lens``, host values; without them
    every context is taken at ``max_context_len``).  Fewer CTAs pay the
    per-partition start and merge fewer times, but below ~3 per SM too few
    stages are in flight to keep HBM busy; more than one wave of CTAs
    leaves a tail of late, long partitions.  Measured on the fused step
    (µs per layer-step, best partition, this rule's choice): 256 pairs of
    4096 tokens 91.8 at 2048 (2048; 1536 gives 94.3); 64 pairs of
    U[32768, 50000] 217.2 at 4352 (4096: 220.1; 3584 gives 230.3);
    32 x U[128, 4096] x 8 heads 54.9 at 1024 (1024; 2048 gives 67.4);
    40 x 4096 x 8 heads 108.3 at 2048 (2048; 1536 gives 115.5)."""
    if device is None and torch.cuda.is_available():
        device = torch.cuda.current_device()
    sms = torch.cuda.get_device_properties(device).multi_processor_count if device is not None \
        else 152
    slots = sms * CTAS_PER_SM
    pairs = max(1, num_seqs * num_kv_heads)
    if max_context_len <= 512:
        p = 512
    elif 2 * pairs >= slots:
        p = 1024
    else:
        if context_lens is None:
            lens = np.full(max(1, num_seqs), max_context_len, dtype=np.int64)
        else:
            if isinstance(context_lens, torch.Tensor):
                context_lens = context_lens.detach().cpu().numpy()
            lens = np.asarray(context_lens, dtype=np.int64).reshape(-1)
        limit = (24 * sms) // 5                        # 4.8 CTAs per SM

        def ctas(units: int) -> int:                   # CTAs at 512 * units tokens
            return num_kv_heads * int(np.sum(-(-lens // (512 * units))))

        # The count falls as the partition grows; one partition per context
        # (pairs < slots / 2 <= limit CTAs) always fits.
        lo, hi = 1, max(1, -(-max_context_len // 512))
        while lo < hi:
            mid = (lo + hi) // 2
            if ctas(mid) <= limit:
                hi = mid
            else:
                lo = mid + 1
        p = 512 * lo
    return max(block_size, p - p % block_size)


def choose_mode(num_seqs: int, num_kv_heads: int, max_context_len: int, partition_size: int,
                device=None) -> str:
    """Single pass when every (sequence, KV head) CTA is short, else split."""
    if max_context_len <= partition_size:
        return "single"
    return "split"


def read_device_errors(device: Optional[torch.device] = None) -> int:
    """Return and clear the library's device error word (PA_DEVERR_* bits)."""
    lib = load()
    dev = device or torch.device("cuda", torch.cuda.current_device())
    flags = ctypes.c_int32(0)
    with torch.cuda.device(dev):
        _check("pa_read_device_errors",
               lib.pa_read_device_errors(ctypes.byref(flags), _stream_handle(dev)))
    return int(flags.value)


def copy_async(dst: torch.Tensor, src: torch.Tensor) -> torch.Tensor:
    """dst <- src by a short kernel (pa_copy_async) on the current stream of
    whichever side is on the device; either may be pinned host memory."""
    if dst.numel() * dst.element_size() != src.numel() * src.element_size():
        raise ValueError("copy_async needs equal byte sizes")
    if not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("copy_async needs contiguous tensors")
    for t in (dst, src):
        if not t.is_cuda and not t.is_pinned():
            raise ValueError("copy_async: host tensors must be pinned")
    dev = dst.device if dst.is_cuda else src.device
    if not dev.type == "cuda":
        raise ValueError("copy_async: one side must be on a CUDA device")
    _check("pa_copy_async", load().pa_copy_async(_ptr(dst), _ptr(src),
                                                 ctypes.c_size_t(dst.numel() * dst.element_size()),
                                                 _stream_handle(dev)))
    return dst


class InputStaging:
    """A layer-step's host inputs (q, new K/V, slots, tables, lengths) as views
    into one pinned host buffer and one device buffer, each view 256-byte
    aligned, so a step uploads all of them with a single host-to-device copy.

    ``specs`` maps names to (shape, dtype); ``h[name]`` / ``d[name]`` are the
    host and device views.  Fill the host views, call ``upload()`` (on the
    current stream), and hand the device views to the kernels.
    """

    def __init__(self, specs: dict, device: torch.device):
        offsets, total = {}, 0
        for name, (shape, dtype) in specs.items():
            nbytes = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
            offsets[name] = (total, nbytes, tuple(shape), dtype)
            total += (nbytes + 255) // 256 * 256
        self.nbytes = total
        self.host = torch.empty(total, dtype=torch.uint8).pin_memory()
        self.dev = torch.empty(total, dtype=torch.uint8, device=device)
        self.h, self.d = {}, {}
        for name, (off, nbytes, shape, dtype) in offsets.items():
            self.h[name] = self.host[off:off + nbytes].view(dtype).view(shape)
            self.d[name] = self.dev[off:off + nbytes].view(dtype).view(shape)

    def upload(self, engine: str = "kernel") -> None:
        """All inputs host -> device in one asynchronous copy on the current
        stream: by a short kernel reading the pinned buffer (``"kernel"``,
        pa_copy_async) or by the copy engine (``"dma"``)."""
        if engine == "kernel":
            copy_async(self.dev, self.host)
        else:
            self.dev.copy_(self.host, non_blocking=True)


class StepPlan:
    """One decode layer-step with its arguments marshalled once.

    Holds the C-ABI argument lists of the step for fixed tensors, so that each
    launch costs one ctypes call. Modes: ``"fused"`` (the default: one
    pa_decode_step launch), ``"split"`` (reshape_and_cache, decode_split,
    reduce), ``"single"`` (reshape_and_cache, decode) and ``"weights"``
    (reshape_and_cache, decode_weights: each step adds the attention weights
    into ``weights``, or reads them there and writes ``weights_out``; with
    ``k_new``, ``v_new`` and ``slot_mapping`` None the step is decode_weights
    alone, for keys that ``rope_and_cache`` has turned and cached: the plan's
    own cache write would put the unturned ones over them). The work goes to
    the caller's current stream at call time, which also makes a step
    capturable into a CUDA graph (``capture_graph``). The tensors must stay
    alive and keep their shapes; their contents (new tokens, tables, lengths)
    may change between steps as long as ``context_lens`` stays within
    ``max_context_len``.

    In the fused mode q, k_new, v_new, slot_mapping, block_tables,
    context_lens and out may be pinned host tensors: the kernel reads the
    inputs and writes the output over the host link through unified
    addressing, with no copy launch (on a Grace-Blackwell node the fastest
    way to move a step's inputs in and its output out).  The caches and the
    workspace stay in device memory.

    ``partition_size=None`` takes ``choose_partition`` for the batch: with
    the lengths counted when ``context_lens`` is in host memory, else every
    context taken at ``max_context_len`` (no device read).  Any multiple of
    the block size gives the same result; the size only sets the speed.
    """

    def __init__(self, q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables,
                 context_lens, scale: float, max_context_len: int, out=None,
                 mode: str = "auto", partition_size: Optional[int] = None, workspace=None,
                 k_scale: Optional[float] = None, v_scale: Optional[float] = None,
                 weights: Optional[torch.Tensor] = None,
                 weights_out: Optional[torch.Tensor] = None):
        self._lib = load()
        self.fp8 = k_cache.dtype == torch.uint8
        if mode == "auto":
            mode = "fused"
        if mode not in ("single", "split", "fused", "balanced", "weights"):
            raise ValueError(f"unknown mode {mode!r}")
        if (weights is None) == (mode == "weights") or (weights_out is not None and weights is None):
            raise ValueError("weights belong to mode \"weights\", which needs them")
        host_ok = mode == "fused"            # pinned host inputs / output allowed
        if self.fp8:
            if k_scale is None or v_scale is None:
                raise ValueError("an FP8 cache needs k_scale and v_scale")
            if mode not in ("fused", "balanced", "weights"):
                raise ValueError("StepPlan runs an FP8 cache through the fused steps and "
                                 "decode_weights only")
            shp, dev = _fp8_common(q, k_cache, v_cache, block_tables, context_lens, host_ok)
        else:
            shp, dev = _decode_common(q, k_cache, v_cache, block_tables, context_lens, host_ok)
        cached = k_new is None and v_new is None and slot_mapping is None
        if cached and mode != "weights":
            raise ValueError("k_new, v_new and slot_mapping may be None in mode \"weights\" only")
        if not cached:
            for t, n in ((k_new, "k_new"), (v_new, "v_new")):
                _need(t, n, q.dtype, dev, host_ok)
            _need(slot_mapping, "slot_mapping", torch.int64, dev, host_ok)
        T = q.shape[0] if cached else slot_mapping.shape[0]
        if not cached and (k_new.shape != (T, k_cache.shape[2], k_cache.shape[3]) or
                           v_new.shape != k_new.shape):
            raise ValueError("k_new and v_new must be [num_tokens][num_kv_heads][head_dim]")
        self.device = dev
        self.out = torch.empty(q.shape, dtype=q.dtype, device=dev) if out is None else out
        _need(self.out, "out", q.dtype, dev, host_ok)
        if mode in ("fused", "balanced", "weights") and T != q.shape[0]:
            raise ValueError("the step takes exactly one new token per sequence")
        self.mode = mode
        if partition_size is None and mode == "weights":
            partition_size = weights_partition(q.shape[0], k_cache.shape[2], int(max_context_len),
                                               self.fp8, dev.index)
        elif partition_size is None:
            partition_size = choose_partition(
                q.shape[0], k_cache.shape[2], max_context_len, k_cache.shape[1], dev,
                context_lens if context_lens.device.type == "cpu" else None)
        self.partition_size = int(partition_size)
        self.num_partitions = num_partitions(max_context_len, partition_size)
        self._shape = shp
        self._keep = [q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables,
                      context_lens, self.out]
        sref = ctypes.byref(self._shape)
        self._reshape_args = (_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache),
                              _ptr(v_cache), ctypes.c_int64(T), sref)
        if mode == "weights":
            B, hkv, tokens = q.shape[0], k_cache.shape[2], block_tables.shape[1] * k_cache.shape[1]
            weights_out = _weights_pair(weights, weights_out, (B, hkv, tokens), dev, dev.index)
            self.weights_out = weights_out
            scales = (ctypes.c_float(k_scale), ctypes.c_float(v_scale)) if self.fp8 else ()
            if self.fp8:
                self._reshape_args = (*self._reshape_args[:-1], *scales, sref)
            if cached:
                self._reshape_args = None
            workspace, nbytes = _workspace(workspace, self._lib.pa_decode_weights_workspace_size(
                sref, int(max_context_len), self.partition_size) if B else 1, "pa_decode_weights", dev)
            self.workspace = workspace
            self._keep += [workspace, weights, weights_out]
            self._decode_args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                 _ptr(context_lens), ctypes.c_float(scale), *scales,
                                 ctypes.c_int32(int(max_context_len)),
                                 ctypes.c_int32(self.partition_size), _ptr(weights),
                                 _ptr(weights_out), ctypes.c_int64(weights_out.shape[2]),
                                 _ptr(workspace), ctypes.c_size_t(nbytes), _ptr(self.out), sref)
            self._weights_out_at = len(self._decode_args) - 6
        elif mode == "single":
            self._decode_args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                 _ptr(context_lens), ctypes.c_float(scale), _ptr(self.out), sref)
        elif mode == "balanced":
            if workspace is None:
                workspace = balanced_workspace(q, k_cache, block_tables)
            self.workspace = workspace
            self._keep.append(workspace)
            scales = (ctypes.c_float(k_scale), ctypes.c_float(v_scale)) if self.fp8 else ()
            self._step_args = (_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                               _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               _ptr(context_lens), ctypes.c_float(scale), *scales,
                               _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                               _ptr(self.out), sref)
        elif mode == "fused":
            if workspace is None:
                workspace = step_workspace(q, k_cache.shape[2], self.num_partitions, dev)
            tmp, ml, es, counters = workspace
            self.workspace = workspace
            self._keep += list(workspace)
            scales = (ctypes.c_float(k_scale), ctypes.c_float(v_scale)) if self.fp8 else ()
            self._step_args = (_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                               _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               _ptr(context_lens), ctypes.c_float(scale), *scales,
                               ctypes.c_int32(self.partition_size),
                               ctypes.c_int32(self.num_partitions), _ptr(tmp), _ptr(ml),
                               _ptr(es), _ptr(counters), _ptr(self.out), sref)
        else:
            if workspace is None:
                workspace = split_workspace(q, self.num_partitions)
            tmp, ml, es = workspace
            B, hq, d = q.shape
            if tmp.numel() < B * hq * self.num_partitions * d or \
                    ml.numel() < B * hq * self.num_partitions or \
                    es.numel() < B * hq * self.num_partitions:
                raise PaError("pa_decode_split", PA_ERR_WORKSPACE)
            self.workspace = workspace
            self._keep += list(workspace)
            S = ctypes.c_int32(self.num_partitions)
            P = ctypes.c_int32(self.partition_size)
            self._decode_args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                 _ptr(context_lens), ctypes.c_float(scale), P, S, _ptr(tmp),
                                 _ptr(ml), _ptr(es), sref)
            self._reduce_args = (_ptr(tmp), _ptr(ml), _ptr(es), _ptr(context_lens), P, S,
                                 _ptr(self.out), sref)
        self._graph = None

    def _stream(self):
        return ctypes.c_void_p(torch.cuda.current_stream(self.device).cuda_stream)

    def reshape_and_cache(self):
        if self.mode in ("fused", "balanced") or self._reshape_args is None:
            return                          # part of the fused step, or done before it
        fn = self._lib.pa_reshape_and_cache_fp8 if self.fp8 else self._lib.pa_reshape_and_cache
        _check("pa_reshape_and_cache", fn(*self._reshape_args, self._stream()))

    def decode(self):
        if self.mode == "weights":
            self._decode_weights(self._decode_args)
        elif self.mode == "balanced":
            fn = self._lib.pa_decode_step_balanced_fp8 if self.fp8 else \
                self._lib.pa_decode_step_balanced
            _check("pa_decode_step_balanced", fn(*self._step_args, self._stream()))
        elif self.mode == "fused" and self.fp8:
            _check("pa_decode_step_fp8",
                   self._lib.pa_decode_step_fp8(*self._step_args, self._stream()))
        elif self.mode == "fused":
            _check("pa_decode_step", self._lib.pa_decode_step(*self._step_args, self._stream()))
        elif self.mode == "single":
            _check("pa_decode", self._lib.pa_decode(*self._decode_args, self._stream()))
        else:
            _check("pa_decode_split",
                   self._lib.pa_decode_split(*self._decode_args, self._stream()))

    def _decode_weights(self, args):
        fn = self._lib.pa_decode_weights_fp8 if self.fp8 else self._lib.pa_decode_weights
        _check("pa_decode_weights", fn(*args, self._stream()))

    def _warm(self):
        """The step without a lasting effect: its cache write and its output are
        those of the next step too, but weights that are added up go elsewhere."""
        if self.mode != "weights":
            self()
            return
        i = self._weights_out_at
        scratch = torch.empty_like(self.weights_out)
        self.reshape_and_cache()
        self._decode_weights((*self._decode_args[:i], _ptr(scratch), *self._decode_args[i + 1:]))

    def reduce(self):
        if self.mode == "split":
            _check("pa_reduce", self._lib.pa_reduce(*self._reduce_args, self._stream()))

    def __call__(self) -> torch.Tensor:
        self.reshape_and_cache()
        self.decode()
        self.reduce()
        return self.out

    def capture_graph(self, before=None, after=None) -> "torch.cuda.CUDAGraph":
        """Capture one step into a CUDA graph (replayed by ``replay``).  The
        step itself is not made: ``weights`` are as they were.

        ``before`` / ``after`` are called inside the capture around the step,
        e.g. ``InputStaging.upload`` and the copy of ``out`` to pinned host
        memory, so that a replay uploads, computes and reads back in one
        graph launch; they are called once before the capture too."""
        s = torch.cuda.Stream(self.device)
        s.wait_stream(torch.cuda.current_stream(self.device))
        with torch.cuda.stream(s):                   # warm the lazy set-up outside capture,
            if before is not None:                   # with the same inputs the graph sees
                before()
            self._warm()
            if after is not None:
                after()
        torch.cuda.current_stream(self.device).wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if before is not None:
                before()
            self()
            if after is not None:
                after()
        self._graph = g
        return g

    def replay(self) -> torch.Tensor:
        if self._graph is None:
            self.capture_graph()
        self._graph.replay()
        return self.out
