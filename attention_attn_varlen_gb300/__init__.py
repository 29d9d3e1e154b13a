"""GB300 (sm_103a) varlen / paged attention: thin Python binding of the C ABI.

Every computation runs in the CUDA kernels of ``libattn_varlen.so`` (built
in-tree from ``csrc/`` by :func:`build`).  This module only checks and
marshals arguments: it takes torch CUDA tensors (PyTorch supplies device
memory and streams) and calls the C entry points of ``include/attn_varlen.h``
with their raw pointers on the current stream.  There is no fallback: if the
library is missing or the device is not sm_103 the calls raise.

Entry points (the C ABI's names):
    attn_varlen_fwd         varlen prefill, contiguous or paged K/V (optionally the fp16 V/16 cache)
    attn_varlen_fwd_host    the same prefill for pinned host tensors (copies overlapped by the library)
    attn_decode_paged       single-token decode through the paged cache
    attn_with_kvcache       several new tokens per sequence against the paged cache (attn_kvcache_fwd)
    attn_padded_fwd         a padded [B, S, H, D] batch with per-sequence lengths
    store_kvcache           slot_mapping scatter into the caches (optionally also V/16 in fp16)
    softmax_rows            row softmax (attn_softmax_rows)
    step_tables             a step's block table, slot mapping, positions and offsets from request lengths
    trim_pages              cut requests to fewer tokens, giving their pages back
    rope_store_kvcache      rotary positions (several axes) on q and k, fused with the paged store
    linear_attn_varlen_fwd  linear attention with a decay per head over packed prompts, fp32 state cache
    linear_attn_decode      the same for one token per sequence
    get_last_device_error   the device error word (index, range and timeout checks)
    selftest_bounded_wait   the failure-detection self-test
and the layer-shaped dispatcher in :mod:`attention_attn_varlen_gb300.attention`.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re
from typing import NamedTuple

import torch

from ._build import LIB as _LIB_PATH
from ._build import build

__all__ = ["attn_varlen_fwd", "attn_varlen_fwd_host", "host_staging", "attn_decode_paged", "attn_with_kvcache",
           "attn_padded_fwd", "softmax_rows", "store_kvcache", "step_tables", "trim_pages", "StepTables",
           "rope_store_kvcache", "linear_attn_varlen_fwd", "linear_attn_decode", "linear_attn_workspace_size",
           "get_last_device_error", "selftest_bounded_wait",
           "lib", "build", "AttnError", "exported_symbols", "set_kernel_events", "decode_num_splits",
           "decode_workspace_size"]

ATTN_OK = 0
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace too small", 4: "launch failed",
           5: "device timeout", 6: "device index out of range", 7: "no device", 8: "input value out of range",
           9: "page pool or table row full"}


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)} (status {status})")


_lib = None
_c = ctypes
_vp, _i32, _i64, _f32, _sz = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_float, _c.c_size_t


def lib():
    """The loaded CUDA library (ctypes.CDLL); raises if it was never built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"CUDA attention library not built ({_LIB_PATH} missing); "
                           "run attention_attn_varlen_gb300.build() on a machine with nvcc")
    L = ctypes.CDLL(_LIB_PATH)
    L.attn_varlen_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _i32, _i32, _i32, _i32,
                                  _f32, _i32, _vp, _i32, _i32, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _sz, _vp]
    L.attn_varlen_fwd.restype = _i32
    L.attn_varlen_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i64]
    L.attn_varlen_workspace_size.restype = _sz
    L.attn_decode_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i64, _i32,
                                    _f32, _i32, _i64, _i64, _vp, _sz, _vp]
    L.attn_decode_paged.restype = _i32
    L.attn_decode_paged_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                            _i64, _i32, _f32, _i32, _i64, _i64, _vp]
    L.attn_decode_paged_noalloc.restype = _i32
    L.attn_decode_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    L.attn_decode_workspace_size.restype = _sz
    L.attn_decode_num_splits.argtypes = [_i32, _i32, _i32, _i32]
    L.attn_decode_num_splits.restype = _i32
    L.store_kvcache.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i64, _i64, _i64, _vp]
    L.store_kvcache.restype = _i32
    L.attn_status_string.argtypes = [_i32]
    L.attn_status_string.restype = _c.c_char_p
    L.attn_get_last_device_error.argtypes = [_vp, _c.POINTER(_c.c_uint32)]
    L.attn_get_last_device_error.restype = _i32
    L.attn_abi_version.argtypes = []
    L.attn_abi_version.restype = _i32
    L.attn_selftest_bounded_wait.argtypes = [_vp, _c.POINTER(_c.c_ulonglong)]
    L.attn_selftest_bounded_wait.restype = _i32
    L.attn_kvcache_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                   _i64, _i32, _f32, _i32, _vp, _vp, _sz, _vp]
    L.attn_kvcache_fwd.restype = _i32
    L.attn_kvcache_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    L.attn_kvcache_workspace_size.restype = _sz
    L.attn_padded_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32,
                                  _vp, _sz, _vp]
    L.attn_padded_fwd.restype = _i32
    L.attn_padded_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    L.attn_padded_workspace_size.restype = _sz
    L.attn_softmax_rows.argtypes = [_vp, _vp, _i64, _i32, _i64, _i64, _i32, _vp]
    L.attn_softmax_rows.restype = _i32
    L.attn_set_kernel_events.argtypes = [_vp, _vp]
    L.attn_set_kernel_events.restype = None
    L.attn_varlen_fwd_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32,
                                       _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i32, _vp, _vp, _vp, _vp, _vp]
    L.attn_varlen_fwd_host.restype = _i32
    L.attn_step_tables.argtypes = [_vp] * 6 + [_i32, _i32, _i32, _i32, _i64, _i64] + [_vp] * 8 + [_sz, _vp]
    L.attn_step_tables.restype = _i32
    L.attn_trim_pages.argtypes = [_vp] * 6 + [_i32, _i32, _i32, _i32, _i64, _vp, _sz, _vp]
    L.attn_trim_pages.restype = _i32
    L.attn_step_tables_workspace_size.argtypes = [_i32]
    L.attn_step_tables_workspace_size.restype = _sz
    L.attn_rope_store_kvcache.argtypes = [_vp] * 6 + [_i32, _i64, _i32, _i32, _f32] + [_vp] * 6 + [_i64, _i32, _i32,
                                                                                                _i32] + [_i64] * 6 + [_vp]
    L.attn_rope_store_kvcache.restype = _i32
    L.attn_linear_varlen_fwd.argtypes = [_vp] * 9 + [_i32, _i64, _i32, _i32, _i32, _i32, _f32] + [_i64] * 5 + [_vp, _sz, _vp]
    L.attn_linear_varlen_fwd.restype = _i32
    L.attn_linear_step_fwd.argtypes = [_vp] * 10 + [_i32, _i64, _i32, _i32, _i32, _i32, _f32] + [_i64] * 5 + [_vp, _sz, _vp]
    L.attn_linear_step_fwd.restype = _i32
    L.attn_linear_workspace_size.argtypes = [_i32] * 5
    L.attn_linear_workspace_size.restype = _sz
    L.attn_linear_decode.argtypes = [_vp] * 8 + [_i32, _i32, _i32, _i32, _f32] + [_i64] * 5 + [_vp]
    L.attn_linear_decode.restype = _i32
    _lib = L
    return L


def exported_symbols() -> list[str]:
    """Function names declared in include/attn_varlen.h."""
    hdr = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "attn_varlen.h")
    src = open(hdr).read()
    return re.findall(r"ATTN_API\s+[\w\s\*]+?\b(\w+)\s*\(", src)


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, where: str):
    if status != ATTN_OK:
        raise AttnError(status, where)


def _row_stride(rows: int, stride: int, packed: int, name: str) -> int:
    """The stride to pass for rows of `packed` elements.  A smaller one (0: a tensor expanded along its
    rows) is refused here: the library takes 0 for packed and would read past the tensor."""
    if rows <= 1:
        return packed
    if stride < packed:
        raise ValueError(f"{name}: rows must not overlap (row stride {stride} of rows of {packed} elements)")
    return stride


def _rows(t: torch.Tensor, name: str, heads: int, dim: int) -> int:
    """Row stride (elements) of a [rows, heads, dim] view whose heads and dim are packed."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name}: expected [rows, {heads}, {dim}], got {tuple(t.shape)}")
    if t.stride(2) != 1 or t.stride(1) != dim:
        raise ValueError(f"{name}: heads and head_dim must be packed (strides {t.stride()})")
    return _row_stride(t.shape[0], t.stride(0), heads * dim, name)


def _bf16_cuda(*named):
    for name, t in named:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16")


def _int_cuda(name, t, dtype):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def _cuda(dtype, dev, *named):
    """Each tensor (None allowed) is contiguous, of this dtype and on CUDA device number dev."""
    for name, t in named:
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{dev}")


def _tokens(t, name, dev, rows, heads, dim) -> int:
    """Row stride of a bf16 [rows, heads, dim] tensor on cuda:dev whose heads and dim are packed."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev:
        raise ValueError(f"{name} must be a bfloat16 tensor on cuda:{dev}")
    stride = t.stride()
    if t.shape != (rows, heads, dim) or stride[2] != 1 or stride[1] != dim:
        raise ValueError(f"{name}: expected [{rows}, {heads}, {dim}] with packed heads, got {tuple(t.shape)} "
                         f"(strides {stride})")
    if rows > 1 and stride[0] < heads * dim:
        return _row_stride(rows, stride[0], heads * dim, name)
    return stride[0] if rows > 1 else heads * dim


def _device(t: torch.Tensor, name: str) -> int:
    """The tensor's CUDA device, which has to be the current one (the library launches there)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, which is not the current device")
    return dev


# the current stream's handle without making a Stream object (3 us a call less)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on_stream(call):
    """`stream` becomes the current stream for the call, so that the outputs and the workspace it makes
    belong to that stream: memory of the current one may still be in use there."""
    @functools.wraps(call)
    def on(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return on


def _address(t):
    return None if t is None else t.data_ptr()


def _bytes(workspace, need: int, dev: int, like) -> tuple:
    """(tensor, address, size) of a caller's workspace, or of a new one."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device) if need else None
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    if workspace is None:
        return None, None, 0
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# --------------------------------------------------------------------------
# C-ABI bindings
# --------------------------------------------------------------------------

def attn_varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                    softmax_scale: float | None = None, causal: bool = True, block_table=None,
                    out=None, lse=None, return_lse: bool = False, total_k: int | None = None,
                    workspace=None, stream=None, v16_cache=None):
    """Varlen prefill.  q [total_q, Hq, D]; k/v [total_k, Hkv, D] or, with
    block_table [B, max_blocks] int32, caches [num_blocks, block_size, Hkv, D].
    total_k (paged only): an upper bound of cu_seqlens_k[-1]; defaults to
    B * max_seqlen_k (no device sync).  v16_cache (paged only): the fp16 V / 16
    cache kept by store_kvcache(..., v16_cache=...); the call then converts nothing.
    Returns out [total_q, Hq, D] (and lse [Hq, total_q] float32 if asked)."""
    _bf16_cuda(("q", q), ("k", k), ("v", v), ("out", out))
    if v16_cache is not None:
        if block_table is None:
            raise ValueError("v16_cache goes with a paged cache (block_table)")
        if not v16_cache.is_cuda or v16_cache.dtype != torch.float16 or v16_cache.shape != k.shape \
                or not v16_cache.is_contiguous():
            raise ValueError("v16_cache must be a contiguous float16 CUDA tensor shaped like the caches")
    _int_cuda("cu_seqlens_q", cu_seqlens_q, torch.int32)
    _int_cuda("cu_seqlens_k", cu_seqlens_k, torch.int32)
    total_q, Hq, D = q.shape
    paged = block_table is not None
    if paged:
        _int_cuda("block_table", block_table, torch.int32)
        if k.dim() != 4 or v.shape != k.shape or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("paged k/v must be contiguous [num_blocks, block_size, Hkv, D]")
        num_blocks, block_size, Hkv, _ = k.shape
        k_stride = v_stride = Hkv * D
        bt_stride = block_table.shape[1]
    else:
        Hkv = k.shape[1]
        k_stride = _rows(k, "k", Hkv, D)
        v_stride = _rows(v, "v", Hkv, D)
        total_k = k.shape[0]
        num_blocks = block_size = bt_stride = 0
    q_stride = _rows(q, "q", Hq, D)
    B = cu_seqlens_q.numel() - 1
    if paged and total_k is None:
        total_k = B * int(max_seqlen_k)
    if cu_seqlens_k.numel() != B + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    out_stride = _rows(out, "out", Hq, D)
    if return_lse and lse is None:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    L = lib()
    ws_bytes = L.attn_varlen_workspace_size(B, Hq, Hkv, D, int(max_seqlen_q), 0 if v16_cache is not None
                                            else int(total_k))
    if workspace is None or workspace.numel() * workspace.element_size() < ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws = workspace
    st = L.attn_varlen_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                           B, total_q, total_k, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D, scale,
                           1 if causal else 0, _ptr(block_table), bt_stride, block_size, num_blocks, _ptr(v16_cache),
                           q_stride, k_stride, v_stride, out_stride, _ptr(ws), ws.numel() * ws.element_size(),
                           _stream(stream))
    _check(st, "attn_varlen_fwd")
    return (out, lse) if return_lse else out


def decode_num_splits(batch: int, num_heads_kv: int, max_cache_seqlen: int, num_splits: int = 0) -> int:
    return lib().attn_decode_num_splits(batch, num_heads_kv, max_cache_seqlen, num_splits)


def decode_workspace_size(batch, num_heads_q, num_heads_kv, head_dim, max_cache_seqlen, num_splits=0) -> int:
    return lib().attn_decode_workspace_size(batch, num_heads_q, num_heads_kv, head_dim, max_cache_seqlen,
                                            num_splits)


def host_staging(batch: int, total_q: int, total_k: int, num_heads_q: int, num_heads_kv: int, head_dim: int,
                 max_seqlen_q: int, device=None) -> dict:
    """Device buffers, copy streams and events that attn_varlen_fwd_host uses;
    make them once and pass them to every call of the same (or smaller) sizes."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    ws = lib().attn_varlen_workspace_size(batch, num_heads_q, num_heads_kv, head_dim, int(max_seqlen_q), int(total_k))
    if ws == 0:
        raise ValueError("unsupported sizes for attn_varlen_fwd_host")
    bf = torch.bfloat16
    st = dict(q=torch.empty((total_q, num_heads_q, head_dim), dtype=bf, device=device),
              k=torch.empty((total_k, num_heads_kv, head_dim), dtype=bf, device=device),
              v=torch.empty((total_k, num_heads_kv, head_dim), dtype=bf, device=device),
              out=torch.empty((total_q, num_heads_q, head_dim), dtype=bf, device=device),
              cu=torch.empty(2 * (batch + 1), dtype=torch.int32, device=device),
              ws=torch.empty(ws, dtype=torch.uint8, device=device),
              s_in=torch.cuda.Stream(device), s_out=torch.cuda.Stream(device),
              ev=(torch.cuda.Event(), torch.cuda.Event()))
    for e in st["ev"]:
        e.record(torch.cuda.current_stream(device))   # torch creates the CUDA event on its first record
    return st


def attn_varlen_fwd_host(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                         softmax_scale: float | None = None, causal: bool = True, out=None, chunks: int = 8,
                         device=None, staging=None, synchronize: bool = True):
    """attn_varlen_fwd for host-resident inputs (C entry attn_varlen_fwd_host):
    q, k, v contiguous bf16 CPU tensors (pinned for the copies to overlap),
    cu_seqlens int32 CPU tensors.  The library copies groups of sequences in,
    runs the attention of each group and copies its output back, overlapped on
    three streams.  Returns the output in a pinned CPU tensor (`out` if given);
    with synchronize=True (default) after it has arrived.  `staging` (from
    host_staging) supplies reusable device buffers, streams and events."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 3:
            raise ValueError(f"{name} must be a contiguous [rows, heads, dim] bf16 CPU tensor")
    cq = torch.as_tensor(cu_seqlens_q)
    ck = torch.as_tensor(cu_seqlens_k)
    for name, t in (("cu_seqlens_q", cq), ("cu_seqlens_k", ck)):
        if t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CPU tensor")
    total_q, Hq, D = q.shape
    total_k, Hkv, _ = k.shape
    B = cq.numel() - 1
    if ck.numel() != B + 1 or v.shape != k.shape:
        raise ValueError("cu_seqlens_q / cu_seqlens_k / k / v do not match")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if staging is None:
        staging = host_staging(B, total_q, total_k, Hq, Hkv, D, max_seqlen_q, device)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype).pin_memory()
    elif out.is_cuda or out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 CPU tensor shaped like q")
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    main = torch.cuda.current_stream(device)
    ws = staging["ws"]
    ev_a, ev_b = staging["ev"]
    st = lib().attn_varlen_fwd_host(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(cq), _ptr(ck), B, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv,
        D, scale, 1 if causal else 0, _ptr(staging["q"]), _ptr(staging["k"]), _ptr(staging["v"]),
        _ptr(staging["out"]), _ptr(staging["cu"]), _ptr(ws), ws.numel(), int(chunks),
        ctypes.c_void_p(main.cuda_stream), ctypes.c_void_p(staging["s_in"].cuda_stream),
        ctypes.c_void_p(staging["s_out"].cuda_stream), ctypes.c_void_p(ev_a.cuda_event),
        ctypes.c_void_p(ev_b.cuda_event))
    _check(st, "attn_varlen_fwd_host")
    if synchronize:
        main.synchronize()
    return out


def attn_decode_paged(q, k_cache, v_cache, cache_seqlens, block_table, softmax_scale: float | None = None,
                      max_cache_seqlen: int | None = None, num_splits: int = 0, out=None, lse=None,
                      return_lse: bool = False, workspace=None, stream=None):
    """Decode: q [B, Hq, D] (or [B, 1, Hq, D]); caches [num_blocks, block_size,
    Hkv, D]; cache_seqlens int32 [B]; block_table int32 [B, max_blocks]; at most
    64 query heads per KV head.  max_cache_seqlen defaults to the block table's
    capacity (no device sync)."""
    if q.dim() == 4:
        if q.shape[1] != 1:
            raise ValueError("attn_decode_paged takes one query token per sequence")
        q = q[:, 0]
    _bf16_cuda(("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("out", out))
    _int_cuda("cache_seqlens", cache_seqlens, torch.int32)
    _int_cuda("block_table", block_table, torch.int32)
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or not k_cache.is_contiguous() \
            or not v_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, D]")
    B, Hq, D = q.shape
    num_blocks, block_size, Hkv, _ = k_cache.shape
    q_stride = _rows(q, "q", Hq, D)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    out_stride = _rows(out, "out", Hq, D)
    if return_lse and lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if max_cache_seqlen is None:
        max_cache_seqlen = block_table.shape[1] * block_size
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    L = lib()
    ws_bytes = L.attn_decode_workspace_size(B, Hq, Hkv, D, int(max_cache_seqlen), int(num_splits))
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_have = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = L.attn_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), _ptr(cache_seqlens),
                             _ptr(block_table), block_table.shape[1], B, Hq, Hkv, D, block_size, num_blocks,
                             int(max_cache_seqlen), scale, int(num_splits), q_stride, out_stride, _ptr(workspace),
                             ws_have, _stream(stream))
    _check(st, "attn_decode_paged")
    return (out, lse) if return_lse else out


def attn_with_kvcache(q, k_cache, v_cache, cache_seqlens, block_table, softmax_scale: float | None = None,
                      causal: bool = True, max_cache_seqlen: int | None = None, out=None, lse=None,
                      return_lse: bool = False, workspace=None, stream=None, v16_cache=None):
    """Several new tokens per sequence against the paged cache: q [B, Sq, Hq, D]
    (Sq >= 1, all sequences the same Sq); caches [num_blocks, block_size, Hkv, D];
    cache_seqlens int32 [B] counts the cached keys including the Sq new ones.
    Returns out [B, Sq, Hq, D] (and lse [Hq, B*Sq]).  Up to 64 query rows per KV
    head (Sq x Hq/Hkv) run on the split-KV decode kernel, more on the prefill kernel
    (which reads v16_cache, the fp16 V / 16 cache, when given)."""
    if v16_cache is not None and (not v16_cache.is_cuda or v16_cache.dtype != torch.float16
                                  or v16_cache.shape != k_cache.shape or not v16_cache.is_contiguous()):
        raise ValueError("v16_cache must be a contiguous float16 CUDA tensor shaped like the caches")
    if q.dim() != 4:
        raise ValueError("q must be [B, seqlen_q, Hq, D]")
    _bf16_cuda(("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("out", out))
    _int_cuda("cache_seqlens", cache_seqlens, torch.int32)
    _int_cuda("block_table", block_table, torch.int32)
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or not k_cache.is_contiguous() \
            or not v_cache.is_contiguous():
        raise ValueError("caches must be contiguous [num_blocks, block_size, Hkv, D]")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    B, Sq, Hq, D = q.shape
    num_blocks, block_size, Hkv, _ = k_cache.shape
    if cache_seqlens.numel() != B or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("cache_seqlens / block_table do not match the batch")
    if out is None:
        out = torch.empty((B, Sq, Hq, D), dtype=torch.bfloat16, device=q.device)
    elif out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped like q")
    if return_lse and lse is None:
        lse = torch.empty((Hq, B * Sq), dtype=torch.float32, device=q.device)
    if max_cache_seqlen is None:
        max_cache_seqlen = block_table.shape[1] * block_size
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    L = lib()
    ws_bytes = L.attn_kvcache_workspace_size(B, Sq, Hq, Hkv, D, int(max_cache_seqlen))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    ws_have = workspace.numel() * workspace.element_size()
    st = L.attn_kvcache_fwd(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), _ptr(cache_seqlens),
                            _ptr(block_table), block_table.shape[1], B, Sq, Hq, Hkv, D, block_size, num_blocks,
                            int(max_cache_seqlen), scale, 1 if causal else 0, _ptr(v16_cache), _ptr(workspace),
                            ws_have, _stream(stream))
    _check(st, "attn_kvcache_fwd")
    return (out, lse) if return_lse else out


def attn_padded_fwd(q, k, v, seqlens_q=None, seqlens_k=None, softmax_scale: float | None = None,
                    causal: bool = True, out=None, lse=None, return_lse: bool = False, workspace=None,
                    stream=None):
    """Padded batch: q [B, Sq, Hq, D], k/v [B, Sk, Hkv, D] (contiguous); only the
    first seqlens_q[b] / seqlens_k[b] rows of sequence b are real (int32 [B],
    None = all).  Returns out [B, Sq, Hq, D] (padding rows are not written) and
    lse [Hq, B*Sq] if asked."""
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("q must be [B, Sq, Hq, D] and k, v [B, Sk, Hkv, D]")
    _bf16_cuda(("q", q), ("k", k), ("v", v), ("out", out))
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    B, Sq, Hq, D = q.shape
    _, Sk, Hkv, _ = k.shape
    if k.shape[0] != B or k.shape[3] != D:
        raise ValueError("k does not match q")
    for name, t in (("seqlens_q", seqlens_q), ("seqlens_k", seqlens_k)):
        if t is not None:
            _int_cuda(name, t, torch.int32)
            if t.numel() != B:
                raise ValueError(f"{name} must have one entry per sequence")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped like q")
    if return_lse and lse is None:
        lse = torch.empty((Hq, B * Sq), dtype=torch.float32, device=q.device)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    L = lib()
    ws_bytes = L.attn_padded_workspace_size(B, Sq, Sk, Hq, Hkv, D)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    ws_have = workspace.numel() * workspace.element_size()
    st = L.attn_padded_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(seqlens_q), _ptr(seqlens_k), B, Sq,
                           Sk, Hq, Hkv, D, scale, 1 if causal else 0, _ptr(workspace), ws_have, _stream(stream))
    _check(st, "attn_padded_fwd")
    return (out, lse) if return_lse else out


def softmax_rows(x, out=None, stream=None):
    """Softmax along the last dimension of a float32 or bfloat16 CUDA tensor
    (any leading shape; rows may be strided, the last dimension contiguous).
    out: same shape and dtype (may be x)."""
    if not x.is_cuda or x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("x must be a float32 or bfloat16 CUDA tensor")
    if x.dim() == 0 or x.stride(-1) != 1:
        raise ValueError("the last dimension of x must be contiguous")
    cols = x.shape[-1]
    x2 = x.reshape(-1, cols) if x.dim() != 2 else x
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    if out.shape != x.shape or out.dtype != x.dtype or out.stride(-1) != 1:
        raise ValueError("out must match x in shape and dtype")
    o2 = out.reshape(-1, cols) if out.dim() != 2 else out
    if o2.data_ptr() != out.data_ptr() or x2.data_ptr() != x.data_ptr():
        raise ValueError("x and out must be viewable as [rows, cols]")
    dtype = 1 if x.dtype == torch.bfloat16 else 0
    rows = x2.shape[0]
    st = lib().attn_softmax_rows(_ptr(x2), _ptr(o2), rows, cols, _row_stride(rows, x2.stride(0), cols, "x"),
                                 _row_stride(rows, o2.stride(0), cols, "out"), dtype, _stream(stream))
    _check(st, "attn_softmax_rows")
    return out


def store_kvcache(k, v, k_cache, v_cache, slot_mapping, stream=None, v16_cache=None):
    """Scatter k/v [N, Hkv, D] into caches [num_blocks, block_size, Hkv, D] (or
    any [num_slots, Hkv, D] view) at the flat slots slot_mapping (int64 [N]).
    v16_cache (float16, shaped like the caches): also receives V / 16."""
    _bf16_cuda(("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache))
    if v16_cache is not None and (not v16_cache.is_cuda or v16_cache.dtype != torch.float16
                                  or v16_cache.shape != v_cache.shape or not v16_cache.is_contiguous()):
        raise ValueError("v16_cache must be a contiguous float16 CUDA tensor shaped like the caches")
    _int_cuda("slot_mapping", slot_mapping, torch.int64)
    N, Hkv, D = k.shape
    if not k_cache.is_contiguous() or not v_cache.is_contiguous() or k_cache.shape != v_cache.shape:
        raise ValueError("caches must be contiguous and of the same shape")
    if k_cache.shape[-2:] != (Hkv, D):
        raise ValueError("cache head layout does not match k")
    num_slots = k_cache.numel() // (Hkv * D)
    ks = _rows(k, "k", Hkv, D)
    vs = _rows(v, "v", Hkv, D)
    if slot_mapping.numel() != N:
        raise ValueError("slot_mapping must have one entry per token")
    st = lib().store_kvcache(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(v16_cache), _ptr(slot_mapping), N,
                             Hkv, D, ks, vs, num_slots, _stream(stream))
    _check(st, "store_kvcache")


class StepTables(NamedTuple):
    """The index tables of one step (see attn_step_tables), all on the device."""
    block_table: torch.Tensor      # int32 [B, max_blocks]
    slot_mapping: torch.Tensor     # int64 [max_tokens]
    positions: torch.Tensor        # int32 [max_tokens]
    cu_seqlens_q: torch.Tensor     # int32 [B + 1]
    cu_seqlens_k: torch.Tensor     # int32 [B + 1]
    cache_seqlens: torch.Tensor    # int32 [B]: cached tokens after the step
    context_lens: torch.Tensor     # int32 [B]: cached tokens before it

    @classmethod
    def empty(cls, batch: int, max_blocks: int, max_tokens: int, device=None) -> "StepTables":
        """Buffers for steps of this size, to keep and pass as `out`."""
        new = lambda dt, *shape: torch.empty(shape, dtype=dt, device=device or "cuda")  # noqa: E731
        i32 = torch.int32
        return cls(new(i32, batch, max_blocks), new(torch.int64, max_tokens), new(i32, max_tokens),
                   new(i32, batch + 1), new(i32, batch + 1), new(i32, batch), new(i32, batch))


def _pool_args(request_rows, lens, seq_lens, page_table, free_pages, num_free, lens_name):
    dev = _device(seq_lens, "seq_lens")
    _cuda(torch.int32, dev, ("request_rows", request_rows), (lens_name, lens), ("seq_lens", seq_lens),
          ("page_table", page_table), ("free_pages", free_pages), ("num_free", num_free))
    if page_table.dim() != 2 or seq_lens.dim() != 1 or page_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("page_table must be [num_rows, max_blocks] and seq_lens [num_rows]")
    if num_free.numel() != 1:
        raise ValueError("num_free must hold one number")
    B = lens.numel()
    if request_rows is not None and request_rows.numel() != B:
        raise ValueError(f"request_rows and {lens_name} must have the same length")
    return dev, B


@_on_stream
def step_tables(request_rows, new_lens, seq_lens, page_table, free_pages, num_free, block_size: int,
                max_tokens: int, out: StepTables | None = None, workspace=None, *, stream=None) -> StepTables:
    """Grow the requests of a step by their new tokens, taking pages off the
    free list, and build the step's tables on the GPU (no host sync).

    Pool, updated in place: seq_lens int32 [R], page_table int32 [R, M],
    free_pages int32 [num_pages] (the first num_free entries), num_free int32
    [1].  Step: request_rows int32 [B] (None: entry b is row b), new_lens int32
    [B]; max_tokens sizes slot_mapping and positions (entries behind the last
    token are -1 and 0).  Entries that cannot be served keep their length, get
    slots of -1 and are reported by get_last_device_error (9: out of pages)."""
    dev, B = _pool_args(request_rows, new_lens, seq_lens, page_table, free_pages, num_free, "new_lens")
    R, M = page_table.shape
    if out is None:
        out = StepTables.empty(B, M, int(max_tokens), seq_lens.device)
    else:
        _cuda(torch.int32, dev, ("block_table", out.block_table), ("positions", out.positions),
              ("cu_seqlens_q", out.cu_seqlens_q), ("cu_seqlens_k", out.cu_seqlens_k),
              ("cache_seqlens", out.cache_seqlens), ("context_lens", out.context_lens))
        _cuda(torch.int64, dev, ("slot_mapping", out.slot_mapping))
        if out.block_table.shape != (B, M) or out.slot_mapping.numel() != max_tokens \
                or out.positions.numel() != max_tokens or out.cu_seqlens_q.numel() != B + 1 \
                or out.cu_seqlens_k.numel() != B + 1 or out.cache_seqlens.numel() != B or out.context_lens.numel() != B:
            raise ValueError("out was made for other sizes")
    L = lib()
    workspace, ws, ws_bytes = _bytes(workspace, L.attn_step_tables_workspace_size(B), dev, seq_lens)
    st = L.attn_step_tables(_address(request_rows), new_lens.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(),
                            free_pages.data_ptr(), num_free.data_ptr(), B, R, M, int(block_size), free_pages.numel(),
                            int(max_tokens), out.block_table.data_ptr(), out.slot_mapping.data_ptr(),
                            out.positions.data_ptr(), out.cu_seqlens_q.data_ptr(), out.cu_seqlens_k.data_ptr(),
                            out.cache_seqlens.data_ptr(), out.context_lens.data_ptr(), ws, ws_bytes,
                            _raw_stream(dev))
    _check(st, "attn_step_tables")
    return out


@_on_stream
def trim_pages(request_rows, keep_lens, seq_lens, page_table, free_pages, num_free, block_size: int, workspace=None,
               *, stream=None) -> None:
    """Cut requests to their first keep_lens tokens (int32 [B]; 0 ends a
    request) and give the pages behind them back to the free list."""
    dev, B = _pool_args(request_rows, keep_lens, seq_lens, page_table, free_pages, num_free, "keep_lens")
    R, M = page_table.shape
    L = lib()
    workspace, ws, ws_bytes = _bytes(workspace, L.attn_step_tables_workspace_size(B), dev, seq_lens)
    st = L.attn_trim_pages(_address(request_rows), keep_lens.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(),
                           free_pages.data_ptr(), num_free.data_ptr(), B, R, M, int(block_size), free_pages.numel(),
                           ws, ws_bytes, _raw_stream(dev))
    _check(st, "attn_trim_pages")


@_on_stream
def rope_store_kvcache(q, k, v, positions, inv_freq, k_cache=None, v_cache=None, slot_mapping=None, pair_axis=None,
                       interleaved: bool = False, scale: float = 1.0, q_out=None, k_out=None, return_k: bool = False,
                       v16_cache=None, *, stream=None):
    """Rotary positions on q [N, Hq, D] and k [N, Hkv, D], and the scatter of the
    rotated k and of v into the caches (as store_kvcache), in one pass.

    positions int32 [N], or [A, N] with pair_axis (a sequence of A-axis numbers,
    one per pair; [N] expanded to [A, N] will do); inv_freq float32 [rot_dim / 2].  Pair i is elements (i, i +
    rot_dim / 2), or (2 i, 2 i + 1) if interleaved; elements past rot_dim pass
    through.  Without caches only q and k are rotated (v may be None).  q_out and
    k_out may be q and k.  Returns the rotated q, or (q, k) with return_k."""
    dev = _device(q, "q")
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    num_slots = 0
    if k_cache is not None or v_cache is not None or slot_mapping is not None or v16_cache is not None:
        if k_cache is None or v_cache is None or slot_mapping is None or v is None:
            raise ValueError("storing needs v, k_cache, v_cache and slot_mapping")
        _cuda(torch.bfloat16, dev, ("k_cache", k_cache), ("v_cache", v_cache))
        _cuda(torch.float16, dev, ("v16_cache", v16_cache))
        _cuda(torch.int64, dev, ("slot_mapping", slot_mapping))
        if k_cache.shape != v_cache.shape or k_cache.shape[-2:] != (Hkv, D) \
                or (v16_cache is not None and v16_cache.shape != v_cache.shape):
            raise ValueError("the caches must have one shape [..., Hkv, D], k's heads and head_dim")
        if slot_mapping.numel() != N:
            raise ValueError("slot_mapping must have one entry per token")
        num_slots = k_cache.numel() // (Hkv * D)
    elif k_out is None:
        return_k = True
    qs, ks = _tokens(q, "q", dev, N, Hq, D), _tokens(k, "k", dev, N, Hkv, D)
    vs = _tokens(v, "v", dev, N, Hkv, D) if v is not None else 0
    if q_out is None:
        q_out = torch.empty((N, Hq, D), dtype=q.dtype, device=q.device)
    if k_out is None and return_k:
        k_out = torch.empty((N, Hkv, D), dtype=q.dtype, device=q.device)
    qos = _tokens(q_out, "q_out", dev, N, Hq, D)
    kos = _tokens(k_out, "k_out", dev, N, Hkv, D) if k_out is not None else 0
    _cuda(torch.float32, dev, ("inv_freq", inv_freq))
    axes = positions.shape[0] if positions.dim() == 2 else 1
    if positions.dtype is not torch.int32 or positions.get_device() != dev or positions.dim() not in (1, 2) \
            or positions.shape[-1] != N or (N > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions must be int32 [{N}] or [axes, {N}] on cuda:{dev}, contiguous along the tokens")
    pairs = inv_freq.numel()
    if pair_axis is not None:
        pair_axis = bytes(pair_axis)
        if len(pair_axis) != pairs:
            raise ValueError("pair_axis must have one entry per pair (inv_freq)")
    elif axes > 1:
        raise ValueError("positions with several axes need pair_axis")
    axis_stride = positions.stride(0) if axes > 1 else N
    if axes > 1 and axis_stride == 0:
        # one row expanded: all axes are that one
        if max(pair_axis, default=0) >= axes:
            raise ValueError(f"pair_axis must name axes below {axes}")
        axes, pair_axis, axis_stride = 1, None, N
    st = lib().attn_rope_store_kvcache(
        q.data_ptr(), k.data_ptr(), _address(v), positions.data_ptr(), inv_freq.data_ptr(), pair_axis, axes,
        axis_stride, 2 * pairs, 1 if interleaved else 0, float(scale), q_out.data_ptr(),
        _address(k_out), _address(k_cache), _address(v_cache), _address(v16_cache), _address(slot_mapping), N, Hq,
        Hkv, D, qs, ks, vs, qos, kos, num_slots, _raw_stream(dev))
    _check(st, "attn_rope_store_kvcache")
    return (q_out, k_out) if return_k else q_out


def _linear_args(q, k, v, log_decay, state_cache, state_slots, context_lens, out, B):
    dev = _device(q, "q")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if out is None:
        out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
    strides = (_tokens(q, "q", dev, T, Hq, D), _tokens(k, "k", dev, T, Hkv, D), _tokens(v, "v", dev, T, Hkv, D),
               _tokens(out, "out", dev, T, Hq, D))
    _cuda(torch.float32, dev, ("log_decay", log_decay), ("state_cache", state_cache))
    _cuda(torch.int32, dev, ("state_slots", state_slots), ("context_lens", context_lens))
    if log_decay.numel() != Hkv:
        raise ValueError("log_decay must have one entry per key/value head")
    if (state_cache is None) != (state_slots is None):
        raise ValueError("state_cache and state_slots go together")
    slots = 0
    if state_cache is not None:
        slots = state_cache.shape[0]
        if state_cache.shape != (slots, Hkv, D, D):
            raise ValueError(f"state_cache must be [num_slots, {Hkv}, {D}, {D}]")
        if state_slots.numel() != B:
            raise ValueError("state_slots must have one entry per sequence")
    if context_lens is not None and context_lens.numel() != B:
        raise ValueError("context_lens must have one entry per sequence")
    return dev, out, T, Hq, Hkv, D, slots, strides


def linear_attn_workspace_size(batch: int, num_heads_q: int, num_heads_kv: int, head_dim: int, max_seqlen: int) -> int:
    return lib().attn_linear_workspace_size(batch, num_heads_q, num_heads_kv, head_dim, max_seqlen)


@_on_stream
def linear_attn_varlen_fwd(q, k, v, log_decay, cu_seqlens, max_seqlen: int, scale: float | None = None,
                           state_cache=None, state_slots=None, context_lens=None, out=None, workspace=None,
                           cache_seqlens=None, *, stream=None):
    """Linear attention with a decay per head over packed sequences:
    S_t = exp(log_decay) S_{t-1} + v_t k_t^T, o_t = scale * S_t q_t.

    q [T, Hq, D], k/v [T, Hkv, D] bf16 (D 64 or 128), log_decay float32 [Hkv] <=
    0, cu_seqlens int32 [B + 1].  state_cache float32 [num_slots, Hkv, Dv, Dk]
    with state_slots int32 [B] receives the final states; a sequence with
    context_lens[b] > 0 (int32 [B]) starts from its slot, any other from zero.
    cache_seqlens (int32 [B], of step_tables): a sequence in which it is not above
    context_lens was refused, and its state stays as it was.  scale defaults to
    1 / sqrt(D).  Returns out [T, Hq, D]."""
    B = cu_seqlens.numel() - 1
    dev, out, T, Hq, Hkv, D, slots, strides = _linear_args(q, k, v, log_decay, state_cache, state_slots, context_lens,
                                                           out, B)
    _cuda(torch.int32, dev, ("cu_seqlens", cu_seqlens), ("cache_seqlens", cache_seqlens))
    if cache_seqlens is not None and cache_seqlens.numel() != B:
        raise ValueError("cache_seqlens must have one entry per sequence")
    L = lib()
    max_seqlen = int(max_seqlen)
    workspace, ws, ws_bytes = _bytes(workspace, L.attn_linear_workspace_size(B, Hq, Hkv, D, max_seqlen), dev, q)
    st = L.attn_linear_step_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), log_decay.data_ptr(),
                                cu_seqlens.data_ptr(), _address(state_cache), _address(state_slots),
                                _address(context_lens), _address(cache_seqlens), B, T, max_seqlen, Hq, Hkv, D,
                                1.0 / math.sqrt(D) if scale is None else scale, slots, *strides, ws, ws_bytes,
                                _raw_stream(dev))
    _check(st, "attn_linear_varlen_fwd")
    return out


@_on_stream
def linear_attn_decode(q, k, v, log_decay, state_cache, state_slots, scale: float | None = None, context_lens=None,
                       out=None, *, stream=None):
    """linear_attn_varlen_fwd for one token per sequence: q [B, Hq, D], k/v [B,
    Hkv, D]; the states in state_cache are updated in place.  A slot < 0 stands
    for a zero state that is not kept; context_lens[b] = 0 starts from zero
    (None: every slot continues).  Returns out [B, Hq, D]."""
    dev, out, B, Hq, Hkv, D, slots, strides = _linear_args(q, k, v, log_decay, state_cache, state_slots, context_lens,
                                                           out, q.shape[0])
    st = lib().attn_linear_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), log_decay.data_ptr(),
                                  _address(state_cache), _address(state_slots), _address(context_lens), B, Hq, Hkv, D,
                                  1.0 / math.sqrt(D) if scale is None else scale, slots, *strides,
                                  _raw_stream(dev))
    _check(st, "attn_linear_decode")
    return out


def set_kernel_events(before=None, after=None) -> None:
    """Record two torch.cuda.Event objects (created with enable_timing=True)
    around the main kernel of every later attention call from this thread:
    the prefill's attention kernel or the decode's split-KV kernel.  Call
    with no arguments to switch it off.  Measurement aid for benchmarks."""
    if (before is None) != (after is None):
        raise ValueError("give both events or neither")
    if before is None:
        lib().attn_set_kernel_events(None, None)
        return
    # torch creates the CUDA event on its first record()
    for e in (before, after):
        if not e.cuda_event:
            e.record()
    if not before.cuda_event or not after.cuda_event:
        raise ValueError("events have no CUDA event handle")
    lib().attn_set_kernel_events(ctypes.c_void_p(before.cuda_event), ctypes.c_void_p(after.cuda_event))


def selftest_bounded_wait(stream=None) -> dict:
    """Run the library's failure-detection self-test (a bounded wait that runs
    out on purpose; see attn_selftest_bounded_wait).  Returns the two waiters'
    success flags and waited nanoseconds; the device error word then holds the
    timeout."""
    res = (ctypes.c_ulonglong * 4)()
    _check(lib().attn_selftest_bounded_wait(_stream(stream), res), "attn_selftest_bounded_wait")
    return {"first_ok": bool(res[0]), "first_ns": int(res[1]), "second_ok": bool(res[2]), "second_ns": int(res[3])}


def get_last_device_error(stream=None) -> tuple[int, int]:
    """Synchronise the stream and read / clear the device error word.
    Returns (status, raw word)."""
    word = ctypes.c_uint32(0)
    st = lib().attn_get_last_device_error(_stream(stream), ctypes.byref(word))
    return st, word.value
