"""Paged KV-cache decode on GB300 (sm_103a).

Python binding over the C ABI of ``libpagedkv.so`` (include/pagedkv.h).  The
functions here only marshal torch tensors into pointers and sizes; all device
work runs in the library's CUDA kernels, and the block manager runs in the
library's C++ host code.  There is no CPU fallback: a missing library raises.

    paged_kv_append(k, v, slot_mapping, k_cache, v_cache, ...)
    paged_attention_decode(q, k_cache, v_cache, block_tables, context_lens, scale, ...)
    paged_attention_decode_append(q, k_new, v_new, slot_mapping, k_cache, v_cache, ...)
    DecodePlan(...).run()   # either of the two above, marshalled once for fixed buffers
    paged_block_copy(k_cache, v_cache, src_dst_pairs, ...)
    paged_extend_tables(block_tables, context_lens, new_lens, free_blocks, free_head, ...)
    paged_rope_append(q, k, v, positions, slot_mapping, inv_freq, k_cache, v_cache, ...)
    paged_kv_append_scaled(k, v, slot_mapping, k_cache, v_cache, k_scales, v_scales)
    paged_attention_decode_scaled(q, k_cache, v_cache, k_scales, v_scales, block_tables, ...)
    BlockManager(num_blocks, block_size, free_list=None)

Cache tensors are [num_blocks, num_kv_heads, block_size, head_dim], float16 or
bfloat16, or uint8 / float8_e4m3fn holding E4M3 codes with float32 scales:
per tensor (1-element CUDA tensors k_scale, v_scale) or, block-scaled, one for
each block and kv head (k_scales, v_scales [num_blocks, num_kv_heads]).
"""
from __future__ import annotations

import ctypes
import functools
import math
import threading
from typing import NamedTuple

import numpy as np
import torch

from . import _native
from ._native import PagedKVError

F16, BF16, E4M3 = 0, 1, 2
PARTITION_SINGLE = 0
PARTITION_AUTO = -1

ERR_INVALID, ERR_SHAPE, ERR_CUDA, ERR_NO_SPACE, ERR_NOT_FOUND = 1, 2, 3, 4, 5
DEV_BAD_BLOCK, DEV_BAD_CONTEXT_LEN, DEV_BAD_SLOT, DEV_BAD_PAIR, DEV_WAIT_TIMEOUT = 1, 2, 4, 8, 16
DEV_NO_SPACE = 32
PATH_AUTO, PATH_CUDA_CORE, PATH_TENSOR, PATH_TENSOR_2CTA = 0, 1, 2, 3
SWAP_OUT, SWAP_IN = 0, 1

__all__ = ["paged_kv_append", "paged_attention_decode", "paged_attention_decode_append", "DecodePlan",
           "paged_block_copy",
           "paged_block_swap", "paged_attention_decode_sparse", "quest_block_minmax", "quest_append_minmax",
           "quest_select", "paged_extend_tables", "ExtendedTables", "rope_inv_freq", "paged_rope_append",
           "paged_kv_append_scaled", "paged_attention_decode_scaled", "workspace_size",
           "resolve_partition_size", "device_error", "set_kernel_path", "BlockManager", "OutOfBlocks", "PagedKVError",
           "F16", "BF16", "E4M3", "PARTITION_SINGLE", "PARTITION_AUTO", "load"]


class OutOfBlocks(PagedKVError):
    pass


def load():
    """Load libpagedkv.so (raises if it was not built)."""
    return _native.lib()


_CODES = {torch.float16: F16, torch.bfloat16: BF16, torch.uint8: E4M3, torch.float8_e4m3fn: E4M3}


def _code(t: torch.Tensor) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported element type {t.dtype}")
    return code


def _ptr(t):
    # ctypes converts a Python int for a c_void_p argument
    return None if t is None else t.data_ptr()


def _stream(stream, device) -> int:
    if stream is None:
        if device.index is not None:
            return torch._C._cuda_getCurrentRawStream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _require_out(device, out):
    """`out` may be a CUDA tensor on `device` or a pinned host tensor, which the
    kernels write directly over the host link."""
    if out.is_cuda and out.get_device() == device.index and out.is_contiguous():
        return
    if out.is_pinned() and not out.is_cuda:
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        return
    _require_cuda(device, out=out)


def _require_cuda(device, **tensors):
    index = device.index if device.index is not None else torch.cuda.current_device()
    for name, t in tensors.items():
        if t is None:
            continue
        if t.get_device() != index:  # -1 for a CPU tensor
            raise ValueError(f"{name} must be a CUDA tensor on {device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def paged_kv_append(k, v, slot_mapping, k_cache, v_cache, k_scale=None, v_scale=None, stream=None):
    """Write k, v [T, Hkv, D] into their slots (int64 [T], negative = skip)."""
    T, Hkv, D = k.shape
    NB, Hkv2, bs, D2 = k_cache.shape
    if v.shape != k.shape or v_cache.shape != k_cache.shape or Hkv2 != Hkv or D2 != D:
        raise ValueError("paged_kv_append: shape mismatch")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,):
        raise ValueError("paged_kv_append: slot_mapping must be int64 [num_tokens]")
    _require_cuda(k.device, k=k, v=v, slot_mapping=slot_mapping, k_cache=k_cache, v_cache=v_cache,
                  k_scale=k_scale, v_scale=v_scale)
    _native.call("paged_kv_append", _ptr(k), _ptr(v), _ptr(slot_mapping), T, _ptr(k_cache), _ptr(v_cache),
                 NB, Hkv, bs, D, _code(k), _code(k_cache), _ptr(k_scale), _ptr(v_scale),
                 _stream(stream, k.device))


def set_kernel_path(path: int) -> int:
    """Select the decode kernel (PATH_*) for later calls; returns the previous choice."""
    prev = int(_native.lib().pkv_set_kernel_path(int(path)))
    if prev < 0:
        raise ValueError(f"unknown kernel path {path}")
    return prev


def resolve_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size,
                           partition_size=PARTITION_AUTO, block_scales=False):
    fn = _native.lib().pkv_scaled_partition_size if block_scales else _native.lib().pkv_resolve_partition_size
    return int(fn(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size, partition_size))


def workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size,
                   partition_size=PARTITION_AUTO, block_scales=False) -> int:
    """Bytes of workspace of paged_attention_decode (block_scales: of paged_attention_decode_scaled)."""
    fn = _native.lib().pkv_scaled_workspace_size if block_scales else _native.lib().pkv_workspace_size
    return int(fn(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size, partition_size))


_ws_lock = threading.Lock()
_ws_cache: dict = {}


def _torch_stream(stream, device) -> torch.cuda.Stream:
    """`stream`, any object with a cuda_stream handle, as torch's own."""
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream, device)


def _output(stream, device, shape, dtype, zero=False) -> torch.Tensor:
    """A new output of a call on `stream` (default: the current one).  It is allocated there, so that no work of the
    current stream still holds its bytes, and marked as used on the current stream, where its reader may be."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    reader = torch.cuda.current_stream(device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        t = make(shape, dtype=dtype, device=device)
    t.record_stream(reader)
    return t


def _workspace(device, stream, nbytes: int, kind: int = 0) -> torch.Tensor:
    """A reusable workspace per (device, stream) and kind of call: calls on one stream are ordered.  It is allocated on
    the stream that uses it (default: the current one), so that a smaller one that it replaces is not handed out again
    before the calls in flight are done with it.  A call that is being captured gets one of its own, from the graph's
    memory: the reusable one may be replaced while the graph lives."""
    if stream is not None:
        with torch.cuda.stream(_torch_stream(stream, device)):
            return _workspace(device, None, nbytes, kind)
    if torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, _stream(None, device), kind)
    with _ws_lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
            _ws_cache[key] = buf
        return buf


def paged_attention_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, k_scale=None,
                           v_scale=None, partition_size=PARTITION_AUTO, workspace=None, stream=None):
    """Decode attention for q [B, Hq, D] over the paged cache; returns out [B, Hq, D]."""
    args, out, _ = _decode_args(q, k_cache, v_cache, block_tables, context_lens, scale, out, k_scale, v_scale,
                                partition_size, workspace, stream)
    _native.call("paged_attention_decode", *args)
    return out


def _decode_args(q, k_cache, v_cache, block_tables, context_lens, scale, out, k_scale, v_scale, partition_size,
                 workspace, stream):
    """Validated C arguments of paged_attention_decode, the output and the workspace."""
    B, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    if D2 != D or v_cache.shape != k_cache.shape:
        raise ValueError("paged_attention_decode: shape mismatch")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("paged_attention_decode: block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("paged_attention_decode: block_tables [B, max_blocks], context_lens [B]")
    if out is None:
        out = _output(stream, q.device, q.shape, q.dtype)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("paged_attention_decode: out must match q")
    _require_out(q.device, out)
    _require_cuda(q.device, q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
                  context_lens=context_lens, k_scale=k_scale, v_scale=v_scale, workspace=workspace)
    max_blocks = block_tables.shape[1]
    s = _stream(stream, q.device)
    if workspace is None:
        need = workspace_size(B, Hq, Hkv, D, max_blocks, bs, partition_size)
        if need:
            workspace = _workspace(q.device, stream, need)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), max_blocks, _ptr(context_lens), B, Hq, Hkv,
            bs, D, NB, float(scale), _ptr(out), _code(q), _code(k_cache), _ptr(k_scale), _ptr(v_scale),
            int(partition_size), _ptr(workspace), ws_bytes, s)
    return args, out, workspace


def paged_attention_decode_append(q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables, context_lens, scale,
                                  out=None, k_scale=None, v_scale=None, partition_size=PARTITION_AUTO, workspace=None,
                                  stream=None):
    """Append each sequence's new K/V row (k_new, v_new [B, Hkv, D] at slot_mapping int64 [B]) and decode, in one
    launch; context_lens count the new token.  Returns out [B, Hq, D]."""
    args, out, _ = _decode_append_args(q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables, context_lens,
                                       scale, out, k_scale, v_scale, partition_size, workspace, stream)
    _native.call("paged_attention_decode_append", *args)
    return out


def _decode_append_args(q, k_new, v_new, slot_mapping, k_cache, v_cache, block_tables, context_lens, scale, out,
                        k_scale, v_scale, partition_size, workspace, stream):
    """Validated C arguments of paged_attention_decode_append, the output and the workspace."""
    B, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    if D2 != D or v_cache.shape != k_cache.shape or k_new.shape != (B, Hkv, D) or v_new.shape != k_new.shape:
        raise ValueError("paged_attention_decode_append: shape mismatch")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (B,):
        raise ValueError("paged_attention_decode_append: slot_mapping must be int64 [num_seqs]")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("paged_attention_decode_append: block_tables and context_lens must be int32")
    if out is None:
        out = _output(stream, q.device, q.shape, q.dtype)
    _require_out(q.device, out)
    _require_cuda(q.device, q=q, k_new=k_new, v_new=v_new, slot_mapping=slot_mapping, k_cache=k_cache,
                  v_cache=v_cache, block_tables=block_tables, context_lens=context_lens, k_scale=k_scale,
                  v_scale=v_scale, workspace=workspace)
    max_blocks = block_tables.shape[1]
    s = _stream(stream, q.device)
    if workspace is None:
        need = workspace_size(B, Hq, Hkv, D, max_blocks, bs, partition_size)
        if need:
            workspace = _workspace(q.device, stream, need)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
            max_blocks, _ptr(context_lens), B, Hq, Hkv, bs, D, NB, float(scale), _ptr(out), _code(q),
            _code(k_cache), _ptr(k_scale), _ptr(v_scale), int(partition_size), _ptr(workspace), ws_bytes, s)
    return args, out, workspace


class DecodePlan:
    """One decode step for fixed tensors, validated and marshalled once.

    With k_new, v_new and slot_mapping it is paged_attention_decode_append,
    with k_scales and v_scales paged_attention_decode_scaled, else
    paged_attention_decode; the arguments mean the same.  run() issues
    the step with a single C call and returns `out`.  Between runs the
    tensors' contents may change (new queries, tables, lengths), their
    storage, shapes and types may not.  Every run goes on the stream given
    here (default: the current stream at construction).  Plans that may run
    at the same time need a workspace each (with k_scales and v_scales the
    default one is the plan's own)."""

    def __init__(self, q, k_cache, v_cache, block_tables, context_lens, scale, out=None, k_scale=None, v_scale=None,
                 partition_size=PARTITION_AUTO, workspace=None, stream=None, k_new=None, v_new=None,
                 slot_mapping=None, k_scales=None, v_scales=None):
        given = [t is not None for t in (k_new, v_new, slot_mapping)]
        if any(given) and not all(given):
            raise ValueError("DecodePlan: k_new, v_new and slot_mapping go together")
        if k_scales is not None or v_scales is not None:
            if any(given) or k_scale is not None or v_scale is not None:
                raise ValueError("DecodePlan: k_scales and v_scales go with neither an append nor k_scale, v_scale")
            self.func = "paged_attention_decode_scaled"
            self._args, self.out, ws = _decode_scaled_args(q, k_cache, v_cache, k_scales, v_scales, block_tables,
                                                           context_lens, scale, out, partition_size, workspace, stream,
                                                           own_workspace=True)
        elif all(given):
            self.func = "paged_attention_decode_append"
            self._args, self.out, ws = _decode_append_args(q, k_new, v_new, slot_mapping, k_cache, v_cache,
                                                           block_tables, context_lens, scale, out, k_scale, v_scale,
                                                           partition_size, workspace, stream)
        else:
            self.func = "paged_attention_decode"
            self._args, self.out, ws = _decode_args(q, k_cache, v_cache, block_tables, context_lens, scale, out,
                                                    k_scale, v_scale, partition_size, workspace, stream)
        # the plan holds its tensors so that their storage outlives it
        self._tensors = (q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale, ws, k_new, v_new,
                         slot_mapping, k_scales, v_scales)
        self._fn = _native.function(self.func)
        self._device = k_cache.device

    def run(self):
        if self._device.index == torch._C._cuda_getDevice():
            code = self._fn(*self._args)
        else:  # the library launches on the current device
            with torch.cuda.device(self._device):
                code = self._fn(*self._args)
        if code != 0:
            _native.check(self.func, code)
        return self.out


def quest_block_minmax(k_cache, block_tables, context_lens, kmeta=None, stream=None, meta_dtype=None):
    """Per-block channel min/max of the keys (QUEST metadata) for every block the sequences use;
    returns kmeta [num_blocks, Hkv, 2, D] in the queries' 16-bit type (meta_dtype: default the
    cache's type, bfloat16 for an E4M3 cache, whose metadata holds the unscaled code values)."""
    NB, Hkv, bs, D = k_cache.shape
    if meta_dtype is None:
        meta_dtype = kmeta.dtype if kmeta is not None else (
            torch.bfloat16 if _code(k_cache) == E4M3 else k_cache.dtype)
    if kmeta is None:
        kmeta = _output(stream, k_cache.device, (NB, Hkv, 2, D), meta_dtype, zero=True)
    if kmeta.dtype != meta_dtype:
        raise ValueError("quest_block_minmax: kmeta must be of meta_dtype")
    _require_cuda(k_cache.device, k_cache=k_cache, block_tables=block_tables, context_lens=context_lens, kmeta=kmeta)
    _native.call("quest_block_minmax", _ptr(k_cache), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
                 block_tables.shape[0], Hkv, bs, D, NB, _code(k_cache), _code(kmeta), _ptr(kmeta),
                 _stream(stream, k_cache.device))
    return kmeta


def quest_append_minmax(k_new, slot_mapping, kmeta, block_size, stream=None, k_scale=None):
    """Widen QUEST metadata with newly appended keys k_new [T, Hkv, D] at slot_mapping (int64 [T]).
    For an E4M3 cache pass its k_scale (device float32 [1]): each key enters as the append stores it."""
    T, Hkv, D = k_new.shape
    _require_cuda(k_new.device, k_new=k_new, slot_mapping=slot_mapping, kmeta=kmeta, k_scale=k_scale)
    _native.call("quest_append_minmax", _ptr(k_new), _ptr(slot_mapping), T, Hkv, block_size, D, kmeta.shape[0],
                 _code(k_new), E4M3 if k_scale is not None else _code(k_new), _ptr(k_scale), _ptr(kmeta),
                 _stream(stream, k_new.device))


def quest_select(q, kmeta, block_tables, context_lens, block_size, budget_blocks, sel_tables=None, sel_lens=None,
                 workspace=None, stream=None):
    """QUEST top-K blocks per (sequence, kv head); returns (sel_tables [B, Hkv, budget], sel_lens [B, Hkv])."""
    B, Hq, D = q.shape
    NB, Hkv = kmeta.shape[0], kmeta.shape[1]
    if sel_tables is None:
        sel_tables = _output(stream, q.device, (B, Hkv, budget_blocks), torch.int32)
    if sel_lens is None:
        sel_lens = _output(stream, q.device, (B, Hkv), torch.int32)
    _require_cuda(q.device, q=q, kmeta=kmeta, block_tables=block_tables, context_lens=context_lens,
                  sel_tables=sel_tables, sel_lens=sel_lens, workspace=workspace)
    s = _stream(stream, q.device)
    need = int(_native.lib().quest_workspace_size(B, Hkv, block_tables.shape[1]))
    if workspace is None:
        workspace = _workspace(q.device, stream, need, kind=1)  # separate from the decode workspace
    _native.call("quest_select", _ptr(q), _ptr(kmeta), _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
                 B, Hq, Hkv, block_size, D, NB, _code(q), int(budget_blocks), _ptr(sel_tables), _ptr(sel_lens),
                 _ptr(workspace), workspace.numel() * workspace.element_size(), s)
    return sel_tables, sel_lens


def paged_attention_decode_sparse(q, k_cache, v_cache, sel_tables, sel_lens, scale, out=None, k_scale=None,
                                  v_scale=None, partition_size=PARTITION_AUTO, workspace=None, stream=None):
    """Decode over per-(sequence, kv head) block lists sel_tables [B, Hkv, max_sel], sel_lens [B, Hkv]."""
    B, Hq, D = q.shape
    NB, Hkv, bs, _ = k_cache.shape
    if out is None:
        out = _output(stream, q.device, q.shape, q.dtype)
    _require_out(q.device, out)
    _require_cuda(q.device, q=q, k_cache=k_cache, v_cache=v_cache, sel_tables=sel_tables, sel_lens=sel_lens,
                  k_scale=k_scale, v_scale=v_scale, workspace=workspace)
    max_sel = sel_tables.shape[2]
    s = _stream(stream, q.device)
    need = workspace_size(B, Hq, Hkv, D, max_sel, bs, partition_size)
    if need and workspace is None:
        workspace = _workspace(q.device, stream, need)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _native.call("paged_attention_decode_sparse", _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(sel_tables), max_sel,
                 _ptr(sel_lens), B, Hq, Hkv, bs, D, NB, float(scale), _ptr(out), _code(q), _code(k_cache),
                 _ptr(k_scale), _ptr(v_scale), int(partition_size), _ptr(workspace), ws_bytes, s)
    return out


_E4M3_TYPES = (torch.uint8, torch.float8_e4m3fn)


_contiguous, _device_of, _pointer = torch.Tensor.is_contiguous, torch.Tensor.get_device, torch.Tensor.data_ptr


def _pointers(name, device, names, *tensors):
    """Data pointers of tensors that have to be contiguous and on `device`; `names` are theirs, space-separated.
    (Mapped builtins: these checks are most of what a small call costs on the host.)"""
    if not all(map(_contiguous, tensors)) or set(map(_device_of, tensors)) != {device.index}:
        for what, t in zip(names.split(), tensors):
            if t.get_device() != device.index or not t.is_contiguous():
                raise ValueError(f"{name}: {what} must be a contiguous CUDA tensor on {device}")
    return map(_pointer, tensors)


def _require_scales(name, k_cache, v_cache, k_scales, v_scales):
    """Checks of a block-scaled cache: E4M3 codes and float32 scales [num_blocks, num_kv_heads]."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError(f"{name}: k_cache and v_cache must be [num_blocks, num_kv_heads, block_size, head_dim]")
    if k_cache.dtype not in _E4M3_TYPES or v_cache.dtype not in _E4M3_TYPES:
        raise ValueError(f"{name}: a block-scaled cache holds E4M3 codes (uint8 or float8_e4m3fn)")
    if k_scales is None or v_scales is None:
        raise ValueError(f"{name}: k_scales and v_scales go together")
    sshape = k_scales.shape
    if (k_scales.dtype is not torch.float32 or v_scales.dtype is not torch.float32 or v_scales.shape != sshape
            or len(sshape) != 2 or sshape[0] != shape[0] or sshape[1] != shape[1]):
        raise ValueError(f"{name}: k_scales and v_scales must be float32 [num_blocks, num_kv_heads]")
    return shape


def _rows(name, what, t, index, shape):
    """Token stride, in elements, of t [T, heads, head_dim] (its shape is given) whose rows are contiguous."""
    T, H, D = shape
    st = t.stride()
    if (st[2] != 1 and D > 1) or (st[1] != D and H > 1):
        raise ValueError(f"{name}: {what} must have contiguous rows [heads, head_dim]")
    if t.get_device() != index:
        raise ValueError(f"{name}: {what} must be a CUDA tensor on cuda:{index}")
    return st[0] if T > 1 else H * D


def _call_on(device, func, *args):
    """The C call `func` with `device` current (it launches on the current device)."""
    if device.index == torch._C._cuda_getDevice():
        _native.call(func, *args)
    else:
        with torch.cuda.device(device):
            _native.call(func, *args)


class ExtendedTables(NamedTuple):
    """What paged_extend_tables writes (block_tables is updated in place)."""
    slot_mapping: torch.Tensor
    positions: torch.Tensor
    seq_starts: torch.Tensor
    block_starts: torch.Tensor
    context_lens: torch.Tensor
    free_head: torch.Tensor


def paged_extend_tables(block_tables, context_lens, new_lens, free_blocks, free_head, block_size, num_blocks,
                        num_tokens=None, slot_mapping=None, positions=None, seq_starts=None, block_starts=None,
                        context_lens_out=None, free_head_out=None, stream=None) -> ExtendedTables:
    """Blocks, slots and positions of a step's tokens from request lengths, on the GPU.

    block_tables int32 [B, max_blocks] (new entries are written), context_lens and new_lens int32 [B],
    free_blocks int32 [F] with free_head int32 [1] the first one not taken, num_blocks the pool's size.  num_tokens
    rows of slots and positions come out, the step's tokens first, -1 behind them (default: the given slot_mapping's
    rows).  context_lens_out and free_head_out may be context_lens and free_head: a captured step can then be
    replayed.  All or nothing on the device: a step that does not fit sets DEV_NO_SPACE or DEV_BAD_CONTEXT_LEN
    and takes nothing."""
    name = "paged_extend_tables"
    device = block_tables.device
    if not block_tables.is_cuda:
        raise ValueError(f"{name}: block_tables must be a CUDA tensor")
    if block_tables.dim() != 2:
        raise ValueError(f"{name}: block_tables must be [B, max_blocks]")
    B, max_blocks = block_tables.shape
    if context_lens.shape != (B,) or new_lens.shape != (B,) or free_blocks.dim() != 1 or free_head.shape != (1,):
        raise ValueError(f"{name}: context_lens and new_lens [B], free_blocks [F], free_head [1]")
    if num_tokens is None:
        if slot_mapping is None:
            raise ValueError(f"{name}: num_tokens (rows of slots to make) or slot_mapping is needed")
        num_tokens = slot_mapping.shape[0]
    i32 = torch.int32

    def output(t, n, dtype, what):
        if t is None:
            return _output(stream, device, (n,), dtype)
        if t.dtype is not dtype or t.shape != (n,):
            raise ValueError(f"{name}: {what} must be {dtype} [{n}]")
        return t

    slot_mapping = output(slot_mapping, num_tokens, torch.int64, "slot_mapping")
    positions = output(positions, num_tokens, i32, "positions")
    seq_starts = output(seq_starts, B + 1, i32, "seq_starts")
    block_starts = output(block_starts, B + 1, i32, "block_starts")
    lens_out = output(context_lens_out, B, i32, "context_lens_out")
    head_out = output(free_head_out, 1, i32, "free_head_out")
    if not (block_tables.dtype is i32 and context_lens.dtype is i32 and new_lens.dtype is i32
            and free_blocks.dtype is i32 and free_head.dtype is i32):
        raise ValueError(f"{name}: block_tables, context_lens, new_lens, free_blocks and free_head must be int32")
    tables, lens, new, free, head, *outs = _pointers(
        name, device, "block_tables context_lens new_lens free_blocks free_head slot_mapping positions seq_starts "
        "block_starts context_lens_out free_head_out", block_tables, context_lens, new_lens, free_blocks, free_head,
        slot_mapping, positions, seq_starts, block_starts, lens_out, head_out)
    _call_on(device, name, tables, max_blocks, lens, new, B, int(block_size), free, free_blocks.shape[0], head,
             int(num_blocks), num_tokens, *outs, _stream(stream, device))
    return ExtendedTables(slot_mapping, positions, seq_starts, block_starts, lens_out, head_out)


def rope_inv_freq(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_context=None, slow_turns=1.0,
                  fast_turns=32.0, device="cuda"):
    """Inverse frequencies float32 [rotary_dim / 2] for paged_rope_append, and the attention factor to pass with them.

    scaling stretches a model trained on original_context tokens to factor times as many:
      None      base ** (-2i / rotary_dim)
      "linear"  every frequency divided by factor (positions interpolated)
      "ntk"     the base raised so that the slowest pair is divided by factor and the fastest is kept
      "yarn"    pairs that turn fewer than slow_turns times over original_context are divided by factor, those that
                turn more than fast_turns times are kept, a linear ramp (over the turns' logarithm, that is over the
                pair's index) between; attention factor 0.1 ln(factor) + 1
      "smooth"  the same bands with a ramp linear in the turns; attention factor 1"""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rope_inv_freq: rotary_dim must be even and positive")
    if scaling not in (None, "linear", "ntk", "yarn", "smooth"):
        raise ValueError(f"rope_inv_freq: unknown scaling {scaling!r}")
    if not (factor >= 1.0 and math.isfinite(factor) and base > 1.0 and math.isfinite(base)):
        raise ValueError("rope_inv_freq: factor must be at least 1 and base above 1")
    half = rotary_dim // 2
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-np.arange(half, dtype=np.float64) * 2.0 / rotary_dim)
    attention = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling in ("yarn", "smooth"):
        if not original_context or not 0 < slow_turns < fast_turns:
            raise ValueError(f"rope_inv_freq: {scaling!r} needs original_context and 0 < slow_turns < fast_turns")
        turns = original_context * f / (2.0 * math.pi)
        if scaling == "yarn":
            ramp = np.log(turns / slow_turns) / math.log(fast_turns / slow_turns)
            attention = 0.1 * math.log(factor) + 1.0
        else:
            ramp = (turns - slow_turns) / (fast_turns - slow_turns)
        keep = np.clip(ramp, 0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return torch.from_numpy(f.astype(np.float32)).to(device), attention


def paged_rope_append(q, k, v, positions, slot_mapping, inv_freq, k_cache, v_cache, interleaved=False,
                      attention_factor=1.0, q_out=None, k_scale=None, v_scale=None, k_scales=None, v_scales=None,
                      stream=None):
    """Rotate q [T, Hq, D] and k [T, Hkv, D] at positions int32 [T] and append the rotated keys and the values at
    slot_mapping int64 [T], in one call; returns the rotated queries (q_out, new by default, may be q).

    The first 2 * len(inv_freq) channels turn, paired (i, i + half) or interleaved (2i, 2i + 1).  q, k, v may be
    parts of one projection's output (rows contiguous, token strides of their own).  The cache is of q's type, or
    E4M3 with k_scale, v_scale (one each) or k_scales, v_scales (block-scaled: tokens of one block must be neighbours
    in the call, but for up to 255 skipped ones, the one at offset 0 first).  A negative position marks a padding row,
    a negative slot a token that is not stored.  q may be None (keys alone)."""
    name = "paged_rope_append"
    kshape, cshape = k.shape, k_cache.shape
    device = k.device
    if not k.is_cuda:
        raise ValueError(f"{name}: k must be a CUDA tensor")
    if len(kshape) != 3 or len(cshape) != 4 or v_cache.shape != cshape or v.shape != kshape:
        raise ValueError(f"{name}: shape mismatch")
    T, Hkv, D = kshape
    NB, Hkv2, bs, D2 = cshape
    if Hkv2 != Hkv or D2 != D:
        raise ValueError(f"{name}: shape mismatch")
    if positions.dtype != torch.int32 or positions.shape != (T,):
        raise ValueError(f"{name}: positions must be int32 [num_tokens]")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,):
        raise ValueError(f"{name}: slot_mapping must be int64 [num_tokens]")
    if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1:
        raise ValueError(f"{name}: inv_freq must be float32 [rotary_dim / 2]")
    if v.dtype != k.dtype or v_cache.dtype != k_cache.dtype:
        raise ValueError(f"{name}: k and v, and the two caches, must have one type")
    if k_scales is not None or v_scales is not None:
        if k_scale is not None or v_scale is not None:
            raise ValueError(f"{name}: k_scale, v_scale or k_scales, v_scales, not both")
        _require_scales(name, k_cache, v_cache, k_scales, v_scales)
        s1 = s2 = None
        kc, vc, pos, slots, freq, sb1, sb2 = _pointers(
            name, device, "k_cache v_cache positions slot_mapping inv_freq k_scales v_scales", k_cache, v_cache,
            positions, slot_mapping, inv_freq, k_scales, v_scales)
    else:
        sb1 = sb2 = None
        for t in (k_scale, v_scale):
            if t is not None and (t.dtype is not torch.float32 or t.numel() != 1):
                raise ValueError(f"{name}: k_scale and v_scale must be float32 with one element")
        kc, vc, pos, slots, freq = _pointers(name, device, "k_cache v_cache positions slot_mapping inv_freq", k_cache,
                                             v_cache, positions, slot_mapping, inv_freq)
        s1, s2 = (None if t is None else next(_pointers(name, device, what, t))
                  for what, t in (("k_scale", k_scale), ("v_scale", v_scale)))
    Hq = qs = os = 0
    index = device.index
    if q is not None:
        qshape = q.shape
        if len(qshape) != 3 or qshape[0] != T or qshape[2] != D or q.dtype != k.dtype:
            raise ValueError(f"{name}: q must be [num_tokens, num_q_heads, head_dim] of k's type")
        Hq = qshape[1]
        if q_out is None:
            q_out = _output(stream, device, qshape, q.dtype)
        elif q_out.shape != qshape or q_out.dtype != q.dtype:
            raise ValueError(f"{name}: q_out must match q")
        qs, os = _rows(name, "q", q, index, qshape), _rows(name, "q_out", q_out, index, qshape)
    elif q_out is not None:
        raise ValueError(f"{name}: q_out without q")
    ks, vs = _rows(name, "k", k, index, kshape), _rows(name, "v", v, index, kshape)
    _call_on(device, name, _ptr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs, pos, slots, T, freq, 2 * inv_freq.shape[0],
             1 if interleaved else 0, attention_factor, _ptr(q_out), os, kc, vc, NB, Hq, Hkv, bs, D, _code(k),
             _code(k_cache), s1, s2, sb1, sb2, _stream(stream, device))
    return q_out


def paged_kv_append_scaled(k, v, slot_mapping, k_cache, v_cache, k_scales, v_scales, stream=None):
    """Quantise k, v [T, Hkv, D] into their slots (int64 [T], negative = skip) of a block-scaled E4M3 cache.

    The scale of a (block, kv head) is the least power of two that holds its largest element; a later token that
    needs a larger one moves the block's codes along.  A token at offset 0 starts its block afresh.  Tokens of one
    block must be neighbours in the call, but for up to 255 skipped ones, the one at offset 0 first."""
    name = "paged_kv_append_scaled"
    kshape = k.shape
    device = k_cache.device
    NB, Hkv2, bs, D2 = _require_scales(name, k_cache, v_cache, k_scales, v_scales)
    if len(kshape) != 3 or v.shape != kshape or v.dtype != k.dtype or Hkv2 != kshape[1] or D2 != kshape[2]:
        raise ValueError(f"{name}: shape or type mismatch")
    T, Hkv, D = kshape
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (T,):
        raise ValueError(f"{name}: slot_mapping must be int64 [num_tokens]")
    ks, vs = _rows(name, "k", k, device.index, kshape), _rows(name, "v", v, device.index, kshape)
    slots, kc, vc, s1, s2 = _pointers(name, device, "slot_mapping k_cache v_cache k_scales v_scales", slot_mapping,
                                      k_cache, v_cache, k_scales, v_scales)
    _call_on(device, name, k.data_ptr(), ks, v.data_ptr(), vs, slots, T, kc, vc, s1, s2, NB, Hkv, bs, D, _code(k),
             _stream(stream, device))


def paged_attention_decode_scaled(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale, out=None,
                                  partition_size=PARTITION_AUTO, workspace=None, stream=None):
    """Decode attention for q [B, Hq, D] over a block-scaled E4M3 cache; returns out [B, Hq, D].  A context length
    of 0 (a padding row) gives zeros."""
    args, out, _ = _decode_scaled_args(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale, out,
                                       partition_size, workspace, stream)
    _call_on(q.device, "paged_attention_decode_scaled", *args)
    return out


@functools.lru_cache(maxsize=1024)
def _scaled_workspace_size(*sizes):  # a function of the sizes alone
    return workspace_size(*sizes, True)


def _decode_scaled_args(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale, out,
                        partition_size, workspace, stream, own_workspace=False):
    """Validated C arguments of paged_attention_decode_scaled, the output and the workspace (own_workspace: not the
    stream's reusable one, so that graphs of two plans may run at once)."""
    name = "paged_attention_decode_scaled"
    NB, Hkv, bs, D = _require_scales(name, k_cache, v_cache, k_scales, v_scales)
    qshape = q.shape
    if len(qshape) != 3 or qshape[2] != D:
        raise ValueError(f"{name}: shape mismatch")
    B, Hq, _ = qshape
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError(f"{name}: block_tables and context_lens must be int32")
    tshape = block_tables.shape
    if len(tshape) != 2 or tshape[0] != B or context_lens.shape != (B,):
        raise ValueError(f"{name}: block_tables [B, max_blocks], context_lens [B]")
    device = k_cache.device
    if out is None:
        out = _output(stream, device, qshape, q.dtype)
    elif out.shape != qshape or out.dtype != q.dtype:
        raise ValueError(f"{name}: out must match q")
    if not q.is_cuda:
        raise ValueError(f"{name}: q must be a CUDA tensor")
    _require_out(device, out)
    s = _stream(stream, device)
    if workspace is None:
        need = _scaled_workspace_size(B, Hq, Hkv, D, tshape[1], bs, partition_size)
        need = max(need, 1)  # (0: an argument that the library refuses)
        workspace = (_output(stream, device, (need,), torch.uint8) if own_workspace
                     else _workspace(device, stream, need))
    qp, kc, vc, s1, s2, tables, lens, ws = _pointers(
        name, device, "q k_cache v_cache k_scales v_scales block_tables context_lens workspace", q, k_cache, v_cache,
        k_scales, v_scales, block_tables, context_lens, workspace)
    args = (qp, kc, vc, s1, s2, tables, tshape[1], lens, B, Hq, Hkv, bs, D, NB, scale, out.data_ptr(), _code(q),
            partition_size, ws, workspace.numel() * workspace.element_size(), s)
    return args, out, workspace


def paged_block_copy(k_cache, v_cache, src_dst_pairs, stream=None, k_scales=None, v_scales=None):
    """Copy whole blocks (K and V) for each (src, dst) row of int32 [P, 2], with their scales for a block-scaled
    cache (k_scales, v_scales float32 [num_blocks, num_kv_heads])."""
    if src_dst_pairs.dtype != torch.int32 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("paged_block_copy: src_dst_pairs must be int32 [P, 2]")
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("paged_block_copy: k_cache and v_cache must match")
    _require_cuda(k_cache.device, k_cache=k_cache, v_cache=v_cache, src_dst_pairs=src_dst_pairs)
    block_bytes = k_cache[0].numel() * k_cache.element_size()
    if k_scales is not None or v_scales is not None:
        _require_scales("paged_block_copy", k_cache, v_cache, k_scales, v_scales)
        _require_cuda(k_cache.device, k_scales=k_scales, v_scales=v_scales)
        _call_on(k_cache.device, "paged_block_copy_scaled", _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
                 _ptr(v_scales), _ptr(src_dst_pairs), src_dst_pairs.shape[0], k_cache.shape[0], k_cache.shape[1],
                 block_bytes, _stream(stream, k_cache.device))
        return
    _native.call("paged_block_copy", _ptr(k_cache), _ptr(v_cache), _ptr(src_dst_pairs), src_dst_pairs.shape[0],
                 k_cache.shape[0], block_bytes, _stream(stream, k_cache.device))


def paged_block_swap(k_cache, v_cache, block_ids, staging, direction, stream=None, k_scales=None, v_scales=None,
                     scale_staging=None):
    """Copy whole blocks between the pools and staging [n, 2, block_bytes] (uint8,
    pinned host or device).  direction: SWAP_OUT (pools -> staging) or SWAP_IN.
    A block-scaled cache moves its scales along, between k_scales, v_scales and
    scale_staging (float32 [n, 2, num_kv_heads], pinned host or device)."""
    if block_ids.dtype != torch.int32 or block_ids.dim() != 1:
        raise ValueError("paged_block_swap: block_ids must be int32 [n]")
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("paged_block_swap: k_cache and v_cache must match")
    _require_cuda(k_cache.device, k_cache=k_cache, v_cache=v_cache, block_ids=block_ids)
    block_bytes = k_cache[0].numel() * k_cache.element_size()
    if staging.numel() * staging.element_size() < block_ids.numel() * 2 * block_bytes or not staging.is_contiguous():
        raise ValueError("paged_block_swap: staging must be contiguous with room for [n, 2, block_bytes]")
    if not staging.is_cuda and not staging.is_pinned():
        raise ValueError("paged_block_swap: host staging must be pinned memory")
    if k_scales is not None or v_scales is not None or scale_staging is not None:
        _require_scales("paged_block_swap", k_cache, v_cache, k_scales, v_scales)
        _require_cuda(k_cache.device, k_scales=k_scales, v_scales=v_scales)
        if (scale_staging is None or scale_staging.dtype != torch.float32 or not scale_staging.is_contiguous()
                or scale_staging.numel() < block_ids.numel() * 2 * k_cache.shape[1]):
            raise ValueError("paged_block_swap: scale_staging must be contiguous float32 [n, 2, num_kv_heads]")
        if not scale_staging.is_cuda and not scale_staging.is_pinned():
            raise ValueError("paged_block_swap: host scale_staging must be pinned memory")
    _native.call("paged_block_swap", _ptr(k_cache), _ptr(v_cache), _ptr(block_ids), block_ids.numel(),
                 k_cache.shape[0], block_bytes, _ptr(staging), int(direction), _stream(stream, k_cache.device))
    if k_scales is not None:
        _call_on(k_cache.device, "paged_block_scales_swap", _ptr(k_scales), _ptr(v_scales), _ptr(block_ids),
                 block_ids.numel(), k_cache.shape[0], k_cache.shape[1], _ptr(scale_staging), int(direction),
                 _stream(stream, k_cache.device))


def device_error(reset: bool = True, stream=None, device=None) -> int:
    """Read (and by default clear) the current device's kernel error bits."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    bits = ctypes.c_int(0)
    _native.call("pkv_device_error", ctypes.byref(bits), int(reset), _stream(stream, device))
    return bits.value


def selftest_wait_timeout(limit_us: int = 1000, stream=None, device=None) -> None:
    """Run the bounded-wait check kernel (a wait on a barrier nothing arrives
    at, given up after limit_us); read the outcome with device_error()."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    _native.call("pkv_selftest_wait_timeout", int(limit_us), _stream(stream, device))


class BlockManager:
    """Host-side block allocator (C++ in libpagedkv.so): FIFO free list,
    per-block reference counts, copy-on-write of a shared last block."""

    def __init__(self, num_blocks: int, block_size: int, free_list=None):
        lib = _native.lib()
        fl = None if free_list is None else np.ascontiguousarray(free_list, dtype=np.int32)
        self._h = lib.pkv_bm_create(num_blocks, block_size,
                                    None if fl is None else fl.ctypes.data_as(ctypes.c_void_p),
                                    0 if fl is None else len(fl))
        if not self._h:
            raise PagedKVError("pkv_bm_create", 1, lib.pkv_last_error().decode())
        self.num_blocks = num_blocks
        self.block_size = block_size

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _native.lib().pkv_bm_destroy(h)
            self._h = None

    def _check(self, func, code):
        if code == ERR_NO_SPACE:
            raise OutOfBlocks(func, code, _native.lib().pkv_last_error().decode())
        _native.check(func, code)

    def add_sequence(self, seq_id: int, num_tokens: int) -> None:
        self._check("pkv_bm_add_sequence", _native.lib().pkv_bm_add_sequence(self._h, int(seq_id), int(num_tokens)))

    def add_sequence_cached(self, seq_id: int, tokens) -> int:
        """Register a prompt by token ids, sharing the longest cached prefix of
        full blocks; returns how many leading tokens are already in the pool."""
        toks = np.ascontiguousarray(tokens, dtype=np.int32)
        cached = ctypes.c_int(0)
        self._check("pkv_bm_add_sequence_cached", _native.lib().pkv_bm_add_sequence_cached(
            self._h, int(seq_id), toks.ctypes.data_as(ctypes.c_void_p), len(toks), ctypes.byref(cached)))
        return cached.value

    def swap_out(self, seq_id: int) -> np.ndarray:
        """Release a sequence's blocks, keeping it as swapped out; returns the
        blocks (logical order) whose contents must be staged out first."""
        n = max(self.num_seq_blocks(seq_id), 0)
        out = np.empty(max(n, 1), np.int32)
        cnt = ctypes.c_int(0)
        self._check("pkv_bm_swap_out", _native.lib().pkv_bm_swap_out(
            self._h, int(seq_id), out.ctypes.data_as(ctypes.c_void_p), len(out), ctypes.byref(cnt)))
        return out[: cnt.value].copy()

    def swap_in(self, seq_id: int, max_blocks: int) -> np.ndarray:
        """Give a swapped-out sequence fresh blocks; returns them (logical order)."""
        out = np.empty(max(max_blocks, 1), np.int32)
        cnt = ctypes.c_int(0)
        self._check("pkv_bm_swap_in", _native.lib().pkv_bm_swap_in(
            self._h, int(seq_id), out.ctypes.data_as(ctypes.c_void_p), len(out), ctypes.byref(cnt)))
        return out[: cnt.value].copy()

    def swap_out_group(self, seq_ids) -> np.ndarray:
        """Swap out sequences together (e.g. one prompt's samples): returns their
        distinct blocks, first-use order, each to be staged once."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        cap = max(sum(max(self.num_seq_blocks(s), 0) for s in ids), 1)
        out = np.empty(cap, np.int32)
        cnt = ctypes.c_int(0)
        self._check("pkv_bm_swap_out_group", _native.lib().pkv_bm_swap_out_group(
            self._h, ids.ctypes.data_as(ctypes.c_void_p), len(ids), out.ctypes.data_as(ctypes.c_void_p), cap,
            ctypes.byref(cnt)))
        return out[: cnt.value].copy()

    def swap_in_group(self, seq_ids, max_blocks: int) -> np.ndarray:
        """Bring a group swapped out together back: one fresh block per staged
        entry (returned in staging order); shared blocks are shared again."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        out = np.empty(max(max_blocks, 1), np.int32)
        cnt = ctypes.c_int(0)
        self._check("pkv_bm_swap_in_group", _native.lib().pkv_bm_swap_in_group(
            self._h, ids.ctypes.data_as(ctypes.c_void_p), len(ids), out.ctypes.data_as(ctypes.c_void_p), len(out),
            ctypes.byref(cnt)))
        return out[: cnt.value].copy()

    @property
    def num_cached_blocks(self) -> int:
        return int(_native.lib().pkv_bm_num_cached_blocks(self._h))

    def append_slots(self, seq_ids):
        """Reserve the next slot of each sequence; returns (slots int64 [n], cow_pairs int32 [k, 2])."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        n = len(ids)
        slots = np.empty(n, np.int64)
        pairs = np.empty((max(n, 1), 2), np.int32)
        npairs = ctypes.c_int(0)
        self._check("pkv_bm_append_slots", _native.lib().pkv_bm_append_slots(
            self._h, ids.ctypes.data_as(ctypes.c_void_p), n, slots.ctypes.data_as(ctypes.c_void_p),
            pairs.ctypes.data_as(ctypes.c_void_p), ctypes.byref(npairs)))
        return slots, pairs[: npairs.value].copy()

    def append_tokens(self, seq_ids, token_ids):
        """append_slots with each new token's id: a token that fills its block
        registers the block in the prefix cache (sequences added by
        add_sequence_cached).  Returns (slots int64 [n], cow_pairs int32 [k, 2])."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        toks = np.ascontiguousarray(token_ids, dtype=np.int32)
        n = len(ids)
        if len(toks) != n:
            raise ValueError("append_tokens: one token id per sequence id")
        slots = np.empty(n, np.int64)
        pairs = np.empty((max(n, 1), 2), np.int32)
        npairs = ctypes.c_int(0)
        self._check("pkv_bm_append_tokens", _native.lib().pkv_bm_append_tokens(
            self._h, ids.ctypes.data_as(ctypes.c_void_p), toks.ctypes.data_as(ctypes.c_void_p), n,
            slots.ctypes.data_as(ctypes.c_void_p), pairs.ctypes.data_as(ctypes.c_void_p), ctypes.byref(npairs)))
        return slots, pairs[: npairs.value].copy()

    def fork(self, parent_id: int, child_id: int) -> None:
        self._check("pkv_bm_fork", _native.lib().pkv_bm_fork(self._h, int(parent_id), int(child_id)))

    def free_sequence(self, seq_id: int) -> None:
        self._check("pkv_bm_free_sequence", _native.lib().pkv_bm_free_sequence(self._h, int(seq_id)))

    def tables(self, seq_ids, max_blocks_per_seq: int | None = None, pad: int = 0):
        """Block tables int32 [n, max_blocks_per_seq] (pad-filled) and context lengths int32 [n]."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        if max_blocks_per_seq is None:
            max_blocks_per_seq = max([self.num_seq_blocks(s) for s in ids] + [1])
        t = np.empty((len(ids), max_blocks_per_seq), np.int32)
        lens = np.empty(len(ids), np.int32)
        self._check("pkv_bm_get_tables", _native.lib().pkv_bm_get_tables(
            self._h, ids.ctypes.data_as(ctypes.c_void_p), len(ids), t.ctypes.data_as(ctypes.c_void_p),
            max_blocks_per_seq, pad, lens.ctypes.data_as(ctypes.c_void_p)))
        return t, lens

    @property
    def num_free(self) -> int:
        return int(_native.lib().pkv_bm_num_free(self._h))

    def ref_count(self, block: int) -> int:
        return int(_native.lib().pkv_bm_ref_count(self._h, int(block)))

    def context_len(self, seq_id: int) -> int:
        return int(_native.lib().pkv_bm_context_len(self._h, int(seq_id)))

    def num_seq_blocks(self, seq_id: int) -> int:
        return int(_native.lib().pkv_bm_num_seq_blocks(self._h, int(seq_id)))

    def free_list(self) -> np.ndarray:
        n = int(_native.lib().pkv_bm_free_list(self._h, None, 0))
        out = np.empty(n, np.int32)
        _native.lib().pkv_bm_free_list(self._h, out.ctypes.data_as(ctypes.c_void_p), n)
        return out
