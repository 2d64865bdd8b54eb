"""PagedKVCache: one layer's paged K/V pools plus the host block manager.

A thin driver around the C ABI for callers that do not want to handle slot
mappings and copy pairs themselves.  Per decode step:

    slots, pairs = block_manager.append_slots(seq_ids)   # host (C++)
    paged_block_copy(pairs)                              # copy-on-write first
    paged_kv_append(k, v, slots)                         # then write the token
    paged_attention_decode(q, tables, lens)              # attend

Copies run before the append on the same stream: the diverging writer's new
block must hold the old tokens before its own token lands in it (iThome "how
to store the KV cache", section "Copy-on-Write").

With block_scales=True the pools hold E4M3 codes with one scale for each block
and kv head (k_scales, v_scales), kept by the scaled append, the copies and the
scaled decode.  rope_append rotates queries and keys on the way in.
"""
from __future__ import annotations

import numpy as np
import torch

from . import (PARTITION_AUTO, BlockManager, _torch_stream, paged_attention_decode, paged_attention_decode_scaled,
               paged_block_copy, paged_kv_append, paged_kv_append_scaled, paged_rope_append)


class PagedKVCache:
    def __init__(self, num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int,
                 dtype=torch.bfloat16, device="cuda", free_list=None, k_cache=None, v_cache=None,
                 k_scale=None, v_scale=None, block_scales=False, k_scales=None, v_scales=None):
        block_scales = block_scales or k_scales is not None or v_scales is not None
        if block_scales:
            if k_scale is not None or v_scale is not None:
                raise ValueError("PagedKVCache: k_scale, v_scale or block scales, not both")
            if (k_scales is None) != (v_scales is None):
                raise ValueError("PagedKVCache: k_scales and v_scales go together")
            dtype = torch.uint8
        self.num_blocks, self.num_kv_heads = num_blocks, num_kv_heads
        self.block_size, self.head_dim = block_size, head_dim
        self.device = torch.device(device)
        shape = (num_blocks, num_kv_heads, block_size, head_dim)
        self.k_cache = k_cache if k_cache is not None else torch.zeros(shape, dtype=dtype, device=self.device)
        self.v_cache = v_cache if v_cache is not None else torch.zeros(shape, dtype=dtype, device=self.device)
        self.k_scale, self.v_scale = k_scale, v_scale
        if block_scales:
            zeros = lambda: torch.zeros(num_blocks, num_kv_heads, dtype=torch.float32, device=self.device)  # noqa: E731
            k_scales = k_scales if k_scales is not None else zeros()
            v_scales = v_scales if v_scales is not None else zeros()
        self.k_scales, self.v_scales = k_scales, v_scales
        self.blocks = BlockManager(num_blocks, block_size, free_list=free_list)

    # -- host-side bookkeeping -------------------------------------------------
    def add_sequence(self, seq_id: int, num_tokens: int) -> None:
        """Allocate blocks for a request whose first num_tokens are already in the pool."""
        self.blocks.add_sequence(seq_id, num_tokens)

    def fork(self, parent_id: int, child_id: int) -> None:
        self.blocks.fork(parent_id, child_id)

    def free(self, seq_id: int) -> None:
        self.blocks.free_sequence(seq_id)

    def tables(self, seq_ids, max_blocks_per_seq=None):
        return tuple(self._upload(a, None) for a in self.blocks.tables(seq_ids, max_blocks_per_seq))

    def _upload(self, array, stream) -> torch.Tensor:
        """A device copy of a host array, which has arrived when this returns.  It belongs to the current stream;
        where a step on another one reads it, it is not handed out again before that step is done with it."""
        t = torch.from_numpy(array).to(self.device)
        if stream is not None:
            t.record_stream(_torch_stream(stream, self.device))
        return t

    # -- device steps ------------------------------------------------------------
    def append(self, seq_ids, k: torch.Tensor, v: torch.Tensor, stream=None):
        """Write one new token per sequence (k, v: [n, Hkv, D]); returns (slots, cow pairs) on the host."""
        slots, pairs = self._reserve(seq_ids, stream)
        d_slots = self._upload(slots, stream)
        if self.k_scales is not None:
            paged_kv_append_scaled(k, v, d_slots, self.k_cache, self.v_cache, self.k_scales, self.v_scales,
                                   stream=stream)
        else:
            paged_kv_append(k, v, d_slots, self.k_cache, self.v_cache, self.k_scale, self.v_scale, stream=stream)
        return slots, pairs

    def rope_append(self, seq_ids, q, k, v, inv_freq, interleaved=False, attention_factor=1.0, q_out=None, stream=None):
        """append with rotary positions: rotate q [n, Hq, D] and k at each sequence's newest position and write k, v;
        returns the rotated queries."""
        slots, _ = self._reserve(seq_ids, stream)
        positions = np.asarray([self.blocks.context_len(s) - 1 for s in np.asarray(seq_ids)], np.int32)
        return paged_rope_append(q, k, v, self._upload(positions, stream), self._upload(slots, stream), inv_freq,
                                 self.k_cache, self.v_cache, interleaved=interleaved,
                                 attention_factor=attention_factor, q_out=q_out, k_scale=self.k_scale,
                                 v_scale=self.v_scale, k_scales=self.k_scales, v_scales=self.v_scales, stream=stream)

    def _reserve(self, seq_ids, stream):
        """Slots of one new token per sequence; the copy-on-write copies run on the stream."""
        slots, pairs = self.blocks.append_slots(seq_ids)
        if len(pairs):
            paged_block_copy(self.k_cache, self.v_cache, self._upload(pairs, stream), stream=stream,
                             k_scales=self.k_scales, v_scales=self.v_scales)
        return slots, pairs

    def decode(self, seq_ids, q: torch.Tensor, scale: float, out=None, partition_size=PARTITION_AUTO,
               max_blocks_per_seq=None, stream=None):
        tables, lens = (self._upload(a, stream) for a in self.blocks.tables(seq_ids, max_blocks_per_seq))
        if self.k_scales is not None:
            return paged_attention_decode_scaled(q, self.k_cache, self.v_cache, self.k_scales, self.v_scales, tables,
                                                 lens, scale, out=out, partition_size=partition_size, stream=stream)
        return paged_attention_decode(q, self.k_cache, self.v_cache, tables, lens, scale, out=out,
                                      k_scale=self.k_scale, v_scale=self.v_scale,
                                      partition_size=partition_size, stream=stream)

    def unused_slots(self, seq_ids) -> int:
        """Slots allocated to these sequences but not yet written (tail waste)."""
        return int(sum(self.blocks.num_seq_blocks(s) * self.block_size - self.blocks.context_len(s)
                       for s in np.asarray(seq_ids)))
