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

attend is the attention of several new tokens a sequence (prompts, their parts,
drafted tokens) once they are in the pools; with a window, attend and decode see
the last tokens and the first ones alone.  decode_scored keeps count of what the
cached tokens are worth, and evict moves the best of them to fewer blocks.
"""
from __future__ import annotations

import numpy as np
import torch

from . import (PARTITION_AUTO, BlockManager, _torch_stream, paged_attention_chunk, paged_attention_decode,
               paged_attention_decode_scaled, paged_attention_decode_scored, paged_attention_decode_window,
               paged_block_copy, paged_kv_append, paged_kv_append_scaled, paged_kv_evict, paged_rope_append)


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
        self._moves = []  # events of evictions that may still read blocks they freed

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

    def _step_stream(self, stream):
        return torch.cuda.current_stream(self.device) if stream is None else _torch_stream(stream, self.device)

    def _await_moves(self, stream) -> None:
        """The step on the stream may write blocks that evictions, maybe on other streams, freed: behind their moves."""
        self._moves = [event for event in self._moves if not event.query()]
        for event in self._moves:
            self._step_stream(stream).wait_event(event)

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
        """append with rotary positions: rotate q [n, Hq, D] and k at each sequence's newest position (evicted tokens
        counted) and write k, v; returns the rotated queries."""
        slots, _ = self._reserve(seq_ids, stream)
        positions = self.blocks.positions(seq_ids)
        return paged_rope_append(q, k, v, self._upload(positions, stream), self._upload(slots, stream), inv_freq,
                                 self.k_cache, self.v_cache, interleaved=interleaved,
                                 attention_factor=attention_factor, q_out=q_out, k_scale=self.k_scale,
                                 v_scale=self.v_scale, k_scales=self.k_scales, v_scales=self.v_scales, stream=stream)

    def _reserve(self, seq_ids, stream):
        """Slots of one new token per sequence; the copy-on-write copies run on the stream."""
        slots, pairs = self.blocks.append_slots(seq_ids)
        self._await_moves(stream)
        if len(pairs):
            paged_block_copy(self.k_cache, self.v_cache, self._upload(pairs, stream), stream=stream,
                             k_scales=self.k_scales, v_scales=self.v_scales)
        return slots, pairs

    def decode(self, seq_ids, q: torch.Tensor, scale: float, out=None, partition_size=PARTITION_AUTO,
               max_blocks_per_seq=None, stream=None, window=None, sinks=0):
        if window is None and sinks:
            raise ValueError("PagedKVCache.decode: sinks without a window")
        tables, lens = (self._upload(a, stream) for a in self.blocks.tables(seq_ids, max_blocks_per_seq))
        if window is not None:
            return paged_attention_decode_window(q, self.k_cache, self.v_cache, tables, lens, scale, window, sinks=sinks,
                                                 out=out, k_scale=self.k_scale, v_scale=self.v_scale,
                                                 k_scales=self.k_scales, v_scales=self.v_scales,
                                                 partition_size=partition_size, stream=stream)
        if self.k_scales is not None:
            return paged_attention_decode_scaled(q, self.k_cache, self.v_cache, self.k_scales, self.v_scales, tables,
                                                 lens, scale, out=out, partition_size=partition_size, stream=stream)
        return paged_attention_decode(q, self.k_cache, self.v_cache, tables, lens, scale, out=out,
                                      k_scale=self.k_scale, v_scale=self.v_scale,
                                      partition_size=partition_size, stream=stream)

    def attend(self, seq_ids, q: torch.Tensor, new_lens, scale: float, window=None, sinks=0, out=None,
               max_blocks_per_seq=None, stream=None):
        """Attention of each sequence's last new_lens tokens, the rows of q [sum(new_lens), Hq, D] in the order of
        seq_ids; they are in the pools already."""
        new = np.asarray(new_lens, np.int64)
        if new.shape != np.asarray(seq_ids).shape or (new < 0).any() or new.sum() != q.shape[0]:
            raise ValueError("PagedKVCache.attend: q has a row for each of the sequences' new tokens")
        if any(n > self.blocks.context_len(s) for s, n in zip(np.asarray(seq_ids), new)):
            raise ValueError("PagedKVCache.attend: more new tokens than a sequence has")
        tables, lens = (self._upload(a, stream) for a in self.blocks.tables(seq_ids, max_blocks_per_seq))
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        return paged_attention_chunk(q, self.k_cache, self.v_cache, tables, lens, self._upload(starts, stream), scale,
                                     window=window, sinks=sinks, out=out, k_scale=self.k_scale, v_scale=self.v_scale,
                                     k_scales=self.k_scales, v_scales=self.v_scales, stream=stream)

    def decode_scored(self, seq_ids, q: torch.Tensor, scale: float, scores: torch.Tensor, out=None,
                      partition_size=PARTITION_AUTO, max_blocks_per_seq=None, stream=None):
        """decode that adds every cached token's weight to scores float32 [n, Hkv, tokens], a row a sequence (not for
        block scales)."""
        if self.k_scales is not None:
            raise ValueError("PagedKVCache.decode_scored: not for a block-scaled cache")
        tables, lens = (self._upload(a, stream) for a in self.blocks.tables(seq_ids, max_blocks_per_seq))
        return paged_attention_decode_scored(q, self.k_cache, self.v_cache, tables, lens, scale, scores, out=out,
                                             k_scale=self.k_scale, v_scale=self.v_scale, partition_size=partition_size,
                                             stream=stream)

    def evict(self, seq_ids, new_ids, scores: torch.Tensor, budget: int, recent: int, sinks=0, stream=None):
        """Replace each sequence by one of at most budget tokens under a new id: those that paged_kv_evict keeps, whose
        result this returns.  The old sequences are freed (blocks that they share with others stay).  Positions go on
        from the old sequence's; a window counts the tokens that are held, not the ones between them that went.
        The pool has to have free blocks for the new sequences before the old ones go.  Later appends and evictions of
        this cache wait for the move whatever their stream; other calls that write into blocks taken after it, on
        another stream, are the caller's to order."""
        if self.k_scales is not None:
            raise ValueError("PagedKVCache.evict: not for a block-scaled cache")
        seq_ids, new_ids = [int(s) for s in np.asarray(seq_ids)], [int(s) for s in np.asarray(new_ids)]
        lens = [self.blocks.context_len(s) for s in seq_ids]
        if len(new_ids) != len(seq_ids) or len(set(seq_ids)) != len(seq_ids) or budget < 1:
            raise ValueError("PagedKVCache.evict: a new id for each sequence, each once, and a positive budget")
        if lens and max(lens) > scores.shape[-1]:
            raise ValueError("PagedKVCache.evict: scores for each token of the sequences")
        added = []
        try:
            for s, n in zip(new_ids, lens):
                self.blocks.add_sequence(s, min(n, int(budget)))
                added.append(s)
            for s, old, n in zip(new_ids, seq_ids, lens):
                self.blocks.set_dropped(s, self.blocks.num_dropped(old) + n - min(n, int(budget)))
            src, length = (self._upload(a, stream) for a in self.blocks.tables(seq_ids))
            dst = self._upload(self.blocks.tables(new_ids)[0], stream)
            self._await_moves(stream)
            got = paged_kv_evict(self.k_cache, self.v_cache, scores, src, length, dst, budget, recent, sinks=sinks,
                                 stream=stream)
        except Exception:
            for s in added:  # as before
                self.blocks.free_sequence(s)
            raise
        if self.device.type == "cuda":
            self._moves.append(self._step_stream(stream).record_event())
        for s in seq_ids:
            self.blocks.free_sequence(s)
        return got

    def unused_slots(self, seq_ids) -> int:
        """Slots allocated to these sequences but not yet written (tail waste)."""
        return int(sum(self.blocks.num_seq_blocks(s) * self.block_size - self.blocks.context_len(s)
                       for s in np.asarray(seq_ids)))
