"""Caches of bounded size, the host's part (no GPU needed): what PagedKVCache and the block manager keep of a sequence
whose tokens were evicted."""
import numpy as np
import pytest
import torch

from paged_kv_cache_102_gb300 import cache as cache_module


@pytest.fixture
def host_cache(pkv_lib, monkeypatch):
    """A PagedKVCache of CPU pools whose device calls are noted instead of run."""
    calls = []
    for name in ("paged_kv_evict", "paged_rope_append", "paged_block_copy", "paged_kv_append"):
        monkeypatch.setattr(cache_module, name, lambda *a, _name=name, **kw: calls.append((_name, a, kw)))
    return cache_module.PagedKVCache(64, 1, 16, 64, dtype=torch.float16, device="cpu"), calls


def test_manager_counts_dropped_tokens(pkv_lib):
    bm = pkv_lib.BlockManager(16, 16)
    bm.add_sequence(1, 20)
    assert bm.num_dropped(1) == 0 and bm.num_dropped(9) == -1
    bm.set_dropped(1, 5)
    bm.fork(1, 2)
    assert bm.num_dropped(2) == 5 and bm.context_len(2) == 20
    assert bm.positions([2, 1]).tolist() == [24, 24] and bm.positions([]).tolist() == []
    with pytest.raises(pkv_lib.PagedKVError):
        bm.positions([1, 9])
    bm.append_slots([1])
    assert bm.num_dropped(1) == 5 and bm.context_len(1) == 21
    bm.swap_out(1)
    bm.swap_in(1, 4)
    assert bm.num_dropped(1) == 5
    bm.free_sequence(1)
    bm.add_sequence(1, 3)
    assert bm.num_dropped(1) == 0
    for seq, n in ((7, 1), (1, -1), (1, 2 ** 31 - 3)):
        with pytest.raises(pkv_lib.PagedKVError):
            bm.set_dropped(seq, n)
    bm.set_dropped(1, 2 ** 31 - 4)


def test_positions_go_on_after_an_eviction(host_cache):
    """Rotary positions count evicted tokens, after a second eviction and in a fork too."""
    cache, calls = host_cache
    cache.add_sequence(1, 100)
    cache.add_sequence(2, 30)
    scores = torch.zeros(2, 1, 128)

    def positions(*ids):
        calls.clear()
        cache.rope_append(ids, None, None, None, None)
        return [a[3].tolist() for name, a, _ in calls if name == "paged_rope_append"][0]

    assert positions(1, 2) == [100, 30]
    cache.evict([1, 2], [11, 12], scores, budget=40, recent=8)
    assert cache.blocks.context_len(11) == 40 and cache.blocks.context_len(12) == 31
    assert positions(11, 12) == [101, 31]
    cache.fork(11, 21)
    assert positions(21) == [102] and positions(11) == [102]
    cache.evict([11], [31], scores[:1], budget=16, recent=8)
    assert cache.blocks.context_len(31) == 16 and positions(31) == [103]
    cache.free(31)
    cache.add_sequence(31, 4)
    assert positions(31) == [4]


class Recorder:
    """A stream that notes what is put on it."""

    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def record_event(self):
        self.log.append(("record", self.cuda_stream))
        return Event(self.cuda_stream)

    def wait_event(self, event):
        self.log.append(("wait", self.cuda_stream, event.handle))


class Event:
    def __init__(self, handle):
        self.handle, self.done = handle, False

    def query(self):
        return self.done


def test_blocks_of_an_eviction_are_written_behind_its_move(host_cache, monkeypatch):
    """Appends and evictions on other streams than an eviction's wait for its move: they may write the blocks it freed."""
    cache, log = host_cache
    monkeypatch.setattr(cache_module, "_torch_stream", lambda s, device: s)
    monkeypatch.setattr(cache, "_upload", lambda array, stream: torch.from_numpy(array))
    monkeypatch.setattr(cache, "device", torch.device("cuda"))
    one, two = Recorder(1, log), Recorder(2, log)
    cache.add_sequence(1, 100)
    cache.add_sequence(2, 30)

    def steps(call):
        log.clear()
        call()
        return [x if x[0] in ("record", "wait") else x[0] for x in log]

    def append(stream):
        return steps(lambda: cache.append([2], None, None, stream=stream))

    def evict(old, new, budget, stream):
        return steps(lambda: cache.evict([old], [new], torch.zeros(1, 1, 128), budget, 8, stream=stream))

    assert append(two) == ["paged_kv_append"]
    assert evict(1, 3, 40, one) == ["paged_kv_evict", ("record", 1)]
    assert append(two) == [("wait", 2, 1), "paged_kv_append"]
    assert append(one) == [("wait", 1, 1), "paged_kv_append"]  # (in order already)
    assert steps(lambda: cache.rope_append([2], None, None, None, None, stream=two)) == [("wait", 2, 1), "paged_rope_append"]
    assert evict(3, 4, 20, two) == [("wait", 2, 1), "paged_kv_evict", ("record", 2)]
    cache._moves[0].done = True  # the finished one is forgotten
    assert append(one) == [("wait", 1, 2), "paged_kv_append"]
    cache._moves[0].done = True
    assert append(one) == ["paged_kv_append"] and not cache._moves


def test_buffers_over_the_pools_are_refused(pkv_lib):
    """Scores inside a pool or a scale, and what an eviction reads or writes inside a pool: refused on the host."""
    lib = pkv_lib._native.lib()
    M = 1 << 24  # buffers of their own; the pools are 512 KB
    at = dict(q=1, k=2, v=3, tables=4, lens=5, scores=6, out=7, k1=8, v1=9, ws=10)

    def scored(**kw):
        a = {n: i * M for n, i in at.items()} | kw
        return lib.paged_attention_decode_scored(
            a["q"], a["k"], a["v"], a["tables"], 4, a["lens"], 2, 8, 8, 16, 128, 16, 0.1, a["scores"], 64, a["out"], 1, 2,
            a["k1"], a["v1"], -1, a["ws"], 1 << 22, None)

    for name, inside in (("k", 2048), ("v", 16 * 8 * 16 * 128 - 4), ("k1", 0), ("v1", 0)):
        assert scored(scores=at[name] * M + inside) == 1
        assert "buffer of its own" in lib.pkv_last_error().decode(), name

    where = dict(k=1, v=2, scores=3, tables=4, lens=5, dst=6, so=7, lo=8, kept=9)

    def evict(**kw):
        a = {n: i * M for n, i in where.items()} | kw
        return lib.paged_kv_evict(a["k"], a["v"], 16, 2, 16, 64, 1, a["scores"], 64, a["tables"], 4, a["lens"], 2, a["dst"], 2,
                                  32, 4, 0, a["so"], 64, a["lo"], a["kept"], None)

    for name in ("scores", "tables", "lens", "dst", "so", "lo", "kept"):
        for pool in (1, 2):
            assert evict(**{name: pool * M + 16 * 2 * 16 * 64 * 2 - 4}) == 1
            assert "buffers of their own" in lib.pkv_last_error().decode(), (name, pool)
