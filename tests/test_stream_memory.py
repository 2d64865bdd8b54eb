"""Which stream the binding's own memory belongs to: on the CPU, with streams and allocations that only record."""
import types

import pytest
import torch


class _Streams:
    """Stands in for CUDA's streams: which is current, which are capturing, and what was allocated on which."""

    def __init__(self, monkeypatch):
        self.current, self.capturing, self.allocated = 0, set(), []
        outer = self

        class Context:
            def __init__(self, stream):
                self.handle = stream.cuda_stream

            def __enter__(self):
                self.before, outer.current = outer.current, self.handle

            def __exit__(self, *exc):
                outer.current = self.before

        real_empty = torch.empty

        def empty(*size, device=None, **kw):
            t = real_empty(*size, **kw)
            outer.allocated.append((outer.current, t))
            return t

        monkeypatch.setattr(torch.cuda, "stream", Context)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _at(handle))
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: self.current in self.capturing,
                            raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: self.current, raising=False)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _at(self.current))


@pytest.fixture
def streams(monkeypatch, pkv_lib):
    monkeypatch.setattr(pkv_lib, "_ws_cache", {})
    return _Streams(monkeypatch)


def _sparse_decode(pkv, monkeypatch, stream, blocks=4):
    """The workspace that a call on `stream` passes to the library: any call of the binding will do."""
    seen = []
    monkeypatch.setattr(pkv._native, "call", lambda func, *args: seen.append(args))
    monkeypatch.setattr(pkv, "_require_cuda", lambda *a, **k: None)
    monkeypatch.setattr(pkv, "_require_out", lambda *a, **k: None)
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    pkv.paged_attention_decode_sparse(q, kc, kc, torch.zeros(2, 2, blocks, dtype=torch.int32),
                                      torch.zeros(2, 2, dtype=torch.int32), 0.1, out=q, stream=stream)
    return seen[0][-3]


def _at(handle):
    return types.SimpleNamespace(cuda_stream=handle)


def test_captured_calls_on_two_given_streams(streams, pkv_lib, monkeypatch):
    """Two calls of one capture, on streams forked from the capturing one, may run at once: each workspace belongs to
    the stream that the call runs on, so that the second is not the first one handed out again."""
    streams.current = 1
    streams.capturing = {1, 2, 3}
    got = [_sparse_decode(pkv_lib, monkeypatch, _at(h)) for h in (2, 3)]
    assert [h for h, _ in streams.allocated] == [2, 3]
    assert [t.data_ptr() for _, t in streams.allocated] == got


def test_only_the_given_stream_captures(streams, pkv_lib, monkeypatch):
    """A capture on a stream that is not the current one: the graph gets memory of its own, not the reusable buffer."""
    first = _sparse_decode(pkv_lib, monkeypatch, _at(2))
    streams.capturing = {2}
    assert _sparse_decode(pkv_lib, monkeypatch, _at(2)) != first
    streams.capturing = {1}
    streams.current = 1  # and an eager call beside a capture keeps to the reusable one
    assert _sparse_decode(pkv_lib, monkeypatch, _at(2)) == first


def test_a_replaced_workspace_belongs_to_its_stream(streams, pkv_lib, monkeypatch):
    """A larger call replaces the reusable buffer; the old one goes back to the stream that may still use it."""
    run = lambda handle, blocks: _sparse_decode(pkv_lib, monkeypatch, _at(handle), blocks)  # noqa: E731
    small = run(2, 40)
    assert run(2, 4) == small
    large = run(2, 4000)
    assert large != small and run(2, 40) == large and run(3, 4) != large
    assert [h for h, _ in streams.allocated] == [2, 2, 3]


@pytest.mark.parametrize("kind", ["plain", "scaled"])
def test_cache_steps_keep_their_uploads_for_the_given_stream(pkv_lib, monkeypatch, kind):
    """Slots, positions, copy pairs, tables and lengths that PagedKVCache uploads for a step on a given stream are
    marked as used there, each of them, before the step is enqueued."""
    from paged_kv_cache_102_gb300 import cache as cache_mod
    recorded, used = [], []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _at(handle))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s.cuda_stream)))

    def launched(name, *own):
        def call(*args, stream=None, **kw):
            used.extend((name, (args[i].data_ptr(), stream.cuda_stream) in recorded) for i in own)
        return call

    for name, own in (("paged_kv_append", (2,)), ("paged_kv_append_scaled", (2,)), ("paged_rope_append", (3, 4)),
                      ("paged_block_copy", (2,)), ("paged_attention_decode", (3, 4)),
                      ("paged_attention_decode_scaled", (5, 6))):
        monkeypatch.setattr(cache_mod, name, launched(name, *own))
    cache = cache_mod.PagedKVCache(8, 2, 16, 64, device="cpu", block_scales=kind == "scaled")
    cache.add_sequence(0, 5)
    cache.fork(0, 1)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    s = _at(7)
    cache.append([0, 1], x, x, stream=s)  # with a copy-on-write copy
    cache.rope_append([0, 1], x, x, x, torch.ones(32), stream=s)
    cache.decode([0, 1], x, 0.1, stream=s)
    assert len(used) == 6 and all(ok for _, ok in used), used
    assert {h for _, h in recorded} == {7}
