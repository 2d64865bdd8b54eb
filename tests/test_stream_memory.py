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

        self.recorded = []

        def on_the_host(real):
            def make(*size, device=None, **kw):
                t = real(*size, **kw)
                outer.allocated.append((outer.current, t))
                return t
            return make

        monkeypatch.setattr(torch.cuda, "stream", Context)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _at(handle))
        monkeypatch.setattr(torch, "empty", on_the_host(torch.empty))
        monkeypatch.setattr(torch, "zeros", on_the_host(torch.zeros))
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: outer.recorded.append((t.data_ptr(), s.cuda_stream)))
        monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: self.current in self.capturing,
                            raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: self.current, raising=False)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _at(self.current))


@pytest.fixture
def streams(monkeypatch, pkv_lib):
    monkeypatch.setattr(pkv_lib, "_ws_cache", {})
    return _Streams(monkeypatch)


def _calls(pkv, monkeypatch):
    """The library's calls from now on, which are not made, with CPU tensors let through."""
    seen = []
    monkeypatch.setattr(pkv._native, "call", lambda func, *args: seen.append(args))
    for check in ("_require_cuda", "_require_out"):
        monkeypatch.setattr(pkv, check, lambda *a, **k: None)
    return seen


def _sparse_decode(pkv, monkeypatch, stream, blocks=4):
    """The workspace that a call on `stream` passes to the library: any call of the binding will do."""
    seen = _calls(pkv, monkeypatch)
    q = torch.ones(2, 8, 64, dtype=torch.bfloat16)
    kc = torch.ones(4, 2, 16, 64, dtype=torch.bfloat16)
    pkv.paged_attention_decode_sparse(q, kc, kc, torch.ones(2, 2, blocks, dtype=torch.int32),
                                      torch.ones(2, 2, dtype=torch.int32), 0.1, out=q, stream=stream)
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


def test_new_outputs_belong_to_the_given_stream(streams, pkv_lib, monkeypatch):
    """Outputs that a call makes: bytes that the current stream's work may still hold are not the given stream's to
    write, and zeros are written there too.  The current stream, which reads them, is recorded."""
    _calls(pkv_lib, monkeypatch)
    streams.current = 1
    q = torch.ones(2, 8, 64, dtype=torch.bfloat16)
    kc = torch.ones(4, 2, 16, 64, dtype=torch.bfloat16)
    tables, lens = torch.ones(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    outs = [pkv_lib.paged_attention_decode(q, kc, kc, tables, lens, 0.1, stream=_at(2)),
            pkv_lib.paged_attention_decode_append(q, kc[:2, :, 0].contiguous(), kc[:2, :, 0].contiguous(), lens.long(),
                                                  kc, kc, tables, lens, 0.1, stream=_at(2)),
            pkv_lib.paged_attention_decode_sparse(q, kc, kc, torch.ones(2, 2, 4, dtype=torch.int32),
                                                  torch.ones(2, 2, dtype=torch.int32), 0.1, stream=_at(2)),
            pkv_lib.quest_block_minmax(kc, tables, lens, stream=_at(2)),
            *pkv_lib.quest_select(q, torch.ones(4, 2, 2, 64), tables, lens, 16, 2, stream=_at(2))]
    assert {h for h, _ in streams.allocated} == {2}
    assert streams.recorded == [(t.data_ptr(), 1) for t in outs]
    streams.allocated.clear()
    pkv_lib.paged_attention_decode(q, kc, kc, tables, lens, 0.1)
    assert {h for h, _ in streams.allocated} == {1}


def test_new_outputs_of_the_step_calls(streams, pkv_lib, monkeypatch):
    """The same of the calls whose checks need pointers on a device."""
    streams.current = 1
    monkeypatch.setattr(pkv_lib, "_pointers", lambda name, device, names, *t: [x.data_ptr() for x in t])
    monkeypatch.setattr(pkv_lib, "_call_on", lambda *a: None)
    monkeypatch.setattr(pkv_lib, "_rows", lambda *a: 0)
    monkeypatch.setattr(pkv_lib, "_require_out", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    q, s = torch.ones(2, 2, 64, dtype=torch.bfloat16), torch.ones(4, 2)
    kc = torch.ones(4, 2, 16, 64, dtype=torch.uint8)
    tables, lens = torch.ones(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    outs = [pkv_lib.paged_attention_decode_scaled(q, kc, kc, s, s, tables, lens, 0.1, stream=_at(2)),
            pkv_lib.paged_rope_append(q, q, q, lens, lens.long(), torch.ones(32), kc, kc, k_scales=s, v_scales=s,
                                      stream=_at(2)),
            *pkv_lib.paged_extend_tables(tables, lens, lens, lens, lens[:1], 16, 4, num_tokens=2, stream=_at(2))]
    assert {h for h, _ in streams.allocated} == {2}
    assert streams.recorded == [(t.data_ptr(), 1) for t in outs]


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
