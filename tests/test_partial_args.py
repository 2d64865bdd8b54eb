"""What chunk attention, windowed and scored decode and eviction refuse, on the host (no GPU needed)."""
import pytest
import torch

A = 1 << 12  # an aligned address that nothing reads: every call here is refused, or has no rows


def _chunk(lib, **kw):
    a = dict(q=A, qs=1024, k=A, v=A, tables=A, maxb=4, lens=A, starts=A, B=2, T=5, Hq=8, Hkv=8, bs=16, D=128, NB=16,
             scale=0.1, window=0, sinks=0, out=A << 8, os=1024, act=1, cache=1, k1=None, v1=None, kb=None, vb=None,
             ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.paged_attention_chunk(*a.values())


def test_chunk_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert _chunk(lib) == 1 and "pkv_chunk_workspace_size" in lib.pkv_last_error().decode()
    assert _chunk(lib, Hq=12, Hkv=8) == 2                                # not a multiple
    assert _chunk(lib, Hq=130, Hkv=2, qs=130 * 128, os=130 * 128) == 1   # 65 query heads for a kv head
    assert _chunk(lib, D=96) == 1 and _chunk(lib, bs=8) == 1
    assert _chunk(lib, act=2) == 1 and _chunk(lib, act=0, cache=1) == 1
    assert _chunk(lib, cache=2) == 1                                     # E4M3 without scales
    assert _chunk(lib, cache=2, k1=A) == 1 and _chunk(lib, cache=2, kb=A) == 1
    assert _chunk(lib, cache=2, k1=A, v1=A, kb=A, vb=A) == 1             # both kinds
    assert _chunk(lib, kb=A, vb=A) == 1                                  # block scales of a 16-bit cache
    assert _chunk(lib, scale=float("nan")) == 1
    assert _chunk(lib, window=-1) == 1 and _chunk(lib, sinks=-1) == 1
    assert _chunk(lib, qs=1020) == 1 and _chunk(lib, os=512) == 1        # strides
    assert _chunk(lib, out=A + 1024) == 1 and "shares memory" in lib.pkv_last_error().decode()
    assert _chunk(lib, q=A + 8) == 1 and _chunk(lib, starts=A + 2) == 1  # alignment
    for name in ("q", "k", "v", "tables", "lens", "starts", "out"):
        assert _chunk(lib, **{name: None}) == 1, name
    assert _chunk(lib, maxb=1 << 28) == 1                                # the table is too long
    assert _chunk(lib, T=0) == 0 and _chunk(lib, B=0) == 0


def _window(lib, **kw):
    a = dict(q=A, k=A, v=A, tables=A, maxb=4, lens=A, B=2, Hq=8, Hkv=8, bs=16, D=128, NB=16, scale=0.1, window=8, sinks=0,
             out=A, act=1, cache=1, k1=None, v1=None, kb=None, vb=None, part=-1, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.paged_attention_decode_window(*a.values())


def test_window_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert _window(lib) == 1 and "pkv_window_workspace_size" in lib.pkv_last_error().decode()
    assert _window(lib, window=0) == 1 and _window(lib, window=-3) == 1 and _window(lib, sinks=-1) == 1
    assert _window(lib, Hq=12) == 2 and _window(lib, Hq=24) == 1 and _window(lib, D=96) == 1 and _window(lib, bs=8) == 1
    assert _window(lib, cache=2) == 1 and _window(lib, cache=2, kb=A) == 1
    assert _window(lib, cache=2, k1=A, v1=A, kb=A, vb=A) == 1 and _window(lib, kb=A, vb=A) == 1
    assert _window(lib, part=48) == 1 and _window(lib, scale=float("inf")) == 1
    assert _window(lib, B=0) == 0


def _scored(lib, **kw):
    a = dict(q=A, k=A, v=A, tables=A, maxb=4, lens=A, B=2, Hq=8, Hkv=8, bs=16, D=128, NB=16, scale=0.1, scores=A, n=64,
             out=A, act=1, cache=1, k1=None, v1=None, part=-1, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.paged_attention_decode_scored(*a.values())


def test_scored_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert _scored(lib) == 1 and "pkv_scored_workspace_size" in lib.pkv_last_error().decode()
    assert _scored(lib, n=63) == 1 and _scored(lib, scores=None) == 1 and _scored(lib, scores=A + 2) == 1
    assert _scored(lib, Hq=24) == 1 and _scored(lib, cache=2) == 1 and _scored(lib, part=48) == 1
    assert _scored(lib, B=0) == 0
    apart = dict(q=A << 1, tables=A << 2, lens=A << 3, scores=A << 4, out=A << 5, ws=A << 6, wsb=1 << 30)
    for name in ("q", "tables", "lens", "out", "ws"):
        assert _scored(lib, **{**apart, name: (A << 4) + 1024}) == 1, name
        assert "buffer of its own" in lib.pkv_last_error().decode(), name


def _evict(lib, **kw):
    a = dict(k=A, v=A, NB=16, Hkv=2, bs=16, D=64, cache=1, scores=A, n=64, tables=A << 4, maxb=4, lens=A << 5, B=2,
             dst=A << 6, maxd=2, budget=32, recent=4, sinks=0, so=A << 7, no=64, lo=A << 8, kept=A << 9, stream=None)
    a.update(kw)
    return lib.paged_kv_evict(*a.values())


def test_evict_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert _evict(lib, budget=0) == 1 and _evict(lib, recent=-1) == 1 and _evict(lib, sinks=-1) == 1
    assert _evict(lib, recent=30, sinks=3) == 1                    # more that have to stay than may
    assert _evict(lib, recent=2 ** 31 - 1, sinks=2 ** 31 - 1) == 1
    assert _evict(lib, D=96) == 1 and _evict(lib, cache=3) == 1 and _evict(lib, bs=0) == 1
    assert _evict(lib, no=31) == 1                                 # no room for the scores that stay
    assert _evict(lib, so=A) == 1 and "buffers of their own" in lib.pkv_last_error().decode()
    assert _evict(lib, lo=A << 5) == 1 and _evict(lib, kept=A << 8) == 1
    for name in ("k", "v", "scores", "tables", "lens", "dst", "so", "lo", "kept"):
        assert _evict(lib, **{name: None}) == 1, name
    assert _evict(lib, k=A + 8) == 1 and _evict(lib, lens=(A << 5) + 2) == 1
    assert _evict(lib, B=0) == 0


def test_workspaces(pkv_lib):
    lib = pkv_lib._native.lib()
    # a window's partitions: 4096 tokens seen through 1024 and 4 first ones are 66 blocks of 16, in three of 384
    assert lib.pkv_window_workspace_size(128, 64, 8, 128, 512, 16, 1024, 4, 0, -1) == (
        256 + -(-128 * 64 * 3 * 8 // 256) * 256 + 128 * 64 * 3 * 128 * 4)
    assert lib.pkv_window_workspace_size(4, 8, 8, 64, 3, 16, 16, 2, 0, -1) == 256  # one partition
    # as large as the tables allow: no partition more than without a window
    assert lib.pkv_window_workspace_size(4, 8, 8, 128, 64, 16, 2 ** 31 - 1, 2 ** 31 - 1, 1, -1) <= lib.pkv_scaled_workspace_size(
        4, 8, 8, 128, 64, 16, -1)
    # scored: statistics of each partition, their outputs, the logits
    assert lib.pkv_scored_workspace_size(2, 8, 1, 128, 64, 16, 512) == 256 + 256 + 2 * 8 * 2 * 128 * 4 + 2 * 8 * 1024 * 4
    assert lib.pkv_scored_workspace_size(2, 8, 1, 128, 64, 16, 48) == 0
    # shares of a long context, none of a short one; sizes that the call refuses need nothing more than the least
    one = lib.pkv_chunk_workspace_size(1, 509, 32, 8, 128, 1024, 32)
    assert one == 256 + 2 * 509 * 32 * 8 + 2 * 509 * 32 * 128 * 4
    assert lib.pkv_chunk_workspace_size(4, 100, 32, 8, 128, 4, 16) == 256
    for bad in ((0, 5, 8, 8, 128, 4, 16), (2, 5, 4, 8, 128, 4, 16), (2, 5, 8, 0, 128, 4, 16), (2, 5, 8, 8, 128, 4, 0)):
        assert lib.pkv_chunk_workspace_size(*bad) == 256


def test_binding_refusals_on_the_cpu(pkv_lib):
    """Shapes, types and devices that the binding refuses (CPU tensors never reach the library)."""
    p = pkv_lib
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    tables, lens, starts = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    scores = torch.zeros(3, 2, 32)
    with pytest.raises(ValueError, match="CUDA"):
        p.paged_attention_chunk(q, kc, kc, tables, lens, starts, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        p.paged_attention_decode_window(q, kc, kc, tables, lens, 0.1, 4)
    with pytest.raises(ValueError, match="CUDA"):
        p.paged_attention_decode_scored(q, kc, kc, tables, lens, 0.1, scores)
    with pytest.raises(ValueError, match="CUDA"):
        p.paged_kv_evict(kc, kc, scores, tables, lens, tables, 16, 4)
    for bad in (kc[0], kc[:, :1], kc.half()):
        with pytest.raises(ValueError, match="one type"):
            p.paged_attention_chunk(q, kc, bad, tables, lens, starts, 0.1)
        with pytest.raises(ValueError, match="one type"):
            p.paged_kv_evict(kc, bad, scores, tables, lens, tables, 16, 4)
    with pytest.raises(ValueError, match="window"):
        p.DecodePlan(q, kc, kc, tables, lens, 0.1, sinks=3)
    with pytest.raises(ValueError, match="append"):
        p.DecodePlan(q, kc, kc, tables, lens, 0.1, window=3, k_new=q, v_new=q, slot_mapping=lens)
