"""Refusals of the block-scaled, rotary and table-extending calls: on the host, before anything is enqueued."""
import pytest
import torch

A = 1 << 12  # a pointer that is never followed


def _extend(lib, **kw):
    a = dict(tables=A, maxb=4, ctx=A, new=A, B=2, bs=16, free=A, nfree=4, head=A, nb=8, T=2, slots=A, pos=A, ss=A,
             bst=A + 64, lens=A + 128, hout=A, stream=None)
    a.update(kw)
    return lib.paged_extend_tables(*a.values())


def test_extend_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert _extend(lib, maxb=0) == 1 and _extend(lib, bs=0) == 1 and _extend(lib, nb=0) == 1
    assert _extend(lib, B=-1) == 1 and _extend(lib, T=-1) == 1 and _extend(lib, nfree=-1) == 1
    assert _extend(lib, maxb=1 << 30, bs=16) == 1
    for name in ("tables", "ctx", "new", "free", "head", "slots", "pos", "ss", "bst", "lens", "hout"):
        assert _extend(lib, **{name: None}) == 1, name
    assert _extend(lib, slots=A + 8) == 1 and _extend(lib, pos=A + 4) == 1 and _extend(lib, ctx=A + 2) == 1
    assert _extend(lib, bst=A) == 1                 # seq_starts and block_starts are one buffer
    assert _extend(lib, lens=A) == 1                # lengths over new_lens (new is A too)


def _append(lib, **kw):
    a = dict(k=A, ks=1024, v=A, vs=1024, slots=A, T=4, kc=A, vc=A, ksc=A, vsc=A, nb=8, hkv=8, bs=16, D=128, act=1,
             stream=None)
    a.update(kw)
    return lib.paged_kv_append_scaled(*a.values())


def test_append_scaled_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert _append(lib, D=100) == 1 and _append(lib, D=264) == 1 and _append(lib, D=0) == 1
    assert _append(lib, act=2) == 1 and _append(lib, T=-1) == 1 and _append(lib, bs=0) == 1
    assert _append(lib, bs=(1 << 20) + 1) == 1 and _append(lib, hkv=65536) == 1
    assert _append(lib, ks=1028) == 1 and _append(lib, vs=-8) == 1
    for name in ("k", "v", "slots", "kc", "vc", "ksc", "vsc"):
        assert _append(lib, **{name: None}) == 1, name
    assert _append(lib, k=A + 8) == 1 and _append(lib, kc=A + 4) == 1 and _append(lib, slots=A + 4) == 1
    assert _append(lib, T=0) == 0


def _rope(lib, **kw):
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, pos=A, slots=A, T=4, f=A, rot=128, inter=0, factor=1.0, qo=A,
             qos=1024, kc=A, vc=A, nb=8, hq=8, hkv=2, bs=16, D=128, act=1, cache=1, k1=None, v1=None, kb=None,
             vb=None, stream=None)
    a.update(kw)
    return lib.paged_rope_append(*a.values())


def test_rope_append_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert _rope(lib, rot=0) == 1 and _rope(lib, rot=7) == 1 and _rope(lib, rot=130) == 1
    assert _rope(lib, factor=float("nan")) == 1 and _rope(lib, factor=float("inf")) == 1
    assert _rope(lib, cache=0) == 1                                 # 16-bit types differ
    assert _rope(lib, cache=2) == 1                                 # no scales
    assert _rope(lib, cache=2, k1=A) == 1 and _rope(lib, cache=2, kb=A) == 1
    assert _rope(lib, cache=2, k1=A, v1=A, kb=A, vb=A) == 1         # both kinds
    assert _rope(lib, qs=1020) == 1 and _rope(lib, qos=512) == 1    # rows of q_out overlap
    assert _rope(lib, qs=2048) == 1                                 # in place with another stride
    assert _rope(lib, hq=-1) == 1 and _rope(lib, D=512, rot=128) == 1
    for name in ("q", "k", "v", "pos", "slots", "f", "qo", "kc", "vc"):
        assert _rope(lib, **{name: None}) == 1, name
    assert _rope(lib, q=A + 2) == 1 and _rope(lib, pos=A + 2) == 1
    assert _rope(lib, T=0) == 0


def _decode(lib, **kw):
    a = dict(q=A, k=A, v=A, ks=A, vs=A, tables=A, maxb=4, lens=A, B=2, Hq=8, Hkv=8, bs=16, D=128, NB=16, scale=0.1,
             out=A, act=1, part=-1, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.paged_attention_decode_scaled(*a.values())


def test_decode_scaled_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert _decode(lib, Hq=12) == 2 and _decode(lib, Hq=24) == 1 and _decode(lib, D=96) == 1 and _decode(lib, bs=8) == 1
    assert _decode(lib, act=2) == 1 and _decode(lib, ks=None) == 1 and _decode(lib, vs=None) == 1
    assert _decode(lib, ks=A + 2) == 1 and _decode(lib, part=48) == 1 and _decode(lib, scale=float("inf")) == 1
    assert _decode(lib, ws=None) == 1 and "pkv_scaled_workspace_size" in lib.pkv_last_error().decode()
    assert _decode(lib, B=0) == 0


def test_scaled_partitions_and_workspace(pkv_lib):
    size, ws = pkv_lib.resolve_partition_size, pkv_lib.workspace_size
    assert size(4, 8, 8, 128, 129, 16, block_scales=True) == 512       # 4 * 8 * 5 = 160 items, whatever the group
    assert size(1, 8, 8, 64, 129, 16, block_scales=True) == 256        # 8 * 5 = 40 items
    assert size(4, 8, 8, 128, 8, 16, block_scales=True) == 128         # the whole context
    assert size(64, 8, 8, 128, 129, 16, block_scales=True) == 2048     # 64 * 8 * 5 = 2560 items
    assert size(64, 8, 8, 128, 100, 16, block_scales=True) == 1600     # 64 * 8 * 4 = 2048, the whole context
    assert size(4, 8, 8, 128, 129, 16, 1024, block_scales=True) == 1024
    assert size(4, 8, 8, 128, 129, 16, 48, block_scales=True) == -1
    rows = 4 * 8 * 5
    assert ws(4, 8, 8, 128, 129, 16, block_scales=True) == 256 + -(-rows * 8 // 256) * 256 + rows * 128 * 4
    assert ws(4, 8, 8, 128, 129, 16, 48, block_scales=True) == 0


def test_copy_and_swap_refusals(pkv_lib):
    lib = pkv_lib._native.lib()
    assert lib.paged_block_copy_scaled(A, A, None, A, A, 1, 8, 2, 4096, None) == 1
    assert lib.paged_block_copy_scaled(A, A, A, A, A, 1, 8, 0, 4096, None) == 1
    assert lib.paged_block_copy_scaled(A, A, A, A, A, 1, 8, 2, 100, None) == 1
    assert lib.paged_block_copy_scaled(A, A, A, A, A, 0, 8, 2, 4096, None) == 0
    assert lib.paged_block_scales_swap(A, A, A, 1, 8, 2, None, 0, None) == 1
    assert lib.paged_block_scales_swap(A, A, A, 1, 8, 2, A, 2, None) == 1
    assert lib.paged_block_scales_swap(A, A, A, 0, 8, 2, A, 1, None) == 0


def test_binding_refusals_on_the_cpu(pkv_lib):
    """Shapes, types and devices that the binding refuses (CPU tensors never reach the library)."""
    p = pkv_lib
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(4, 2)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots, pos = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        p.paged_kv_append_scaled(k, k, slots, kc, kc, s, s)
    with pytest.raises(ValueError, match="E4M3"):
        p.paged_kv_append_scaled(k, k, slots, kc.float(), kc.float(), s, s)
    with pytest.raises(ValueError, match="float32"):
        p.paged_kv_append_scaled(k, k, slots, kc, kc, s[:3], s[:3])
    with pytest.raises(ValueError, match="go together"):
        p.paged_kv_append_scaled(k, k, slots, kc, kc, s, None)
    with pytest.raises(ValueError, match="CUDA"):
        p.paged_rope_append(k, k, k, pos, slots, torch.zeros(32), kc, kc, k_scales=s, v_scales=s)
    with pytest.raises(ValueError, match="CUDA"):
        p.paged_attention_decode_scaled(k, kc, kc, s, s, torch.zeros(3, 1, dtype=torch.int32), pos, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        p.paged_extend_tables(torch.zeros(3, 2, dtype=torch.int32), pos, pos, pos, pos[:1], 16, 4, num_tokens=3)
    with pytest.raises(ValueError, match="neither"):
        p.DecodePlan(k, kc, kc, None, None, 0.1, k_scales=s, v_scales=s, k_scale=s)
    with pytest.raises(ValueError, match="not both"):
        from paged_kv_cache_102_gb300.cache import PagedKVCache
        PagedKVCache(4, 2, 16, 64, device="cpu", block_scales=True, k_scale=s, v_scale=s)
