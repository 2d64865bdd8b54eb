"""Caches of bounded size on the GPU: rotary positions across an eviction, and what follows a step that went wrong."""
import numpy as np
import pytest
import torch

from tests import partial_ref as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture
def pkv(pkv_lib, cuda_device):
    pkv_lib.device_error()
    yield pkv_lib
    assert pkv_lib.device_error() == 0


def test_rotation_after_an_eviction(pkv):
    """Tokens appended before and after an eviction are rotated by their positions in the text: the same queries and
    attention as over a cache that holds every token and is asked for the ones that stayed."""
    from paged_kv_cache_102_gb300.cache import PagedKVCache
    hq, hkv, bs, dim, n, more, budget = 4, 2, 16, 64, 90, 20, 33
    g = torch.Generator().manual_seed(5)
    k, v, q = (torch.randn(n + more, h, dim, generator=g).to(F16).cuda() for h in (hkv, hkv, hq))
    inv_freq, _ = pkv.rope_inv_freq(dim)
    # every token, rotated by its position, at slot i
    kc, vc = (torch.zeros(8, hkv, bs, dim, dtype=F16, device="cuda") for _ in range(2))
    at = torch.arange(n + more, dtype=torch.int32, device="cuda")
    rotated = pkv.paged_rope_append(q, k, v, at, at.long(), inv_freq, kc, vc)
    held_k, held_v = (c.transpose(1, 2).reshape(-1, hkv, dim)[:n + more].double().cpu() for c in (kc, vc))

    cache = PagedKVCache(16, hkv, bs, dim, dtype=F16)
    cache.add_sequence(1, 0)
    for i in range(n):
        got = cache.rope_append([1], q[i:i + 1], k[i:i + 1], v[i:i + 1], inv_freq)
        assert torch.equal(got[0], rotated[i])
    scores = torch.rand(1, hkv, 96, generator=g).cuda()
    kept = cache.evict([1], [2], scores, budget, 8, sinks=2).kept[0].cpu()
    for i in range(n, n + more):
        got = cache.rope_append([2], q[i:i + 1], k[i:i + 1], v[i:i + 1], inv_freq)
        assert torch.equal(got[0], rotated[i])
    out = cache.decode([2], got, 0.125).double().cpu()
    for h in range(hkv):
        stay = torch.cat([kept[h].long(), torch.arange(n, n + more)])
        for e in range(h * hq // hkv, (h + 1) * hq // hkv):
            p = torch.softmax(0.125 * (held_k[stay, h] @ rotated[-1, e].double().cpu()), 0)
            want, size = p @ held_v[stay, h], p @ held_v[stay, h].abs()
            # binary16: the output's rounding, half a step; float32 logits and sums
            assert torch.all((out[0, e] - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -12 * size + 1e-6)


def test_nothing_to_do_is_done_in_order(pkv):
    """Batches without a token or a row: what follows on the stream finds the call's zeros, and the call nothing of what
    follows."""
    B, hq, hkv, dim = 4096, 64, 8, 128
    kc = torch.zeros(4, hkv, 16, dim, dtype=BF16, device="cuda")
    tables = torch.zeros(B, 64, dtype=torch.int32, device="cuda")
    q = torch.randn(B, hq, dim, device="cuda").to(BF16)
    scores = torch.zeros(B, hkv, 64 * 16, device="cuda")
    empty = torch.zeros(B, dtype=torch.int32, device="cuda")
    out, seen = torch.empty_like(q), torch.empty_like(q)
    for _ in range(10):
        lens = empty.clone()
        out.fill_(3.0)
        pkv.paged_attention_decode_scored(q, kc, kc, tables, lens, 0.1, scores, out=out)
        seen.copy_(out)
        lens.fill_(16)
        assert torch.all(seen == 0) and torch.all(scores == 0)
        out.fill_(3.0)
        lens.zero_()
        pkv.paged_attention_decode_window(q, kc, kc, tables, lens, 0.1, 600, out=out)
        seen.copy_(out)
        assert torch.all(seen == 0)
    # no new tokens, and several shares
    tables, lens = tables[:2].repeat(1, 64).contiguous(), torch.full((2,), 60000, dtype=torch.int32, device="cuda")
    valid = torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda")
    assert pkv._native.lib().pkv_chunk_workspace_size(2, 200, hq, hkv, dim, tables.shape[1], 16) > 256
    for _ in range(10):
        starts = torch.zeros_like(valid)
        out[:200] = 3.0
        pkv.paged_attention_chunk(q[:200], kc, kc, tables, lens, starts, 0.1, out=out[:200])
        starts.copy_(valid)
        torch.cuda.synchronize()
        assert torch.all(out[:200] == 3.0)


@pytest.mark.parametrize("cache,group,dim", [("act", 1, 64), ("act", 2, 128), ("act", 4, 64), ("act", 8, 128),
                                             ("e4m3", 1, 128), ("e4m3", 4, 128), ("e4m3", 8, 64), ("e4m3", 8, 128)])
def test_scores_of_a_bad_table_stay(pkv, cache, group, dim):
    """A step over a table with an entry outside the pool leaves that sequence's scores as they are, the others' are right,
    and the next step with the table put right adds as ever."""
    lens, hkv = [700, 1300, 90, 1300, 40], 2
    paged = ref.Paged(lens, hkv, 16, dim, F16, cache, seed=group)
    (k, v, tables, n), scales = paged.cuda()
    one = dict(k_scale=scales["k_scale"], v_scale=scales["v_scale"])
    q = torch.randn(len(lens), hkv * group, dim, generator=torch.Generator().manual_seed(3)).to(F16).cuda()
    base = torch.rand(len(lens), hkv, tables.shape[1] * 16).cuda()
    right = base.clone()
    out = pkv.paged_attention_decode_scored(q, k, v, tables, n, 0.1, right, **one)
    for b, i, entry in ((1, 0, -1), (1, 81, k.shape[0]), (3, 40, 2 ** 30), (2, 5, -2 ** 31), (4, 2, k.shape[0])):
        for part in (-1, 0, 64):
            broken, scores = tables.clone(), base.clone()
            broken[b, i] = entry
            got = pkv.paged_attention_decode_scored(q, k, v, broken, n, 0.1, scores, partition_size=part, **one)
            assert pkv.device_error() == 1
            assert torch.equal(scores[b], base[b]), (b, i, part)
            rest = [x for x in range(len(lens)) if x != b]
            if part == -1:
                assert torch.equal(scores[rest], right[rest]) and torch.equal(got[rest], out[rest])
            assert torch.all((scores[rest] - right[rest]).abs() < 1e-4)
            pkv.paged_attention_decode_scored(q, k, v, tables, n, 0.1, scores, partition_size=part, **one)
            assert torch.all((scores[b] - right[b]).abs() < 1e-4)


def test_an_eviction_on_a_stream_that_is_behind(pkv):
    """Appends on the current stream, into blocks that an eviction on a busy stream has freed, come after its move."""
    from paged_kv_cache_102_gb300.cache import PagedKVCache
    hkv, dim, n = 2, 64, 64
    g = torch.Generator().manual_seed(2)
    k, v, q = (torch.randn(n, h, dim, generator=g).to(F16).cuda() for h in (hkv, hkv, 4))
    scores = torch.rand(1, hkv, 64, generator=g).cuda()
    outs = []
    for busy in (False, True):
        cache = PagedKVCache(6, hkv, 16, dim, dtype=F16)
        cache.add_sequence(1, 0)
        for i in range(n):
            cache.append([1], k[i:i + 1], v[i:i + 1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        if busy:
            with torch.cuda.stream(side):
                torch.cuda._sleep(100_000_000)
        cache.evict([1], [2], scores, 32, 4, stream=side)
        cache.add_sequence(3, 0)
        for i in range(n):  # every other block
            cache.append([3], v[i:i + 1], k[i:i + 1])
        assert cache.blocks.num_free == 0
        torch.cuda.current_stream().wait_stream(side)
        outs.append(cache.decode([2, 3], q[:2], 0.125))
    assert torch.equal(outs[0], outs[1])


def test_eviction_without_a_limit(pkv):
    """The largest budget there is: everything stays, and the list of it is -1 behind that to its end."""
    n, most = 40, 2 ** 31 - 1
    paged = ref.Paged([n], 1, 16, 64, F16, seed=4, extra_blocks=4)
    (k, v, tables, lens), _ = paged.cuda()
    scores, dst = torch.rand(1, 1, 48).cuda(), paged.free[:3].view(1, 3).to(torch.int32).cuda()
    kept = torch.zeros(1, 1, most, dtype=torch.int32, device="cuda")
    got = pkv.paged_kv_evict(k, v, scores, tables, lens, dst, most, 8, kept=kept)
    assert got.context_lens.tolist() == [n] and torch.equal(got.scores[0, 0, :n], scores[0, 0, :n])
    assert kept[0, 0, :n].tolist() == list(range(n))
    rest = kept.view(-1)[n:]
    assert all(bool(torch.all(part == -1)) for part in rest.split(1 << 28))
    for j in range(n):
        a, b = (int(t[0, j // 16]) for t in (tables, dst))
        assert torch.equal(k[a, 0, j % 16], k[b, 0, j % 16]) and torch.equal(v[a, 0, j % 16], v[b, 0, j % 16])
