"""Chunk attention, windowed and scored decode and eviction as programs call them: through PagedKVCache and plans, on
streams that are not the current one, in captured graphs, twice at once."""
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


def calls(pkv, seed, lens=(700, 40, 1300, 257), scaled=False):
    """The calls over a cache of its own, as (call, outputs): each writes its outputs anew."""
    act = BF16 if scaled else F16
    paged = ref.Paged(lens, 2, 16, 64, act, "scaled" if scaled else "act", seed=seed, extra_blocks=40)
    args, scales = paged.cuda()
    g = torch.Generator().manual_seed(seed)
    new = [5, 3, 70, 1]
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    q, q1 = (torch.randn(n, 8, 64, generator=g).to(act).cuda() for n in (sum(new), len(lens)))
    outs = [torch.zeros_like(q), torch.zeros_like(q1)]
    todo = [lambda **kw: pkv.paged_attention_chunk(q, *args, starts, 0.125, out=outs[0], **scales, **kw),
            lambda **kw: pkv.paged_attention_decode_window(q1, *args, 0.125, 300, sinks=5, out=outs[1], **scales, **kw)]
    if not scaled:
        base = torch.rand(len(lens), 2, paged.tables.shape[1] * 16, generator=g).cuda()
        scores, moved, kept = base.clone(), torch.zeros_like(base), torch.zeros(len(lens), 2, 64, dtype=torch.int32).cuda()
        n, out = torch.zeros(len(lens), dtype=torch.int32).cuda(), torch.zeros_like(q1)
        dst = paged.free[:16].view(4, 4).to(torch.int32).cuda()

        def scored(stream=None):
            with torch.cuda.stream(stream or torch.cuda.current_stream()):
                scores.copy_(base)
            pkv.paged_attention_decode_scored(q1, *args, 0.125, scores, out=out, stream=stream)

        todo += [scored, lambda **kw: pkv.paged_kv_evict(args[0], args[1], base, *args[2:], dst, 64, 10, sinks=2,
                                                         scores_out=moved, lens_out=n, kept=kept, **kw)]
        outs += [scores, out, moved, kept, n]

    def run(**kw):
        for call in todo:
            call(**kw)

    return run, outs


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("given", [True, False], ids=["stream argument", "current stream"])
def test_two_sets_of_one_capture(pkv, scaled, given):
    """Two sets of calls on streams forked from a capturing one, as branches that may run at once, replayed."""
    sets = [calls(pkv, s, scaled=scaled) for s in (1, 2)]
    for run, _ in sets:
        run()
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs in sets]
    main, s1, s2 = (torch.cuda.Stream() for _ in range(3))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        for s, (run, _) in zip((s1, s2), sets):
            s.wait_stream(main)
            if given:
                run(stream=s)
            else:
                with torch.cuda.stream(s):
                    run()
        main.wait_stream(s1)
        main.wait_stream(s2)
    for _ in range(10):
        for _, outs in sets:
            for o in outs:
                o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for (_, outs), w in zip(sets, want):
            assert all(torch.equal(o, x) for o, x in zip(outs, w))


def test_two_streams_at_once(pkv):
    """Calls in flight on two streams, of sizes that take other workspaces in turn."""
    sets = [calls(pkv, 3), calls(pkv, 4, lens=(90, 33, 2100, 5)), calls(pkv, 5, scaled=True)]
    for run, _ in sets:
        run()
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for s, (run, outs) in zip(streams, sets):
            with torch.cuda.stream(s):
                for o in outs:
                    o.zero_()
                run()
    torch.cuda.synchronize()
    for (_, outs), w in zip(sets, want):
        assert all(torch.equal(o, x) for o, x in zip(outs, w))


def test_new_outputs_of_a_given_stream(pkv):
    """Calls that make their outputs on a given stream, behind work of the current one that still holds its memory."""
    paged = ref.Paged([300, 77], 2, 16, 64, F16, seed=3, extra_blocks=8)
    args, _ = paged.cuda()
    q = torch.randn(20, 4, 64).to(F16).cuda()
    starts = torch.tensor([0, 9, 17], dtype=torch.int32).cuda()
    want = pkv.paged_attention_chunk(q, *args, starts, 0.125)
    assert torch.all(want[17:] == 0)
    scores = torch.rand(2, 2, 304).cuda()
    dst = paged.free[:6].view(2, 3).to(torch.int32).cuda()
    first = pkv.paged_kv_evict(args[0], args[1], scores, *args[2:], dst, 48, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        noise = torch.full((4, 1 << 20), 9.0, device="cuda")
        del noise
        got = pkv.paged_attention_chunk(q, *args, starts, 0.125, stream=side)
        moved = pkv.paged_kv_evict(args[0], args[1], scores, *args[2:], dst, 48, 8, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        assert all(torch.equal(a, b) for a, b in zip(moved, first))


@pytest.mark.parametrize("cache", ["act", "scaled"])
def test_plan_with_a_window(pkv, cache):
    paged = ref.Paged([700, 33, 1, 90], 2, 16, 128, BF16, cache, seed=2)
    args, scales = paged.cuda()
    q = torch.randn(4, 8, 128).to(BF16).cuda()
    plan = pkv.DecodePlan(q, *args, 0.1, window=100, sinks=7, **scales)
    for _ in range(2):
        want = pkv.paged_attention_decode_window(q, *args, 0.1, 100, sinks=7, **scales)
        assert torch.equal(plan.run(), want)
        q.normal_()
        args[3][0] -= 5


def test_chunk_runs_again_the_same(pkv):
    """Many runs of one call: the same bits, and no wait that gives up."""
    paged = ref.Paged([900, 400, 1700], 4, 16, 128, BF16, seed=6)
    args, _ = paged.cuda()
    q = torch.randn(900 + 400 + 30, 16, 128).to(BF16).cuda()
    starts = torch.tensor([0, 900, 1300, 1330], dtype=torch.int32).cuda()
    want = pkv.paged_attention_chunk(q, *args, starts, 0.09)
    for _ in range(300):
        assert torch.equal(pkv.paged_attention_chunk(q, *args, starts, 0.09), want)


@pytest.mark.parametrize("cache,dim,factor", [("act", 64, 1.0), ("act", 64, 1.5), ("act", 128, 1.0), ("act", 128, 1.5),
                                              ("scaled", 64, 1.0), ("scaled", 128, 1.0), ("act", 64, 4.0)])
def test_chunk_references_that_move(pkv, cache, dim, factor):
    """Rows whose first tile, four tokens in front of the window, has far smaller logits than the window, so that what
    they summed up is multiplied when their reference moves, in few of many rows or (factor 4) in most: the same bits
    every time, and the right ones."""
    n, hq, hkv = 3000, 32, 32
    paged = ref.Paged([n, n], hkv, 16, dim, F16, cache, seed=41)
    q = (factor * torch.randn(2 * n, hq, dim, generator=torch.Generator().manual_seed(42))).to(F16)
    args, scales = paged.cuda()
    starts = torch.tensor([0, n, 2 * n], dtype=torch.int32).cuda()
    dev, scale = q.cuda(), dim ** -0.5
    run = lambda: pkv.paged_attention_chunk(dev, *args, starts, scale, window=300, sinks=4, **scales)  # noqa: E731
    first = run()
    differing = sum(not torch.equal(run(), first) for _ in range(300))
    assert differing == 0
    for r in range(310, 2 * n, 373):
        b, pos = divmod(r, n)
        want, _, tol = ref.attend(paged, b, q[r], ref.visible(pos, 300, 4), scale)
        ref.check(first[r], want, tol)


@pytest.mark.parametrize("kind", ["16-bit", "block scales"])
def test_cache_prompts_windows_and_drafts(pkv, kind):
    """PagedKVCache: a prompt appended token by token, its chunk attention in two parts, drafts, windowed steps."""
    from paged_kv_cache_102_gb300.cache import PagedKVCache
    hq, hkv, bs, dim, n = 8, 2, 16, 64, 45
    cache = PagedKVCache(32, hkv, bs, dim, dtype=BF16, block_scales=kind == "block scales")
    g = torch.Generator().manual_seed(0)
    k, v, q = (torch.randn(n, h, dim, generator=g).to(BF16).cuda() for h in (hkv, hkv, hq))
    for s in (7, 8):
        cache.add_sequence(s, 0)
    for i in range(n):
        cache.append([7], k[i:i + 1], v[i:i + 1])
        if i < 20:
            cache.append([8], v[i:i + 1], k[i:i + 1])
    tables, lens = cache.tables([7, 8])
    got = cache.attend([7, 8], torch.cat([q[40:], q[:3]]), [5, 3], 0.125)
    starts = torch.tensor([0, 5, 8], dtype=torch.int32).cuda()
    want = pkv.paged_attention_chunk(torch.cat([q[40:], q[:3]]), cache.k_cache, cache.v_cache, tables, lens, starts, 0.125,
                                     k_scales=cache.k_scales, v_scales=cache.v_scales)
    assert torch.equal(got, want)
    one = cache.decode([7, 8], q[[44, 2]], 0.125)
    tol = 2.0 ** -6  # of values of at most about 4: both forms' roundings
    assert torch.all((one.float() - got[[4, 7]].float()).abs() < tol * 4)
    win = cache.decode([7, 8], q[[44, 2]], 0.125, window=9, sinks=2)
    many = cache.attend([7, 8], torch.cat([q[40:], q[:3]]), [5, 3], 0.125, window=9, sinks=2)
    assert torch.all((win.float() - many[[4, 7]].float()).abs() < tol * 4)
    with pytest.raises(ValueError):
        cache.attend([7, 8], q[:8], [5, 4], 0.125)
    with pytest.raises(ValueError):
        cache.attend([7, 8], q[:26], [5, 21], 0.125)
    with pytest.raises(ValueError):
        cache.decode([7, 8], q[:2], 0.125, sinks=2)
    if kind == "block scales":
        with pytest.raises(ValueError):
            cache.decode_scored([7], q[:1], 0.125, torch.zeros(1, hkv, 64).cuda())
        with pytest.raises(ValueError):
            cache.evict([7], [9], torch.zeros(1, hkv, 64).cuda(), 16, 4)


def test_cache_evicts_a_sequence_with_shared_blocks(pkv):
    """PagedKVCache.evict: the new sequence holds the tokens that stay, a fork of the old one still sees all."""
    from paged_kv_cache_102_gb300.cache import PagedKVCache
    from paged_kv_cache_102_gb300 import OutOfBlocks
    hq, hkv, bs, dim, n = 4, 2, 16, 64, 75
    cache = PagedKVCache(8, hkv, bs, dim, dtype=F16)
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn(n, h, dim, generator=g).to(F16).cuda() for h in (hkv, hkv, hq))
    cache.add_sequence(1, 0)
    for i in range(n):
        cache.append([1], k[i:i + 1], v[i:i + 1])
    cache.fork(1, 2)
    scores = torch.zeros(1, hkv, 80).cuda()
    before = cache.decode_scored([1], q[:1], 0.125, scores)
    free = cache.blocks.num_free
    with pytest.raises(OutOfBlocks):  # no room for another copy of everything
        cache.evict([1], [5], scores, 75, 0)
    with pytest.raises(pkv.PagedKVError):
        cache.evict([1], [5], scores, 30, 31)  # more recent ones than may stay
    assert cache.blocks.num_free == free and cache.blocks.context_len(5) == -1 and cache.blocks.context_len(1) == n
    got = cache.evict([1], [5], scores, 30, 8, sinks=1)
    assert got.context_lens.tolist() == [30] and cache.blocks.context_len(5) == 30 and cache.blocks.context_len(1) == -1
    assert torch.equal(cache.decode([2], q[:1], 0.125), pkv.paged_attention_decode(
        q[:1], cache.k_cache, cache.v_cache, *cache.tables([2]), 0.125))
    assert torch.all((cache.decode([2], q[:1], 0.125).float() - before.float()).abs() < 2.0 ** -8)
    out = cache.decode([5], q[1:2], 0.125).double().cpu()
    for h in range(hkv):
        stay = got.kept[0, h].cpu()
        assert stay.tolist() == ref.evict(scores[0, h].cpu().numpy(), n, 30, 8, 1)
        kk, vv = k[stay.cuda(), h].double().cpu(), v[stay.cuda(), h].double().cpu()
        for e in range(h * hq // hkv, (h + 1) * hq // hkv):
            p = torch.softmax(0.125 * (kk @ q[1, e].double().cpu()), 0)
            # binary16: the output's and (on either path) the weights' rounding, half a step each, and float32 sums
            bound = 2.0 ** -11 * (p @ vv).abs() + (2.0 ** -11 + 2.0 ** -12) * (p @ vv.abs()) + 1e-6
            assert torch.all((out[0, e] - p @ vv).abs() <= bound)
    cache.append([5], k[:1], v[:1])
    assert cache.blocks.context_len(5) == 31
