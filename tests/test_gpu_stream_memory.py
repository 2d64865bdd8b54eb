"""The binding's own memory on streams that are not the current one, on the GPU."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def pkv(pkv_lib, cuda_device):
    pkv_lib.device_error(reset=True)
    yield pkv_lib
    assert pkv_lib.device_error(reset=True) == 0


def _case(seed, blocks, hq=32, hkv=4, D=128, bs=16):
    """Arguments of paged_attention_decode_scaled for sequences of so many blocks."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = sum(blocks)
    at = np.cumsum([0] + blocks)
    tables = torch.zeros(len(blocks), max(blocks), dtype=torch.int32)
    for b, n in enumerate(blocks):
        tables[b, :n] = torch.arange(at[b], at[b] + n)
    def codes():
        return torch.randint(0, 0x70, (nb, hkv, bs, D), dtype=torch.uint8, device="cuda", generator=g)

    scales = lambda: torch.exp2(torch.randint(-9, -4, (nb, hkv), device="cuda", generator=g).float())  # noqa: E731
    q = torch.randn(len(blocks), hq, D, device="cuda", generator=g).to(torch.bfloat16)
    lens = torch.tensor([n * bs - 3 for n in blocks], dtype=torch.int32, device="cuda")
    return q, codes(), codes(), scales(), scales(), tables.cuda(), lens, 0.1


@pytest.mark.parametrize("given", [True, False], ids=["stream argument", "current stream"])
def test_two_decodes_of_one_capture(pkv, given):
    """Two decodes on streams forked from a capturing one, as branches that may run at once."""
    args = [_case(s, [120, 90, 7, 200, 64, 128]) for s in (1, 2)]
    want = [pkv.paged_attention_decode_scaled(*a) for a in args]
    outs = [torch.empty_like(w) for w in want]
    main, s1, s2 = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        for s, a, out in ((s1, args[0], outs[0]), (s2, args[1], outs[1])):
            s.wait_stream(main)
            if given:
                pkv.paged_attention_decode_scaled(*a, out=out, stream=s)
            else:
                with torch.cuda.stream(s):
                    pkv.paged_attention_decode_scaled(*a, out=out)
        main.wait_stream(s1)
        main.wait_stream(s2)
    for _ in range(20):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_larger_call_on_a_given_stream(pkv):
    """A call that outgrows the stream's workspace while the call before it is still waiting to run."""
    small, large = _case(3, [100, 64]), _case(4, [150] * 10)
    want = [pkv.paged_attention_decode_scaled(*a) for a in (small, large)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # about ten milliseconds
    first = pkv.paged_attention_decode_scaled(*small, stream=s)
    second = pkv.paged_attention_decode_scaled(*large, stream=s)
    junk = [torch.full((1 << 18,), 77, dtype=torch.uint8, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    assert torch.equal(first, want[0]) and torch.equal(second, want[1])
    assert all(bool((j == 77).all()) for j in junk)


@pytest.mark.parametrize("kind", ["plain", "scaled"])
def test_cache_steps_on_a_given_stream(pkv, kind):
    """Many steps of a PagedKVCache queued up behind a wait on a given stream, with uploads and other allocations of
    the current one between them, against the same steps one after the other on one stream."""
    from paged_kv_cache_102_gb300.cache import PagedKVCache
    g = torch.Generator(device="cuda").manual_seed(11)
    n, hq, hkv, D, steps = 5, 8, 2, 64, 40
    rand = lambda h: torch.randn(steps, n, h, D, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    q, k, v = rand(hq), rand(hkv), rand(hkv)
    freq, _ = pkv.rope_inv_freq(D)

    def run(stream):
        cache = PagedKVCache(64, hkv, 16, D, block_scales=kind == "scaled")
        for i in range(n):
            cache.add_sequence(i, 0)
        outs, q_outs = torch.empty_like(q), torch.empty_like(q)
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(40_000_000)  # about twenty milliseconds
        for t in range(steps):
            if t == 9:
                cache.free(n - 1)
                cache.fork(0, n - 1)  # the next step copies the shared block
            if t % 2:
                cache.append(range(n), k[t], v[t], stream=stream)
            else:
                cache.rope_append(range(n), q[t], k[t], v[t], freq, q_out=q_outs[t], stream=stream)
            cache.decode(range(n), q[t], 0.1, out=outs[t], stream=stream)
            torch.full((64,), -1, dtype=torch.int64, device="cuda")  # reuses what was given back too early
        torch.cuda.synchronize()
        return outs, q_outs[::2], cache.k_cache, cache.v_cache

    for a, b in zip(run(torch.cuda.Stream()), run(None)):
        assert torch.equal(a, b)


def test_captured_calls_with_new_outputs_on_given_streams(pkv):
    """Branches of one capture that make their own outputs and workspaces: rotation, tables and decode on streams
    forked from the capturing one, read on the capturing one, and the same again in the next branches."""
    a, b = _case(5, [40, 90, 7]), _case(6, [64, 3, 120])
    freq, _ = pkv.rope_inv_freq(128)
    q, k = (torch.randn(3, h, 128, device="cuda").to(torch.bfloat16) for h in (32, 4))
    pos = torch.tensor([5, 70000, 3], dtype=torch.int32, device="cuda")
    skip = torch.full((3,), -1, dtype=torch.int64, device="cuda")
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    free, head = torch.arange(8, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    tables = [torch.zeros(3, 4, dtype=torch.int32, device="cuda") for _ in range(2)]

    def branch(args, t, s):
        turned = pkv.paged_rope_append(q, k, k, pos, skip, freq, args[1], args[2], k_scales=args[3], v_scales=args[4],
                                       stream=s)
        out = pkv.paged_attention_decode_scaled(*args, stream=s)
        ext = pkv.paged_extend_tables(t, one, one, free, head, 16, 8, num_tokens=5, stream=s)
        return [turned, out, *ext]

    want = [branch(x, t, None) for x, t in zip((a, b), tables)]
    torch.cuda.synchronize()
    main, s1, s2 = (torch.cuda.Stream() for _ in range(3))
    graph = torch.cuda.CUDAGraph()
    kept = []
    with torch.cuda.graph(graph, stream=main):
        for _ in range(2):
            got = []
            for s, args, t in ((s1, a, tables[0]), (s2, b, tables[1])):
                s.wait_stream(main)
                got.append(branch(args, t, s))
            main.wait_stream(s1)
            main.wait_stream(s2)
            kept.append([[t.clone() for t in g] for g in got])
            del got
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for pair in kept:
            for g, w in zip(pair, want):
                assert all(torch.equal(x, y) for x, y in zip(g, w))
