"""Block tables, slots and positions built on the GPU (paged_extend_tables), against the host block manager and a
plain restatement; and a whole step -- tables, rotary append, decode -- captured into a graph."""
import numpy as np
import pytest
import torch

from oracle.block_manager_ref import RefBlockManager
from tests import scaled_ref as ref

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture
def pkv(pkv_lib, cuda_device):
    pkv_lib.device_error(reset=True)
    yield pkv_lib
    assert pkv_lib.device_error(reset=True) == 0


def _plain(tables, ctx, new, free, head, bs, rows):
    """The definition, request by request."""
    tables = tables.copy()
    slots, pos, starts, blocks = [], [], [0], [0]
    for b, (c, n) in enumerate(zip(ctx, new)):
        have, need = -(-c // bs), -(-(c + n) // bs)
        for j in range(have, need):
            tables[b, j] = free[head + blocks[-1] + j - have]
        for p in range(c, c + n):
            pos.append(p)
            slots.append(int(tables[b, p // bs]) * bs + p % bs)
        starts.append(starts[-1] + n)
        blocks.append(blocks[-1] + need - have)
    pad = rows - len(slots)
    return tables, slots + [-1] * pad, pos + [-1] * pad, starts, blocks


def _run(pkv, tables, ctx, new, free, head, bs, nb, rows, in_place=False):
    t = torch.from_numpy(tables).cuda()
    c, n = torch.tensor(ctx, dtype=I32).cuda(), torch.tensor(new, dtype=I32).cuda()
    f, h = torch.tensor(free, dtype=I32).cuda(), torch.tensor([head], dtype=I32).cuda()
    kw = dict(context_lens_out=c, free_head_out=h) if in_place else {}
    r = pkv.paged_extend_tables(t, c, n, f, h, bs, nb, num_tokens=rows, **kw)
    torch.cuda.synchronize()
    return t.cpu().numpy(), r


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,bs,hi,new_hi,pad", [
    (1, 16, 0, 1, 0), (1, 16, 40, 1, 3), (4, 16, 60, 1, 0), (64, 16, 2000, 1, 0), (257, 32, 300, 3, 5),
    (1023, 16, 100, 1, 1), (1025, 16, 100, 2, 0), (5000, 16, 50, 1, 0), (3, 16, 100, 5000, 7), (64, 32, 10, 900, 0),
    (7, 1, 9, 40, 2), (2000, 5, 30, 8, 11), (16, 16, 0, 16, 0), (9, 256, 3000, 1, 0),
])
def test_extend_matches_the_definition(pkv, B, bs, hi, new_hi, pad, in_place):
    rng = np.random.default_rng(B * 31 + bs)
    ctx = rng.integers(0, hi + 1, B).tolist()
    new = (rng.integers(0, new_hi + 1, B) if new_hi > 1 else np.ones(B, int)).tolist()
    cols = max(-(-(c + n) // bs) for c, n in zip(ctx, new)) + 2
    have = [-(-c // bs) for c in ctx]
    take = sum(-(-(c + n) // bs) - h for c, n, h in zip(ctx, new, have))
    nb = sum(have) + take + 9
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((B, cols), -7, np.int32)
    at = 0
    for b, h in enumerate(have):
        tables[b, :h] = perm[at:at + h]
        at += h
    free = perm[at:].tolist()
    head = len(free) - take if B % 2 else 3  # to the last block, or from the middle
    rows = sum(new) + pad
    want = _plain(tables, ctx, new, free, head, bs, rows)
    got, r = _run(pkv, tables, ctx, new, free, head, bs, nb, rows, in_place)
    assert np.array_equal(got, want[0])
    assert r.slot_mapping.tolist() == want[1] and r.positions.tolist() == want[2]
    assert r.seq_starts.tolist() == want[3] and r.block_starts.tolist() == want[4]
    assert r.context_lens.tolist() == [c + n for c, n in zip(ctx, new)]
    assert r.free_head.tolist() == [head + take]


def test_extend_without_tokens_or_requests(pkv):
    tables = np.full((3, 4), 5, np.int32)
    got, r = _run(pkv, tables, [16, 0, 7], [0, 0, 0], [1, 2], 0, 16, 8, 6)
    assert np.array_equal(got, tables) and r.slot_mapping.tolist() == [-1] * 6 and r.positions.tolist() == [-1] * 6
    assert r.seq_starts.tolist() == [0] * 4 and r.context_lens.tolist() == [16, 0, 7] and r.free_head.tolist() == [0]
    got, r = _run(pkv, tables, [16, 0, 7], [0, 0, 0], [], 0, 16, 8, 0)
    assert r.block_starts.tolist() == [0] * 4
    _, r = _run(pkv, np.zeros((0, 4), np.int32), [], [], [1], 0, 16, 8, 5)
    assert r.slot_mapping.tolist() == [-1] * 5 and r.seq_starts.tolist() == [0]
    _, r = _run(pkv, np.zeros((0, 4), np.int32), [], [], [1, 2, 3], 2, 16, 8, 0)  # nothing at all: the head stays
    assert r.free_head.tolist() == [2] and r.seq_starts.tolist() == [0] and r.block_starts.tolist() == [0]


@pytest.mark.parametrize("rows", [40, 9000])  # one launch, two launches
@pytest.mark.parametrize("what", ["blocks", "rows", "negative", "negative_ctx", "too_long", "head", "overflow"])
def test_extend_is_all_or_nothing(pkv, what, rows):
    ctx, new, free, head = [16, 30, 5], [4, 4, 4], [4, 5, 6], 0
    bits = pkv.DEV_NO_SPACE
    if what == "blocks":
        head = 2  # one left, two needed
    elif what == "rows":
        rows, new = (11, new) if rows == 40 else (9000, [4, 4, 9000])
    elif what == "head":
        head = -1
    else:
        bits = pkv.DEV_BAD_CONTEXT_LEN
        new = {"negative": [4, -1, 4], "too_long": [4, 4, 10000], "overflow": [4, 2 ** 31 - 1, 4]}.get(what, new)
        if what == "negative_ctx":
            ctx = [16, -30, 5]
    tables = np.arange(3 * 600, dtype=np.int32).reshape(3, 600) % 7
    if what == "rows":
        free = list(range(7)) * 100
    for in_place in (False, True):
        got, r = _run(pkv, tables, ctx, new, free, head, 16, 7, rows, in_place)
        assert pkv.device_error(reset=True) == bits
        assert np.array_equal(got, tables)
        assert set(r.slot_mapping.tolist()) == {-1} and set(r.positions.tolist()) == {-1}
        assert r.seq_starts.tolist() == [0] * 4 and r.block_starts.tolist() == [0] * 4
        assert r.context_lens.tolist() == ctx and r.free_head.tolist() == [head]


def test_extend_flags_bad_blocks(pkv):
    tables = np.asarray([[99, 0], [1, 0], [2, 0]], np.int32)
    got, r = _run(pkv, tables, [3, 16, 4], [1, 1, 1], [-5, 3], 0, 16, 8, 3)
    assert pkv.device_error(reset=True) == pkv.DEV_BAD_BLOCK
    assert r.slot_mapping.tolist() == [-1, -1, 2 * 16 + 4] and r.positions.tolist() == [3, 16, 4]


def test_extend_follows_the_block_manager(pkv):
    """Prompts, then decode steps: the device's tables are those of the host manager and of its restatement."""
    rng = np.random.default_rng(5)
    bs, nb, B, steps = 16, 400, 24, 40
    fl = rng.permutation(nb).astype(np.int32)
    host, want = pkv.BlockManager(nb, bs, free_list=fl), RefBlockManager(nb, bs, free_list=fl)
    prompts = rng.integers(0, 90, B)
    for i, n in enumerate(prompts):
        host.add_sequence(i, int(n))
        want.add_sequence(i, int(n))
    cols = 12
    tables = torch.zeros(B, cols, dtype=I32, device="cuda")
    lens, head = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    free = torch.from_numpy(fl).cuda()
    pkv.paged_extend_tables(tables, lens, torch.from_numpy(prompts.astype(np.int32)).cuda(), free, head, bs, nb,
                            num_tokens=int(prompts.sum()), context_lens_out=lens, free_head_out=head)
    one = torch.ones(B, dtype=I32, device="cuda")
    for _ in range(steps):
        r = pkv.paged_extend_tables(tables, lens, one, free, head, bs, nb, num_tokens=B, context_lens_out=lens,
                                    free_head_out=head)
        slots, pairs = host.append_slots(np.arange(B))
        assert len(pairs) == 0 and r.slot_mapping.tolist() == slots.tolist()
        assert slots.tolist() == [want.append_slot(i)[0] for i in range(B)]
    t, n = host.tables(np.arange(B), cols)
    assert lens.tolist() == n.tolist()
    for i in range(B):
        k = -(-int(n[i]) // bs)
        assert tables[i, :k].tolist() == t[i, :k].tolist()


def _model_step(pkv, st):
    """One layer's step: tables, rotary append into the block-scaled cache, attention."""
    r = pkv.paged_extend_tables(st["tables"], st["lens"], st["new"], st["free"], st["head"], st["bs"], st["nb"],
                                slot_mapping=st["slots"], positions=st["pos"], seq_starts=st["starts"],
                                block_starts=st["blocks"], context_lens_out=st["lens"], free_head_out=st["head"])
    q = pkv.paged_rope_append(st["qkv"][:, :st["hq"]], st["qkv"][:, st["hq"]:-st["hkv"]], st["qkv"][:, -st["hkv"]:],
                              r.positions, r.slot_mapping, st["freq"], st["kc"], st["vc"], k_scales=st["ks"],
                              v_scales=st["vs"], q_out=st["q"])
    return pkv.paged_attention_decode_scaled(q, st["kc"], st["vc"], st["ks"], st["vs"], st["tables"], st["lens"],
                                             0.1, out=st["out"], workspace=st["ws"])


@pytest.mark.parametrize("hq,hkv,D", [(16, 2, 128), (4, 4, 64), (16, 4, 64)])
def test_a_whole_step_captured_and_replayed(pkv, hq, hkv, D):
    """Prompts go in, then a captured step runs eight times, its last row padding; every step's output is held
    against the definition over the cache as it then is, and the cache against the tokens that went in."""
    g = torch.Generator().manual_seed(hq)
    bs, B, cols = 16, 5, 8
    nb = 40
    prompts = [1, 15, 33, 64, 0]
    dev = torch.device("cuda")
    freq, _ = pkv.rope_inv_freq(D)
    z = dict(device=dev)
    st = dict(bs=bs, nb=nb, hq=hq, hkv=hkv, freq=freq, tables=torch.zeros(B, cols, dtype=I32, **z),
              lens=torch.zeros(B, dtype=I32, **z), head=torch.zeros(1, dtype=I32, **z),
              free=torch.randperm(nb, generator=g).to(I32).to(dev),
              kc=torch.zeros(nb, hkv, bs, D, dtype=torch.uint8, **z), ks=torch.zeros(nb, hkv, **z),
              slots=torch.empty(B, dtype=torch.int64, **z), pos=torch.empty(B, dtype=I32, **z),
              starts=torch.empty(B + 1, dtype=I32, **z), blocks=torch.empty(B + 1, dtype=I32, **z),
              q=torch.zeros(B, hq, D, dtype=torch.bfloat16, **z), out=torch.zeros(B, hq, D, dtype=torch.bfloat16, **z),
              qkv=torch.zeros(B, hq + 2 * hkv, D, dtype=torch.bfloat16, **z),
              new=torch.tensor([1, 1, 1, 1, 0], dtype=I32, **z),
              ws=torch.empty(pkv.workspace_size(B, hq, hkv, D, cols, bs, block_scales=True), dtype=torch.uint8, **z))
    st["vc"], st["vs"] = st["kc"].clone(), st["ks"].clone()
    # prompts
    T = sum(prompts)
    r = pkv.paged_extend_tables(st["tables"], st["lens"], torch.tensor(prompts, dtype=I32, **z), st["free"],
                                st["head"], bs, nb, num_tokens=T + 2, context_lens_out=st["lens"],
                                free_head_out=st["head"])
    rows = torch.randn(T + 2, hq + 2 * hkv, D, generator=g).to(torch.bfloat16)
    d = rows.to(dev)
    pkv.paged_rope_append(d[:, :hq], d[:, hq:-hkv], d[:, -hkv:], r.positions, r.slot_mapping, freq, st["kc"], st["vc"],
                          k_scales=st["ks"], v_scales=st["vs"])
    starts = np.cumsum([0] + prompts)
    seen = [[rows[t, -hkv:] for t in range(starts[b], starts[b + 1])] for b in range(B)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # a warm-up on a copy of the state, then the capture
        warm = {k: v.clone() if torch.is_tensor(v) else v for k, v in st.items()}
        _model_step(pkv, warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _model_step(pkv, st)
    for step in range(8):
        x = torch.randn(B, hq + 2 * hkv, D, generator=g).to(torch.bfloat16)
        x[:, -hkv:] *= 2.0 ** (step - 4)  # the values' scales grow block by block
        st["qkv"].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        lens = [n + step + 1 if b < 4 else 0 for b, n in enumerate(prompts)]
        assert st["lens"].tolist() == lens and st["pos"].tolist() == [n - 1 for n in lens[:4]] + [-1]
        assert st["slots"].tolist()[-1] == -1
        for b in range(4):
            seen[b].append(x[b, -hkv:])
        want, bound = ref.decode_scaled(ref.f64(st["q"]), st["kc"].cpu().numpy(), st["vc"].cpu().numpy(),
                                        st["ks"].cpu().numpy(), st["vs"].cpu().numpy(), st["tables"].cpu().numpy(),
                                        lens, 0.1, bs, torch.bfloat16)
        assert np.all(np.abs(ref.f64(st["out"]) - want) <= bound)
        assert st["out"][4].count_nonzero() == 0
    # the values that the cache stands for are the tokens': half a code's step, 2^-4, or among the subnormal codes
    # 2^-10 of the block's scale for the token's own rounding and half as much again for each doubling before
    for b in range(4):
        t = st["tables"][b].cpu().numpy()
        for i, v in enumerate(seen[b]):
            sc = st["vs"].cpu().numpy()[t[i // bs]][:, None]
            got = ref.VALUES[st["vc"].cpu().numpy()[t[i // bs], :, i % bs]] * sc
            assert np.all(np.abs(got - ref.f64(v)) <= 2.0 ** -4 * np.abs(ref.f64(v)) + 2.0 ** -9 * sc)
