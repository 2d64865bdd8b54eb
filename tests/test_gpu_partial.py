"""Chunk attention, windowed and scored decode and eviction against their float64 statements (tests/partial_ref.py)."""
import numpy as np
import pytest
import torch

from tests import partial_ref as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _clean(pkv_lib, cuda_device):
    pkv_lib.device_error()
    yield
    assert pkv_lib.device_error() == 0


def chunk_ref(paged, q, starts, scale, window=None, sinks=0):
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.ones(q.shape, dtype=torch.float64)
    for b, n in enumerate(paged.lens):
        new = starts[b + 1] - starts[b]
        for i in range(new):
            r = starts[b] + i
            out[r], _, tol[r] = ref.attend(paged, b, q[r], ref.visible(n - new + i, window, sinks), scale)
    return out, tol


def run_chunk(pkv, paged, q, starts, scale, window=None, sinks=0, **kw):
    args, scales = paged.cuda()
    return pkv.paged_attention_chunk(q.cuda(), *args, torch.tensor(starts, dtype=torch.int32).cuda(), scale,
                                     window=window, sinks=sinks, **scales, **kw)


def chunk_case(pkv, lens, new, hq, hkv, dim, bs, act, cache="act", window=None, sinks=0, seed=0, pad=0, width=None):
    paged = ref.Paged(lens, hkv, bs, dim, act, cache, seed=seed, width=width)
    starts = [0] + list(np.cumsum(new))
    if window is not None:  # what no row sees may hold anything, and its blocks' table entries too
        for b, (n, m) in enumerate(zip(lens, new)):
            if not m:
                continue
            gone = [j for j in range(sinks, max(0, n - m - window + 1))]
            paged.poison(b, gone)
            for i in range(-(-n // bs)):
                if gone and set(range(i * bs, (i + 1) * bs)) <= set(gone):
                    paged.tables[b, i] = -5
    q = torch.randn(starts[-1] + pad, hq, dim, generator=torch.Generator().manual_seed(seed + 1)).to(act)
    scale = dim ** -0.5
    out = torch.full((starts[-1] + pad, hq, dim), 7.0, dtype=act).cuda()
    got = run_chunk(pkv, paged, q, starts, scale, window, sinks, out=out)
    assert got is out
    assert torch.all(out[starts[-1]:] == 7.0)  # rows of no sequence
    want, tol = chunk_ref(paged, q[:starts[-1]], starts, scale, window, sinks)
    ref.check(out[:starts[-1]], want, tol, "chunk")


@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("act", [F16, BF16])
def test_chunk_types(pkv_lib, act, dim, cache):
    chunk_case(pkv_lib, [200, 37, 16, 129], [70, 37, 1, 5], 8, 2, dim, 16, act, cache, pad=3, seed=dim)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 12, 16, 33, 64])
def test_chunk_groups(pkv_lib, group):
    chunk_case(pkv_lib, [90, 41], [50, 2], 2 * group, 2, 64, 16, BF16, seed=group)


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 300])
def test_chunk_prompts(pkv_lib, n, bs):
    chunk_case(pkv_lib, [n], [n], 4, 2, 128, bs, BF16, seed=n)


@pytest.mark.parametrize("n,m", [(1000, 1), (1000, 2), (1000, 3), (513, 130), (640, 128), (640, 129), (900, 40)])
def test_chunk_after_a_prefix(pkv_lib, n, m):
    chunk_case(pkv_lib, [n, 64], [m, 0], 4, 4, 64, 32, F16, seed=m)
    chunk_case(pkv_lib, [n], [m], 16, 2, 128, 16, BF16, seed=m)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (16, 16), (128, 0), (129, 3), (100, 140), (4096, 4),
                                          (2 ** 31 - 1, 0), (40, 2 ** 31 - 1)])
@pytest.mark.parametrize("cache", ["act", "scaled"])
def test_chunk_windows(pkv_lib, window, sinks, cache):
    chunk_case(pkv_lib, [400, 33, 260], [150, 33, 1], 4, 2, 128, 16, BF16, cache, window, sinks, seed=window % 97)
    chunk_case(pkv_lib, [500], [260], 2, 2, 64, 32, F16, cache, window, sinks, seed=window % 89)


def test_chunk_mixed_batch(pkv_lib):
    new = [1, 0, 33, 1, 1, 5, 128, 1, 0, 2]
    lens = [300, 0, 33, 1, 64, 200, 300, 17, 40, 2]
    chunk_case(pkv_lib, lens, new, 8, 2, 128, 16, BF16, pad=9, width=40)
    chunk_case(pkv_lib, lens, new, 8, 8, 64, 16, F16, "scaled", pad=1, width=40)


def test_chunk_rows_apart(pkv_lib):
    """q as a part of a projection's output, out as a part of a wider buffer, a first row behind others."""
    paged = ref.Paged([50, 20], 2, 16, 64, BF16)
    starts = [3, 33, 35]
    wide = torch.randn(40, 3 * 8 * 64, generator=torch.Generator().manual_seed(1)).to(BF16)
    q = wide[:, 512:1024].unflatten(1, (8, 64))
    out = torch.full((40, 1040), 3.0, dtype=BF16).cuda()
    args, scales = paged.cuda()
    pkv_lib.paged_attention_chunk(wide.cuda()[:, 512:1024].unflatten(1, (8, 64)), *args,
                                  torch.tensor(starts, dtype=torch.int32).cuda(), 0.125,
                                  out=out[:, 8:520].unflatten(1, (8, 64)))
    want, tol = chunk_ref(paged, q, starts, 0.125)
    ref.check(out[3:35, 8:520].unflatten(1, (8, 64)), want[3:35], tol[3:35])
    out[3:35, 8:520] = 3.0
    assert torch.all(out == 3.0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window,sinks", [(None, 0), (40, 3)])
def test_chunk_rows_do_not_see_later_tokens(pkv_lib, value, window, sinks):
    """A token whose K and V are no numbers reaches the rows that see it alone."""
    lens, new, at = [300], [260], 170
    paged = ref.Paged(lens, 2, 16, 128, BF16, seed=5)
    q = torch.randn(260, 4, 128, generator=torch.Generator().manual_seed(6)).to(BF16)
    want, tol = chunk_ref(paged, q, [0, 260], 0.09, window, sinks)
    blk, off = paged.slot(0, at)
    paged.v[blk, :, off, 5:9] = value
    got = run_chunk(pkv_lib, paged, q, [0, 260], 0.09, window, sinks).cpu()
    sees = torch.tensor([at in ref.visible(40 + i, window, sinks) for i in range(260)])
    ref.check(got[~sees], want[~sees], tol[~sees], "rows that do not see it")
    assert not torch.isfinite(got[sees][..., 5:9]).any()
    ref.check(got[sees][..., :5], want[sees][..., :5], tol[sees][..., :5], "its other channels")
    paged.k[blk, :, off] = value
    got = run_chunk(pkv_lib, paged, q, [0, 260], 0.09, window, sinks).cpu()
    ref.check(got[~sees], want[~sees], tol[~sees], "rows that do not see it")


@pytest.mark.parametrize("factor", [1e-4, 30.0, 200.0])
def test_chunk_logits_of_any_size(pkv_lib, factor):
    paged = ref.Paged([333], 2, 16, 128, BF16, seed=8)
    q = (torch.randn(200, 4, 128, generator=torch.Generator().manual_seed(9)) * factor).to(BF16)
    want, tol = chunk_ref(paged, q, [0, 200], 0.0884)
    ref.check(run_chunk(pkv_lib, paged, q, [0, 200], 0.0884), want, tol)


def test_chunk_same_as_decode(pkv_lib):
    """One new token each: what the decode gives, within both roundings."""
    lens = [5, 100, 257, 700]
    paged = ref.Paged(lens, 4, 16, 128, BF16, seed=3)
    q = torch.randn(4, 16, 128, generator=torch.Generator().manual_seed(4)).to(BF16)
    args, _ = paged.cuda()
    a = run_chunk(pkv_lib, paged, q, [0, 1, 2, 3, 4], 0.1)
    b = pkv_lib.paged_attention_decode(q.cuda(), *args, 0.1)
    _, tol = chunk_ref(paged, q, [0, 1, 2, 3, 4], 0.1)
    assert torch.all((a.cpu().double() - b.cpu().double()).abs() <= 2 * tol)


def test_chunk_bad_sequences_are_flagged_and_left(pkv_lib):
    paged = ref.Paged([64, 64, 64], 2, 16, 64, F16)
    q = torch.randn(12, 4, 64, generator=torch.Generator().manual_seed(4)).to(F16)
    starts = [0, 4, 8, 12]
    want, tol = chunk_ref(paged, q, starts, 0.125)
    for bad, rows in (([64, 3, 64], (4, 8)), ([64, 65, 64], (4, 8)), ([-1, 64, 64], (0, 4))):
        args, _ = paged.cuda()
        out = torch.full((12, 4, 64), 7.0, dtype=F16).cuda()
        pkv_lib.paged_attention_chunk(q.cuda(), *args[:3], torch.tensor(bad, dtype=torch.int32).cuda(),
                                      torch.tensor(starts, dtype=torch.int32).cuda(), 0.125, out=out)
        assert pkv_lib.device_error() == pkv_lib.DEV_BAD_CONTEXT_LEN
        assert torch.all(out[rows[0]:rows[1]] == 7.0)
        keep = [r for r in range(12) if not rows[0] <= r < rows[1]]
        ref.check(out[keep], want[keep], tol[keep])
    args, _ = paged.cuda()
    for bad in ([0, 4, 8, 13], [-1, 4, 8, 12], [0, 4, 2, 12]):
        out = torch.full((12, 4, 64), 7.0, dtype=F16).cuda()
        pkv_lib.paged_attention_chunk(q.cuda(), *args, torch.tensor(bad, dtype=torch.int32).cuda(), 0.125, out=out)
        assert pkv_lib.device_error() & pkv_lib.DEV_BAD_CONTEXT_LEN
    args[2][1, 2] = 10 ** 6
    pkv_lib.paged_attention_chunk(q.cuda(), *args, torch.tensor(starts, dtype=torch.int32).cuda(), 0.125)
    assert pkv_lib.device_error() == pkv_lib.DEV_BAD_BLOCK


# --------------------------------------------------------------------------- windowed decode
def window_case(pkv, lens, hq, hkv, dim, bs, act, cache, window, sinks, seed=0, width=None, **kw):
    paged = ref.Paged(lens, hkv, bs, dim, act, cache, seed=seed, width=width)
    q = torch.randn(len(lens), hq, dim, generator=torch.Generator().manual_seed(seed + 1)).to(act)
    scale = dim ** -0.5
    want, tol = torch.zeros(q.shape, dtype=torch.float64), torch.full(q.shape, 1e-9, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n:
            want[b], _, tol[b] = ref.attend(paged, b, q[b], ref.visible(n - 1, window, sinks), scale)
    for b, n in enumerate(lens):  # hidden tokens hold anything, the entries of their blocks too
        gone = list(range(sinks, n - window))
        paged.poison(b, gone)
        for i in range(-(-n // bs)):
            if gone and set(range(i * bs, (i + 1) * bs)) <= set(gone):
                paged.tables[b, i] = -5
    args, scales = paged.cuda()
    got = pkv.paged_attention_decode_window(q.cuda(), *args, scale, window, sinks=sinks, **scales, **kw)
    ref.check(got, want, tol, "window")


LENS = [1, 2, 15, 16, 17, 31, 33, 64, 100, 0, 129, 300, 511, 513, 700]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 17), (16, 16), (33, 4), (64, 0), (500, 20), (1000, 5),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (31, 2 ** 31 - 1)])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
def test_window(pkv_lib, cache, group, window, sinks):
    window_case(pkv_lib, LENS, 2 * group, 2, 128, 16, BF16, cache, window, sinks, seed=group)


@pytest.mark.parametrize("act,dim,hkv,bs", [(F16, 64, 2, 16), (F16, 64, 3, 32), (F16, 128, 1, 32), (BF16, 64, 4, 32)])
@pytest.mark.parametrize("group", [1, 4, 8])
@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
def test_window_layouts(pkv_lib, cache, group, act, dim, hkv, bs):
    window_case(pkv_lib, LENS, hkv * group, hkv, dim, bs, act, cache, 90, 19, seed=bs, width=60)


@pytest.mark.parametrize("partition_size", [0, 32, 256, 512])
@pytest.mark.parametrize("cache", ["act", "scaled"])
@pytest.mark.parametrize("group", [1, 4])
def test_window_partitions(pkv_lib, group, cache, partition_size):
    for window, sinks in ((300, 40), (10, 33), (260, 0)):
        window_case(pkv_lib, [2000, 40, 1200, 295, 31], 2 * group, 2, 128, 32, BF16, cache, window, sinks,
                    partition_size=partition_size)


def test_window_many_rows(pkv_lib):
    """More sequences than one tensor-core launch takes."""
    lens = [(37 * i) % 200 for i in range(600)]
    window_case(pkv_lib, lens, 8, 2, 64, 16, F16, "act", 50, 3, seed=2)
    window_case(pkv_lib, lens, 4, 1, 128, 16, BF16, "scaled", 50, 3, seed=3)


# --------------------------------------------------------------------------- scored decode
@pytest.mark.parametrize("cache", ["act", "e4m3"])
@pytest.mark.parametrize("act,dim,hkv,group,bs", [(BF16, 128, 2, 1, 16), (BF16, 128, 2, 8, 16), (F16, 128, 1, 4, 32),
                                                  (F16, 64, 2, 4, 16), (BF16, 64, 3, 8, 32), (BF16, 64, 4, 2, 16)])
@pytest.mark.parametrize("partition_size", [-1, 64, 0])
def test_scored(pkv_lib, act, dim, hkv, group, bs, cache, partition_size):
    lens = [1, 40, 0, 513, 17, 1100]
    paged = ref.Paged(lens, hkv, bs, dim, act, cache, seed=dim + group)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(len(lens), hkv * group, dim, generator=g).to(act)
    tokens = paged.tables.shape[1] * bs
    before = torch.rand(len(lens), hkv, tokens + 5, generator=g)
    scores = before.cuda()
    args, scales = paged.cuda()
    scales = {k: scales[k] for k in ("k_scale", "v_scale")}
    out = pkv_lib.paged_attention_decode_scored(q.cuda(), *args, 0.1, scores, partition_size=partition_size, **scales)
    again = before.cuda()
    pkv_lib.paged_attention_decode_scored(q.cuda(), *args, 0.1, again, partition_size=partition_size, **scales)
    assert torch.equal(scores, again)  # the same sums every time
    want, tol = torch.zeros(q.shape, dtype=torch.float64), torch.full(q.shape, 1e-9, dtype=torch.float64)
    sums = before.double()
    for b, n in enumerate(lens):
        if n:
            want[b], p, tol[b] = ref.attend(paged, b, q[b], list(range(n)), 0.1)
            sums[b, :, :n] += p.view(hkv, group, n).sum(1)
    ref.check(out, want, tol, "scored")
    # a weight moves by e^(2d) - 1 with d as in attend(); logits here are below 16, their magnitudes' sums below 64
    # (2^-11 with E4M3's queries in parts, 2^-18 of the largest element per product)
    rel = 2.0 ** -10 if cache == "act" else 2.0 ** -8
    ref.check(scores, sums, rel * (sums - before.double()) + 2.0 ** -20 * (1 + sums), "scores")
    for b, n in enumerate(lens):
        assert torch.equal(scores[b, :, n:].cpu(), before[b, :, n:])


# --------------------------------------------------------------------------- eviction
def evict_case(pkv, lens, hkv, bs, dim, act, cache, budget, recent, sinks, seed=0, make=None, out_tokens=None):
    rng = np.random.default_rng(seed)
    paged = ref.Paged(lens, hkv, bs, dim, act, cache, seed=seed, extra_blocks=3 + sum(-(-min(n, budget) // bs) for n in lens))
    tokens = paged.tables.shape[1] * bs
    scores = rng.lognormal(size=(len(lens), hkv, tokens)).astype(np.float32)
    if make is not None:
        make(scores, rng)
    room = [-(-min(n, budget) // bs) for n in lens]
    dst = torch.full((len(lens), max(1, max(room))), -1, dtype=torch.int32)
    at = 0
    for b, r in enumerate(room):
        dst[b, :r] = paged.free[at:at + r]
        at += r
    args, _ = paged.cuda()
    dev = torch.from_numpy(scores).cuda()
    kw = {} if out_tokens is None else dict(scores_out=torch.full((len(lens), hkv, out_tokens), 9.0).cuda())
    got = pkv.paged_kv_evict(args[0], args[1], dev, args[2], args[3], dst.cuda(), budget, recent, sinks=sinks, **kw)
    assert torch.equal(dev.cpu(), torch.from_numpy(scores)) or np.isnan(scores).any()
    k, v = args[0].cpu(), args[1].cpu()
    assert got.context_lens.tolist() == [min(n, budget) for n in lens]
    new_k, new_v = paged.k.clone(), paged.v.clone()
    kept, moved = got.kept.cpu().numpy(), got.scores.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(hkv):
            stay = ref.evict(scores[b, h], n, budget, recent, sinks)
            assert kept[b, h].tolist() == stay + [-1] * (budget - len(stay))
            np.testing.assert_array_equal(moved[b, h, :len(stay)], scores[b, h, stay])
            assert not moved[b, h, len(stay):].any()
            for i, j in enumerate(stay):
                blk, off = paged.slot(b, j)
                to = int(dst[b, i // bs])
                new_k[to, h, i % bs], new_v[to, h, i % bs] = paged.k[blk, h, off], paged.v[blk, h, off]
    bits = torch.uint8 if cache != "act" else torch.int16
    assert torch.equal(k.view(bits), new_k.view(bits)) and torch.equal(v.view(bits), new_v.view(bits))


@pytest.mark.parametrize("cache", ["act", "e4m3"])
@pytest.mark.parametrize("dim,bs", [(64, 16), (128, 32)])
@pytest.mark.parametrize("budget,recent,sinks", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (33, 10, 3), (64, 64, 0), (64, 30, 34),
                                                 (100, 0, 0), (600, 5, 5)])
def test_evict(pkv_lib, budget, recent, sinks, dim, bs, cache):
    evict_case(pkv_lib, [0, 1, 33, 34, 64, 65, 99, 500, 311], 3, bs, dim, BF16, cache, budget, recent, sinks, seed=budget)


def ties(scores, rng):
    scores[:] = rng.integers(0, 3, scores.shape)


def zeros(scores, rng):
    scores[:] = np.where(rng.random(scores.shape) < 0.5, 0.0, -0.0)


def odd_values(scores, rng):
    flat = scores.reshape(-1)
    for i, x in enumerate((np.nan, np.inf, -np.inf, -1.0, 1e-40, -1e-40, 3e38)):
        flat[rng.random(flat.size) < 0.08] = x


@pytest.mark.parametrize("make", [ties, zeros, odd_values])
def test_evict_scores_of_any_kind(pkv_lib, make):
    for budget, recent, sinks in ((50, 7, 2), (200, 0, 0), (120, 100, 0)):
        evict_case(pkv_lib, [400, 201, 50, 121], 2, 16, 64, F16, "act", budget, recent, sinks, seed=4, make=make)


def test_evict_long_rows(pkv_lib):
    """More than one turn of the ordered pass, and rows longer than the keys that fit shared memory."""
    evict_case(pkv_lib, [9000, 4097], 1, 16, 64, F16, "act", 4100, 64, 4, seed=1)
    evict_case(pkv_lib, [50000, 49153], 1, 32, 64, F16, "act", 1000, 64, 4, seed=2, make=ties)


def test_evict_output_widths(pkv_lib):
    evict_case(pkv_lib, [100, 20], 2, 16, 64, F16, "act", 32, 4, 4, out_tokens=32)
    evict_case(pkv_lib, [100, 20], 2, 16, 64, F16, "act", 32, 4, 4, out_tokens=500)


def test_evict_bad_rows(pkv_lib):
    paged = ref.Paged([64, 64, 64], 1, 16, 64, F16, extra_blocks=12)
    args, _ = paged.cuda()
    dst = paged.free[:6].view(3, 2).to(torch.int32).cuda()
    scores = torch.rand(3, 1, 64).cuda()
    k0 = args[0].clone()
    got = pkv_lib.paged_kv_evict(args[0], args[1], scores, args[2], torch.tensor([64, 65, -1], dtype=torch.int32).cuda(),
                                 dst, 32, 4)
    assert pkv_lib.device_error() == pkv_lib.DEV_BAD_CONTEXT_LEN
    assert got.context_lens.tolist() == [32, 0, 0]
    assert not got.scores[1:].any() and torch.all(got.kept[1:] == -1)
    touched = dst[0].long().cpu()
    keep = [i for i in range(k0.shape[0]) if i not in touched.tolist()]
    assert torch.equal(args[0][keep].view(torch.int16), k0[keep].view(torch.int16))
    got = pkv_lib.paged_kv_evict(args[0], args[1], scores, args[2], args[3], dst[:, :1].contiguous(), 32, 4)
    assert pkv_lib.device_error() == pkv_lib.DEV_NO_SPACE and got.context_lens.tolist() == [0, 0, 0]
    dst[1, 1] = 10 ** 6
    pkv_lib.paged_kv_evict(args[0], args[1], scores, args[2], args[3], dst, 32, 4)
    assert pkv_lib.device_error() == pkv_lib.DEV_BAD_BLOCK


# --------------------------------------------------------------------------- together
def test_bounded_cache_together(pkv_lib):
    """A prompt in chunks, scored steps, an eviction through the block manager, and windowed steps after it."""
    hq, hkv, bs, dim, budget = 8, 2, 16, 64, 48
    g = torch.Generator().manual_seed(0)
    paged = ref.Paged([100], hkv, bs, dim, F16, seed=7, extra_blocks=9)
    args, _ = paged.cuda()
    q = torch.randn(100, hq, dim, generator=g).to(F16)
    scale = dim ** -0.5
    for lo, hi in ((0, 60), (60, 100)):  # the prompt in two parts
        got = pkv_lib.paged_attention_chunk(q[lo:hi].cuda(), *args[:3], torch.tensor([hi], dtype=torch.int32).cuda(),
                                            torch.tensor([0, hi - lo], dtype=torch.int32).cuda(), scale)
        part = ref.Paged([100], hkv, bs, dim, F16, seed=7, extra_blocks=9)
        part.lens = [hi]
        want, tol = chunk_ref(part, q[lo:hi], [0, hi - lo], scale)
        ref.check(got, want, tol)
    scores = torch.zeros(1, hkv, args[2].shape[1] * bs).cuda()
    sums = np.zeros((hkv, 100))
    for i in range(3):
        qi = torch.randn(1, hq, dim, generator=g).to(F16)
        pkv_lib.paged_attention_decode_scored(qi.cuda(), *args, scale, scores)
        _, p, _ = ref.attend(paged, 0, qi[0], list(range(100)), scale)
        sums += p.view(hkv, -1, 100).sum(1).numpy()
    np.testing.assert_allclose(scores[0, :, :100].cpu().numpy(), sums, rtol=2e-4)
    dst = paged.free[:3].view(1, 3).to(torch.int32)
    got = pkv_lib.paged_kv_evict(args[0], args[1], scores, args[2], args[3], dst.cuda(), budget, 16, sinks=2)
    stay = got.kept.cpu()
    qi = torch.randn(1, hq, dim, generator=g).to(F16)
    out = pkv_lib.paged_attention_decode_window(qi.cuda(), args[0], args[1], dst.cuda(), got.context_lens, scale, 20,
                                                sinks=4)
    for h in range(hkv):
        seen = [int(stay[0, h, i]) for i in ref.visible(budget - 1, 20, 4)]
        want, _, tol = ref.attend(paged, 0, qi[0], seen, scale)
        rows = slice(h * hq // hkv, (h + 1) * hq // hkv)
        ref.check(out[0, rows], want[rows], tol[rows])


# --------------------------------------------------------------------------- sizes and values at the edge
@pytest.mark.parametrize("scale", [0.0, -0.11])
@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
def test_chunk_scale_of_any_sign(pkv_lib, cache, scale):
    paged = ref.Paged([300, 20], 2, 16, 128, BF16, cache, seed=11)
    q = torch.randn(153, 8, 128, generator=torch.Generator().manual_seed(12)).to(BF16)
    want, tol = chunk_ref(paged, q, [0, 150, 153], scale)
    ref.check(run_chunk(pkv_lib, paged, q, [0, 150, 153], scale), want, tol)


@pytest.mark.parametrize("bad_v", [False, True], ids=["V finite", "V not finite"])
def test_chunk_logits_of_minus_infinity(pkv_lib, bad_v):
    """Tokens whose logits are -inf weigh nothing, the first ones of a row among them."""
    paged = ref.Paged([200], 2, 16, 64, F16, seed=13)
    q = torch.randn(170, 4, 64, generator=torch.Generator().manual_seed(14)).to(F16)
    q[..., 3] = q[..., 3].abs() + 0.01
    for j in list(range(20)) + [40, 100]:
        blk, off = paged.slot(0, j)
        paged.k[blk, :, off, 3] = -float("inf")
    want, tol = chunk_ref(paged, q, [0, 170], 0.125)
    tol = torch.nan_to_num(tol, nan=1.0, posinf=1.0)  # (the magnitudes' sums are infinite)
    sums = torch.zeros_like(want)  # so they are taken over the tokens that weigh something
    for i in range(170):
        js = [j for j in range(30 + i + 1) if j >= 20 and j not in (40, 100)]
        sums[i], _, tol[i] = ref.attend(paged, 0, q[i], js, 0.125)
    assert torch.equal(torch.isfinite(want), torch.ones_like(want, dtype=torch.bool))
    sees = torch.zeros(170, dtype=torch.bool)
    if bad_v:
        blk, off = paged.slot(0, 150)
        paged.v[blk, :, off] = float("nan")
        sees = torch.arange(170) + 30 >= 150
    got = run_chunk(pkv_lib, paged, q, [0, 170], 0.125).cpu()
    ref.check(got[~sees], sums[~sees], tol[~sees])
    assert not torch.isfinite(got[sees]).any()


def test_chunk_rows_do_not_see_later_scales(pkv_lib):
    """A block whose scales are no numbers reaches the rows that see it alone."""
    paged = ref.Paged([300], 2, 16, 128, BF16, "scaled", seed=5)
    q = torch.randn(260, 4, 128, generator=torch.Generator().manual_seed(6)).to(BF16)
    want, tol = chunk_ref(paged, q, [0, 260], 0.09)
    blk, _ = paged.slot(0, 176)
    sees = torch.arange(260) + 40 >= 176
    for value in (float("inf"), float("nan")):
        for scales in (paged.v_scales, paged.k_scales):
            old = scales[blk].clone()
            scales[blk] = value
            got = run_chunk(pkv_lib, paged, q, [0, 260], 0.09).cpu()
            scales[blk] = old
            ref.check(got[~sees], want[~sees], tol[~sees], "rows that do not see it")


@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (8, 2, 64), (2, 2, 64)])
def test_scored_many_rows(pkv_lib, hq, hkv, dim):
    """More sequences than one tensor-core launch takes."""
    lens = [(37 * i) % 200 for i in range(600)]
    paged = ref.Paged(lens, hkv, 16, dim, BF16, seed=21)
    q = torch.randn(600, hq, dim, generator=torch.Generator().manual_seed(22)).to(BF16)
    args, _ = paged.cuda()
    tokens = paged.tables.shape[1] * 16
    scores = torch.zeros(600, hkv, tokens).cuda()
    out = pkv_lib.paged_attention_decode_scored(q.cuda(), *args, 0.1, scores, partition_size=64)
    want, tol = torch.zeros(q.shape, dtype=torch.float64), torch.full(q.shape, 1e-9, dtype=torch.float64)
    sums = torch.zeros(scores.shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n:
            want[b], p, tol[b] = ref.attend(paged, b, q[b], list(range(n)), 0.1)
            sums[b, :, :n] = p.view(hkv, hq // hkv, n).sum(1)
    ref.check(out, want, tol, "scored")
    ref.check(scores, sums, 2.0 ** -10 * sums + 2.0 ** -20 * (1 + sums), "scores")  # as in test_scored


@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
def test_blocks_past_32_bits(pkv_lib, cache):
    """Pools whose last blocks lie behind 2^32 elements: what the same blocks at the front give, bit for bit."""
    hkv, bs, dim = 8, 32, 128
    paged = ref.Paged([700, 61], hkv, bs, dim, BF16, cache, seed=31, extra_blocks=8)
    q = torch.randn(90, 4 * hkv, dim, generator=torch.Generator().manual_seed(32)).to(BF16).cuda()
    (k, v, tables, lens), scales = paged.cuda()
    blocks = 2 ** 32 // (hkv * bs * dim) + 64
    shift = blocks - k.shape[0]
    K, V = (torch.empty((blocks, *k.shape[1:]), dtype=k.dtype, device="cuda") for _ in range(2))
    K[shift:], V[shift:] = k, v
    far = torch.where(tables >= 0, tables + shift, tables)
    Scales = dict(scales)
    for name in ("k_scales", "v_scales"):
        if scales[name] is not None:
            Scales[name] = torch.ones(blocks, hkv, device="cuda")
            Scales[name][shift:] = scales[name]
    starts = torch.tensor([0, 80, 90], dtype=torch.int32).cuda()
    a, b = (pkv_lib.paged_attention_chunk(q, *pools, lens, starts, 0.09, **s)
            for pools, s in (((k, v, tables), scales), ((K, V, far), Scales)))
    assert torch.equal(a, b)
    a, b = (pkv_lib.paged_attention_decode_window(q[:2], *pools, lens, 0.09, 300, sinks=5, **s)
            for pools, s in (((k, v, tables), scales), ((K, V, far), Scales)))
    assert torch.equal(a, b)
    if cache == "scaled":
        return
    one = {n: scales[n] for n in ("k_scale", "v_scale")}
    sums = [torch.zeros(2, hkv, tables.shape[1] * bs).cuda() for _ in range(2)]
    a, b = (pkv_lib.paged_attention_decode_scored(q[:2], *pools, lens, 0.09, s, **one)
            for pools, s in zip(((k, v, tables), (K, V, far)), sums))
    assert torch.equal(a, b) and torch.equal(*sums)
    dst = paged.free[:8].view(2, 4).to(torch.int32).cuda()
    a = pkv_lib.paged_kv_evict(k, v, sums[0], tables, lens, dst, 128, 32, sinks=4)
    b = pkv_lib.paged_kv_evict(K, V, sums[1], far, lens, dst + shift, 128, 32, sinks=4)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    bits = torch.uint8 if cache != "act" else torch.int16
    assert torch.equal(k.view(bits), K[shift:].view(bits)) and torch.equal(v.view(bits), V[shift:].view(bits))


def test_no_rows(pkv_lib):
    """Calls over no sequences and over no tokens do nothing."""
    paged = ref.Paged([20], 2, 16, 64, F16)
    (k, v, tables, lens), _ = paged.cuda()
    none, empty = tables[:0], lens[:0]
    q = torch.empty(0, 4, 64, dtype=F16, device="cuda")
    assert pkv_lib.paged_attention_chunk(q, k, v, tables, lens, torch.zeros(2, dtype=torch.int32).cuda(), 1.0).shape == q.shape
    assert pkv_lib.paged_attention_chunk(q, k, v, none, empty, torch.zeros(1, dtype=torch.int32).cuda(), 1.0).shape == q.shape
    out = torch.full((3, 4, 64), 2.0, dtype=F16).cuda()
    rows = torch.zeros(3, 4, 64, dtype=F16).cuda()
    pkv_lib.paged_attention_chunk(rows, k, v, tables, lens, torch.zeros(2, dtype=torch.int32).cuda(), 1.0, out=out)
    assert torch.all(out == 2.0)
    assert pkv_lib.paged_attention_decode_window(q, k, v, none, empty, 1.0, 5).shape == q.shape
    scores = torch.zeros(0, 2, tables.shape[1] * 16).cuda()
    assert pkv_lib.paged_attention_decode_scored(q, k, v, none, empty, 1.0, scores).shape == q.shape
    assert pkv_lib.paged_kv_evict(k, v, scores, none, empty, none, 4, 1).kept.shape == (0, 2, 4)
