"""Chunk attention whose items are several blocks', joined by a kernel of its own, against the float64 statement: wide tables,
sequences that leave shares empty, windows, every cache, and values that are no numbers."""
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


def shares(pkv, seqs, tokens, hq, hkv, dim, width, bs):
    """Shares that the workspace of a call is sized for."""
    size = pkv._native.lib().pkv_chunk_workspace_size(seqs, tokens, hq, hkv, dim, width, bs)
    rows = tokens * hq
    fits = [s for s in range(2, 33) if size == 256 + -(-s * rows * 8 // 256) * 256 + s * rows * dim * 4]
    return fits[0] if fits else 1


def case(pkv, lens, new, hq, hkv, dim, act, cache="act", bs=16, width=512, window=None, sinks=0, seed=0, at_least=4, value=None,
         scales_from=(-8, -4), rows=None):
    """rows: the rows to check (None: all); value: what V of (sequence, token) is, which rows before it must not notice."""
    paged = ref.Paged(lens, hkv, bs, dim, act, cache, seed=seed, width=width, scales_from=scales_from)
    if value is not None:
        b, j, x = value
        blk, off = paged.slot(b, j)
        paged.v[blk, :, off] = x if cache == "act" else 0x7F
    starts = [0] + list(np.cumsum(new))
    assert shares(pkv, len(lens), starts[-1], hq, hkv, dim, width, bs) >= at_least
    q = torch.randn(starts[-1], hq, dim, generator=torch.Generator().manual_seed(seed + 1)).to(act)
    scale = dim ** -0.5
    args, scales = paged.cuda()
    out = torch.full(q.shape, 7.0, dtype=act).cuda()
    pkv.paged_attention_chunk(q.cuda(), *args, torch.tensor(starts, dtype=torch.int32).cuda(), scale, window=window, sinks=sinks,
                              out=out, **scales)
    for b, n in enumerate(lens):
        for i in range(new[b]):
            r = starts[b] + i
            if rows is None or r in rows:
                want, _, tol = ref.attend(paged, b, q[r], ref.visible(n - new[b] + i, window, sinks), scale)
                ref.check(out[r], want, tol, f"sequence {b}, row {i}")


@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("act", [F16, BF16])
def test_shares_of_every_cache(pkv, act, dim, cache):
    """A single token, drafts, a part of a prompt (two row tiles) and a sequence of one tile, most of whose shares are empty."""
    case(pkv, [1, 4200, 100, 2500], [1, 37, 5, 1], 8, 2, dim, act, cache, at_least=8, seed=dim)
    case(pkv, [4100, 200], [70, 3], 16, 2, dim, act, cache, bs=32, width=256, at_least=8, seed=dim + 1)


@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
@pytest.mark.parametrize("window,sinks", [(1024, 4), (3000, 0), (3000, 300), (2600, 2000)])
def test_shares_of_windows(pkv, window, sinks, cache):
    case(pkv, [4300, 40, 3050], [40, 7, 1], 4, 2, 128, BF16, cache, window=window, sinks=sinks, seed=sinks, at_least=8)
    case(pkv, [4500], [90], 2, 1, 64, F16, cache, window=window, sinks=sinks, seed=sinks + 1, at_least=8)


@pytest.mark.parametrize("act", [F16, BF16])
def test_shares_of_far_scales(pkv, act):
    """Block scales 2^40 apart: shares whose sums are in units of their own."""
    case(pkv, [4200, 90], [33, 2], 8, 2, 128, act, "scaled", scales_from=(-24, 2), at_least=8, seed=3)
    case(pkv, [4200], [1], 8, 2, 64, act, "scaled", scales_from=(-24, 2), at_least=8, seed=4)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("cache,window,sinks,value", [("act", None, 0, INF), ("act", 3000, 5, -INF), ("act", None, 0, NAN),
                                                      ("e4m3", None, 0, NAN), ("scaled", 3000, 5, NAN)])
def test_shares_with_a_value_that_is_no_number(pkv, cache, window, sinks, value):
    """Rows after a token whose V is no number see it, those before it are right: the item's rows one by one, in the share
    that has it alone."""
    case(pkv, [4200, 60], [60, 9], 4, 2, 128, BF16, cache, window=window, sinks=sinks, value=(0, 4165, value), at_least=8, seed=8)
    case(pkv, [4200], [60], 4, 2, 64, F16, cache, window=window, sinks=sinks, value=(0, 4140, value), at_least=8, seed=9)


@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
def test_shares_of_one_token(pkv, cache):
    """One token behind 32K over eight kv heads: nineteen shares."""
    case(pkv, [32765], [1], 32, 8, 64, BF16, cache, width=2048, at_least=19, seed=6)


def test_shares_of_many_rows(pkv):
    """More rows than one block's, two shares each, some of them checked."""
    case(pkv, [20000], [509], 32, 8, 64, F16, bs=32, width=1024, at_least=2, seed=7, rows={0, 1, 63, 64, 127, 255, 256, 508})
