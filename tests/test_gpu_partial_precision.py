"""Chunk attention, windowed and scored decode keep what the outputs' type can hold, where weights and contexts are such
that parts of few bits would show.

The bounds are those of tests/partial_ref.py with w, what a weight's rounding may take, of the outputs' type: half a step,
2^-11 for binary16 (weights in three E4M3 parts keep 2^-14 of themselves, weights in binary32 all)."""
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


def narrow(paged, b, q, js, scale):
    """partial_ref.attend with the bound of the outputs' type for the weights: (out, weights, bound of a logit's error, of the output's)."""
    out, p, _ = ref.attend(paged, b, q, js, scale)
    k, v = paged.tokens(b, js)
    dim = q.shape[-1]
    qd = q.double().view(paged.hkv, -1, dim)
    a = (p.view(paged.hkv, -1, len(js)) @ v.abs()).reshape(out.shape)
    top = abs(scale) * (qd.abs() @ k.abs().transpose(1, 2)).amax((-1, -2))
    d = 2.0 ** -17 * top.clamp(min=1.0)
    if paged.cache != "act":
        d = d + abs(scale) * 2.0 ** -18 * qd.abs().amax((1, 2)) * k.abs().sum(-1).amax(-1)
    d = d.repeat_interleave(q.shape[0] // paged.hkv)[:, None]
    u = ref.U[paged.act]
    return out, p, d, u * out.abs() + (u + 2.0 ** -14 + 2 * d) * a + 1e-6


@pytest.mark.parametrize("act", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_weights_over_one_scale(pkv, group, dim, act):
    """Few tokens of comparable weights over a per-tensor E4M3 cache: nothing averages a weight's error away."""
    lens = [2, 3, 4, 5, 7, 9, 17, 33] * 4
    paged = ref.Paged(lens, 2, 16, dim, act, "e4m3", seed=group)
    args, scales = paged.cuda()
    g = torch.Generator().manual_seed(dim + group)
    q = torch.randn(len(lens), 2 * group, dim, generator=g).to(act)
    scale = dim ** -0.5
    one = dict(k_scale=scales["k_scale"], v_scale=scales["v_scale"])
    win = pkv.paged_attention_decode_window(q.cuda(), *args, scale, 30, sinks=1, **one)
    scores = torch.zeros(len(lens), 2, 48).cuda()
    out = pkv.paged_attention_decode_scored(q.cuda(), *args, scale, scores, **one)
    for b, n in enumerate(lens):
        want, _, _, tol = narrow(paged, b, q[b], ref.visible(n - 1, 30, 1), scale)
        ref.check(win[b], want, tol, f"window {n}")
        want, p, d, tol = narrow(paged, b, q[b], list(range(n)), scale)
        ref.check(out[b], want, tol, f"scored {n}")
        got = scores[b, :, :n].double().cpu()
        off = ((2 * d + 2.0 ** -20) * p).view(2, group, n).sum(1)  # the logits' errors, the exponential's
        assert torch.all((got - p.view(2, group, n).sum(1)).abs() <= off + 1e-6)


def one_of_many(n, act, cache, gap, bs=16, dim=64, hkv=1):
    """A sequence of n tokens: logit `gap` (log2) and V = 0 for the first, logit 0 and V = 1 for the others, for a query
    whose first channel alone is 1.  Returns it and the call's scale."""
    paged = ref.Paged([n], hkv, bs, dim, act, cache, extra_blocks=0)
    k, v = torch.zeros(paged.k.shape), torch.ones(paged.v.shape)
    blk, off = paged.slot(0, 0)
    k[blk, :, off, 0] = 1.0
    v[blk, :, off] = 0.0
    paged.k, paged.v = (x.to(act) if cache == "act" else paged._codes(x) for x in (k, v))
    if cache == "e4m3":
        paged.k_scale, paged.v_scale = torch.ones(1), torch.ones(1)
    if cache == "scaled":
        paged.k_scales, paged.v_scales = torch.ones_like(paged.k_scales), torch.ones_like(paged.v_scales)
    return paged, gap * 0.6931471805599453


def small_weights(n, gap, act, least=2.0 ** -32):
    """Output of n tokens of 2^-gap beside one of weight 1 and V = 0, and what it may be off by: the output's and a weight's
    half step (a weight below 2^-21 of the largest: 2^-32 of that; an output that is a subnormal binary16 value: half of
    2^-24), the logit of the first token in float32 (2^-17 of it), and 2^-14 of the sum for float32 sums.

    Weights in three E4M3 parts, the block-scaled kernel's on the tensor cores: least = 2^-28.  A weight times 2^8 is a sum
    of codes, 2^-5 of codes and 2^-10 of codes, each part the nearest code to 2^5 times what the part before left; codes
    below 2^-6 are 2^-9 apart, so the last part leaves up to 2^-10, which counts 2^-10 * 2^-10 * 2^-8 of the largest."""
    x = n * 2.0 ** -gap
    o = x / (1 + x)
    u = ref.U[act]
    return o, (2 * u + 2.0 ** -14 + 2.0 ** -16 * gap) * o + n * least + (2.0 ** -25 if act is F16 else 0.0)


@pytest.mark.parametrize("gap", [15.7, 19.1, 21.6, 25.2])
@pytest.mark.parametrize("new", [1, 200], ids=["folded", "two row tiles"])
@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
@pytest.mark.parametrize("act", [F16, BF16])
def test_chunk_small_weights(pkv, act, cache, new, gap):
    """A first token that has nearly all the weight and no V: the output is what the others' small weights make it."""
    n, dim = 4000, 64
    paged, scale = one_of_many(n, act, cache, gap, dim=dim)
    args, scales = paged.cuda()
    q = torch.zeros(new, 1, dim, dtype=act)
    q[..., 0] = 1.0
    out = pkv.paged_attention_chunk(q.cuda(), *args, torch.tensor([0, new], dtype=torch.int32).cuda(), scale, **scales)
    for i in range(new):
        want, tol = small_weights(n - new + i, gap, act)
        assert torch.all((out[i].double() - want).abs() <= tol), (i, want, tol)


@pytest.mark.parametrize("gap", [15.7, 21.6, 25.2])
@pytest.mark.parametrize("group,dim", [(1, 64), (2, 128), (4, 64), (8, 128)])
@pytest.mark.parametrize("cache", ["act", "e4m3", "scaled"])
@pytest.mark.parametrize("act", [F16, BF16])
def test_decode_small_weights(pkv, act, cache, group, dim, gap):
    """The same for one row, under a window with the first token in front of it and scored, and the weights added."""
    n, hkv = 1300, 2
    paged, scale = one_of_many(n, act, cache, gap, dim=dim, hkv=hkv)
    args, scales = paged.cuda()
    q = torch.zeros(1, hkv * group, dim, dtype=act).cuda()
    q[..., 0] = 1.0
    least = 2.0 ** -28 if cache == "scaled" or (cache == "e4m3" and group >= 4) else 2.0 ** -32
    for part in (-1, 0):  # of the library's choice, and one
        out = pkv.paged_attention_decode_window(q, *args, scale, 1000, sinks=1, partition_size=part, **scales)
        want, tol = small_weights(1000, gap, act, least)
        assert torch.all((out.double() - want).abs() <= tol), (part, want, tol)
        if cache == "scaled":
            continue
        scores = torch.zeros(1, hkv, paged.tables.shape[1] * 16).cuda()
        one = dict(k_scale=scales["k_scale"], v_scale=scales["v_scale"])
        out = pkv.paged_attention_decode_scored(q, *args, scale, scores, partition_size=part, **one)
        want, tol = small_weights(n - 1, gap, act, least)
        assert torch.all((out.double() - want).abs() <= tol), (part, want, tol)
        p = group * 2.0 ** -gap / (1 + (n - 1) * 2.0 ** -gap)
        off = (2.0 ** -16 * gap + 2.0 ** -14) * p
        assert torch.all((scores[0, :, 1:n].double() - p).abs() <= off)
