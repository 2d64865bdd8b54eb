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


def small_weights(n, gap, u):
    """Output of n tokens of 2^-gap beside one of weight 1 and V = 0, and what it may be off by: the output's and a weight's
    half step (a weight below 2^-21 of the largest: 2^-32 of that), the logit of the first token in float32 (2^-17 of it),
    and 2^-14 of the sum for float32 sums."""
    x = n * 2.0 ** -gap
    o = x / (1 + x)
    return o, (2 * u + 2.0 ** -14 + 2.0 ** -16 * gap) * o + n * 2.0 ** -32


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
        want, tol = small_weights(n - new + i, gap, ref.U[act])
        assert torch.all((out[i].double() - want).abs() <= tol), (i, want, tol)
