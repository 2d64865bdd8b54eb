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
