"""Float64 statements of chunk attention, windowed and scored decode and eviction, written from their definitions, one
row at a time; and the paged inputs of their tests.  Nothing here runs the library.

Tolerances.  With u the half step of the outputs' type (2^-8 bfloat16, 2^-11 binary16), A = sum_j p_j |v_j| of a row
and o its exact output, an output may be off by

    u |o|                the output's own rounding,
    w A                  the weights': w = u for weights rounded to the outputs' type before the product with V; over
                         per-tensor E4M3 caches tensor cores take a weight in two E4M3 parts, the second the nearest
                         code of what the first leaves: 2^-4 * 2^-4 = 2^-8 of the weight, and no less than half the
                         least code (2^-10) of a scale on which 1 is 2^8, for each of the n tokens: 2^-18 each;
                         with block scales 2^-14 of the weight and 2^-28 of the largest,
    2 d A                the logits': an error d of every logit moves each weight by at most a factor e^(2d), and
                         d = 2^-17 max(1, sum_c |q_c k_c| scale) covers D = 128 products summed in float32 (at most
                         D 2^-24 of the sum of magnitudes), the exponential (2^-22) and the scale's rounding; over
                         E4M3 caches also the queries' parts (2^-18 of the largest element each, see the kernel).

Sums of up to a few thousand float32 terms (n 2^-24 < 2^-12 A would be the worst case, sqrt(n) 2^-24 the usual one)
are covered by 2^-14 A.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
VALUES = torch.from_numpy(oracle.decode_elements(np.arange(256, dtype=np.uint8), oracle.E4M3))


class Paged:
    """Pools of random keys and values, block tables in random order, and every slot that no sequence owns NaN."""

    def __init__(self, lens, hkv, bs, dim, act, cache="act", seed=0, extra_blocks=3, width=None, scales_from=(-8, -4)):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.bs, self.dim, self.act, self.cache = list(lens), hkv, bs, dim, act, cache
        n_blk = [-(-n // bs) for n in lens]
        nb = sum(n_blk) + extra_blocks
        perm = torch.randperm(nb, generator=g)
        width = width or max(1, max(n_blk, default=1))
        self.tables = torch.full((len(lens), width), -1, dtype=torch.int32)  # nothing may go by these
        at = 0
        for b, n in enumerate(n_blk):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:]
        shape = (nb, hkv, bs, dim)
        spread = 1.0 + 2.0 * (torch.rand(1, hkv, 1, dim, generator=g) < 0.05)
        k, v = torch.randn(shape, generator=g) * spread, torch.randn(shape, generator=g)
        if cache == "act":
            self.k, self.v, nan = k.to(act), v.to(act), float("nan")
        else:
            self.k, self.v = (self._codes(x * 60) for x in (k, v))
            nan = 0x7F
        self.k_scale = self.v_scale = self.k_scales = self.v_scales = None
        if cache == "e4m3":
            self.k_scale, self.v_scale = torch.tensor([0.0171]), torch.tensor([0.0113])
        if cache == "scaled":
            self.k_scales, self.v_scales = (
                torch.exp2(torch.randint(*scales_from, (nb, hkv), generator=g).float()) * (1.0 + 0.3 * i) for i in (0, 1))
        owned = torch.zeros(nb, bs, dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(n_blk[b]):
                owned[self.tables[b, i], :min(bs, n - i * bs)] = True
        self.k.transpose(1, 2)[~owned] = nan
        self.v.transpose(1, 2)[~owned] = nan
        self.nan = nan

    @staticmethod
    def _codes(x):
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    def slot(self, b, j):
        return int(self.tables[b, j // self.bs]), j % self.bs

    def poison(self, b, tokens, k=True, v=True):
        """Make tokens of sequence b NaN."""
        for j in tokens:
            blk, off = self.slot(b, j)
            if k:
                self.k[blk, :, off] = self.nan
            if v:
                self.v[blk, :, off] = self.nan

    def cuda(self):
        """Arguments of a call: (k_cache, v_cache, tables, lens) and the scales."""
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        return ((up(self.k), up(self.v), up(self.tables), torch.tensor(self.lens, dtype=torch.int32).cuda()),
                dict(k_scale=up(self.k_scale), v_scale=up(self.v_scale), k_scales=up(self.k_scales),
                     v_scales=up(self.v_scales)))

    def tokens(self, b, js):
        """K and V of tokens js of sequence b in float64, [Hkv, n, D] each."""
        blk = torch.tensor([int(self.tables[b, j // self.bs]) for j in js], dtype=torch.long)
        off = torch.tensor([j % self.bs for j in js], dtype=torch.long)
        out = []
        for pool, one, many in ((self.k, self.k_scale, self.k_scales), (self.v, self.v_scale, self.v_scales)):
            x = pool[blk, :, off]
            x = x.double() if self.cache == "act" else VALUES[x.long()]
            if one is not None:
                x = x * one.double()
            if many is not None:
                x = x * many.double()[blk][..., None]
            out.append(x.transpose(0, 1))
        return out


def visible(pos, window=None, sinks=0):
    """The tokens that a row at pos sees."""
    lo = 0 if window is None else max(0, pos - window + 1)
    return list(range(min(sinks, lo))) + list(range(lo, pos + 1))


def attend(paged, b, q, js, scale):
    """One row q [Hq, D] of sequence b over its tokens js: (out [Hq, D], weights [Hq, n], tolerance [Hq, D])."""
    k, v = paged.tokens(b, js)
    hq, dim = q.shape
    qd = q.double().view(paged.hkv, hq // paged.hkv, dim)
    s = scale * (qd @ k.transpose(1, 2))
    p = torch.softmax(s, -1)
    a, o = p @ v.abs(), p @ v
    top = abs(scale) * (qd.abs() @ k.abs().transpose(1, 2)).amax((-1, -2))  # per kv head
    d = 2.0 ** -17 * top.clamp(min=1.0)
    extra = 0.0
    w = U[paged.act]
    if paged.cache != "act":
        ksum = k.abs().sum(-1).amax(-1)
        d = d + abs(scale) * 2.0 ** -18 * qd.abs().amax((1, 2)) * ksum
        if paged.cache == "e4m3":
            w, extra = max(w, 2.0 ** -8), 2.0 ** -18 * v.abs().sum(1)
        else:
            w, extra = max(w, 2.0 ** -14), 2.0 ** -26 * v.abs().sum(1)
        extra = extra[:, None] if torch.is_tensor(extra) else extra
    tol = U[paged.act] * o.abs() + (w + 2.0 ** -14 + 2 * d[:, None, None]) * a + extra + 1e-6
    return o.reshape(hq, dim), p.reshape(hq, -1), tol.reshape(hq, dim)


def check(got, want, tol, what=""):
    got = got.detach().double().cpu()
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), finite), f"{what}: finite where it should not be, or the other way"
    err = torch.where(finite, (got - want).abs(), 0.0)
    over = (err / tol)[finite]
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance, max error {float(err.max()):.3e}"


def evict(scores, n, budget, recent, sinks):
    """The tokens of n that stay, by scores (a 1-d array)."""
    if n <= budget:
        return list(range(n))
    others = sorted(range(sinks, n - recent), key=lambda j: (-np.inf if np.isnan(scores[j]) else scores[j], -j), reverse=True)
    # (a NaN below -inf)
    others = sorted(others, key=lambda j: bool(np.isnan(scores[j])))
    return sorted(list(range(sinks)) + list(range(n - recent, n)) + others[:budget - sinks - recent])
