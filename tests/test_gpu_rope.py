"""Rotary positions with the append (paged_rope_append) on the GPU, against a float64 statement."""
import zlib

import numpy as np
import pytest
import torch

from tests import scaled_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# float32 error of a rotated channel, relative to (|a| + |b|) * factor: cos and sin to 2 steps of sincospi plus the
# rounding of its argument (pi/4 * 2^-24) and of the factor's product, two products and a sum: under 8 * 2^-24
F32 = 8 * 2.0 ** -24


@pytest.fixture
def pkv(pkv_lib, cuda_device):
    pkv_lib.device_error(reset=True)
    yield pkv_lib
    assert pkv_lib.device_error(reset=True) == 0


def _gen(case):
    return torch.Generator().manual_seed(zlib.crc32(repr(case).encode()))


def _inputs(case):
    act, T, Hq, Hkv, D, rot, inter, bs, top, packed = case
    g = _gen(case)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(DT[act])
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, top, (T,), generator=g).to(torch.int32)
    pos[0] = 0
    pos[-1] = top - 1
    nb = -(-T // bs) * 2 + 2
    perm = torch.randperm(nb, generator=g)
    # stretches of neighbours over shuffled blocks, the first one in the middle of its block
    at = torch.arange(T) + bs // 2
    slots = perm[at // bs] * bs + at % bs
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    return g, q, k, v, pos, slots, nb, f.float()


CASES = [
    # act, tokens, Hq, Hkv, D, rotary_dim, interleaved, bs, positions below, packed
    ("bf16", 1, 8, 1, 128, 128, False, 16, 10, True),
    ("bf16", 70, 64, 8, 128, 128, False, 16, 131072, True),
    ("f16", 37, 8, 8, 64, 64, True, 32, 2 ** 31 - 1, True),
    ("bf16", 50, 5, 5, 64, 24, False, 16, 1000003, True),   # half of the pairs off the 8-channel grid
    ("f16", 33, 6, 2, 80, 20, True, 16, 5000, False),
    ("bf16", 19, 4, 2, 128, 32, False, 16, 5000, True),
    ("f16", 300, 32, 8, 128, 64, True, 16, 40000, True),
    ("bf16", 40, 2, 1, 256, 256, False, 16, 5000, True),
    ("f16", 9, 3, 1, 8, 2, False, 4, 5000, False),
    ("bf16", 2600, 8, 2, 64, 64, False, 16, 70000, True),
]


def _check_q(out, q, pos, f, inter, factor):
    want, mag = ref.rotate(ref.f64(q), pos.numpy(), f.numpy(), inter, factor)
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(want) + F32 * mag + 2.0 ** -25 * (mag > 0)
    err = np.abs(ref.f64(out) - want)
    assert np.all(err <= tol), f"{(err > tol).sum()} elements, worst {np.max(err / np.maximum(tol, 1e-30)):.2f}"
    rot = 2 * len(f)
    assert torch.equal(out[..., rot:].cpu(), q[..., rot:])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_append_16bit(pkv, case):
    act, T, Hq, Hkv, D, rot, inter, bs, top, packed = case
    g, q, k, v, pos, slots, nb, f = _inputs(case)
    factor = 1.25
    dq = torch.cat([q, k, v], 1).cuda()
    kc = torch.randn(nb, Hkv, bs, D, generator=g).to(DT[act]).cuda()
    vc = kc.clone()
    before = kc.clone()
    out = pkv.paged_rope_append(dq[:, :Hq], dq[:, Hq:Hq + Hkv], dq[:, Hq + Hkv:], pos.cuda(), slots.cuda(), f.cuda(),
                                kc, vc, interleaved=inter, attention_factor=factor)
    torch.cuda.synchronize()
    _check_q(out, q, pos, f, inter, factor)
    b, o = slots // bs, slots % bs
    _check_q(kc[b.cuda(), :, o.cuda()].cpu(), k, pos, f, inter, factor)
    assert torch.equal(vc[b.cuda(), :, o.cuda()].cpu(), v)
    used = torch.zeros(nb, bs, dtype=torch.bool)
    used[b, o] = True
    keep = ~used[:, None, :, None].expand(kc.shape)
    assert torch.equal(kc.cpu()[keep], before.cpu()[keep]) and torch.equal(vc.cpu()[keep], before.cpu()[keep])


def _near(codes, scale, want, slack):
    """Codes that are a nearest one to `want`, or nearest to something within slack of it."""
    got = ref.VALUES[codes] * scale
    best = ref.VALUES[ref.encode(want / scale)] * scale
    return np.abs(got - want) <= np.abs(best - want) + 2 * slack


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_append_e4m3(pkv, case, blocks):
    act, T, Hq, Hkv, D, rot, inter, bs, top, packed = case
    g, q, k, v, pos, slots, nb, f = _inputs(case)
    factor = 0.75
    d = torch.cat([q, k, v], 1).cuda()
    kc = torch.randint(0, 0x70, (nb, Hkv, bs, D), dtype=torch.uint8, generator=g).cuda()
    vc = kc.clone()
    kc0 = kc.cpu().numpy()
    if blocks:
        s0 = torch.exp2(torch.randint(-12, -6, (nb, Hkv), generator=g).float())
        kw = dict(k_scales=s0.cuda(), v_scales=s0.cuda())
    else:
        kw = dict(k_scale=torch.tensor([0.02], device="cuda"), v_scale=torch.tensor([0.003], device="cuda"))
    out = pkv.paged_rope_append(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], pos.cuda(), slots.cuda(), f.cuda(), kc,
                                vc, interleaved=inter, attention_factor=factor, **kw)
    torch.cuda.synchronize()
    _check_q(out, q, pos, f, inter, factor)
    want, mag = ref.rotate(ref.f64(k), pos.numpy(), f.numpy(), inter, factor)
    b, o = (slots // bs).numpy(), (slots % bs).numpy()
    if blocks:
        # the keys' scales: the definition's, as long as no rotated maximum is so near a border that float32 may
        # pass it (channels that do not turn are exact)
        wk, ws = ref.append_scaled(want, list(slots.numpy()), kc0, s0.numpy(), bs)
        lo, hi = (ref.append_scaled(want * (1 + e * (mag > 0)), list(slots.numpy()), kc0, s0.numpy(), bs)[1]
                  for e in (-1e-6, 1e-6))
        assert np.array_equal(lo, hi), "a maximum on a border: draw other inputs"
        assert np.array_equal(kw["k_scales"].cpu().numpy(), ws)
        wv, wvs = ref.append_scaled(ref.f64(v), list(slots.numpy()), kc0, s0.numpy(), bs)
        assert np.array_equal(kw["v_scales"].cpu().numpy(), wvs) and ref.same_codes(vc.cpu().numpy(), wv)
        sc = ws[b][:, :, None]
        stored = np.zeros((nb, bs), bool)
        stored[b, o] = True
        other = ~stored[:, None, :, None] & np.ones(kc0.shape, bool)
        assert np.array_equal(kc.cpu().numpy()[other], wk[other])  # requantised, not rotated: bit for bit
    else:
        sc = np.float64(np.float32(0.02))
        x = (ref.f64(v).astype(np.float32) / np.float32(0.003)).astype(np.float64)
        assert ref.same_codes(vc.cpu().numpy()[b, :, o], ref.encode(x))
    slack = F32 * mag + 2.0 ** -23 * np.abs(want)  # and the division by a scale that is no power of two
    top_of = 448.0 * sc
    assert np.all(_near(kc.cpu().numpy()[b, :, o], sc, np.clip(want, -top_of, top_of), slack))


def test_rope_append_in_place_padding_and_keys_alone(pkv):
    case = ("bf16", 24, 8, 2, 128, 128, False, 16, 9000, True)
    g, q, k, v, pos, slots, nb, f = _inputs(case)
    pos[[3, 23]] = -1          # padding rows
    slots[[5, 6]] = -1         # rotated, not stored
    slots[9] = nb * 16 + 1     # outside the pool
    d = torch.cat([q, k, v], 1).cuda()
    caches = [torch.zeros(nb, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    args = (pos.cuda(), slots.cuda(), f.cuda())
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    pkv.paged_rope_append(d[:, :8], d[:, 8:10], d[:, 10:], *args, *caches[:2], q_out=out)
    assert pkv.device_error(reset=True) == pkv.DEV_BAD_SLOT
    assert bool((out[[3, 23]] == 7.0).all())
    live = [t for t in range(24) if t not in (3, 23)]
    _check_q(out[live], q[live], pos[live], f, False, 1.0)
    stored = [t for t in live if t not in (5, 6, 9)]
    assert int((caches[1] != 0).any(-1).any(1).sum()) == len(stored)
    keys = pkv.paged_rope_append(None, d[:, 8:10], d[:, 10:], *args, *caches[2:])
    assert keys is None and pkv.device_error(reset=True) == pkv.DEV_BAD_SLOT
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    # in place, in the packed buffer itself
    want = out.clone()
    want[[3, 23]] = d[[3, 23], :8]
    pkv.paged_rope_append(d[:, :8], d[:, 8:10], d[:, 10:], *args, *caches[:2], q_out=d[:, :8])
    assert torch.equal(d[:, :8], want) and pkv.device_error(reset=True) == pkv.DEV_BAD_SLOT


def test_rope_in_place_off_the_grid(pkv):
    """rotary_dim / 2 off the 8-channel grid, in place: partners are read before anything is written."""
    case = ("f16", 40, 7, 1, 64, 24, False, 16, 9000, True)
    g, q, k, v, pos, slots, nb, f = _inputs(case)
    d = torch.cat([q, k, v], 1).cuda()
    kc = torch.zeros(nb, 1, 16, 64, dtype=torch.float16, device="cuda")
    pkv.paged_rope_append(d[:, :7], d[:, 7:8], d[:, 8:], pos.cuda(), slots.cuda(), f.cuda(), kc, kc.clone(),
                          q_out=d[:, :7])
    _check_q(d[:, :7], q, pos, f, False, 1.0)


def test_rope_scalings(pkv_lib):
    """The frequency tables: fastest pairs kept, slowest divided, linear divides all, everything monotonic."""
    base, _ = pkv_lib.rope_inv_freq(128, device="cpu")
    i = torch.arange(64, dtype=torch.float64)
    assert torch.allclose(base.double(), 10000.0 ** (-i / 64), rtol=2.0 ** -24)
    lin, a = pkv_lib.rope_inv_freq(128, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(lin, (10000.0 ** (-i / 64) / 4).float()) and a == 1.0
    ntk, _ = pkv_lib.rope_inv_freq(128, scaling="ntk", factor=4.0, device="cpu")
    assert abs(float(ntk[-1] / base[-1]) - 0.25) < 1e-6 and ntk[0] == 1.0
    for kind in ("yarn", "smooth"):
        f, a = pkv_lib.rope_inv_freq(128, scaling=kind, factor=8.0, original_context=4096, device="cpu")
        turns = 4096 * base.double() / (2 * np.pi)
        fast, slow = turns >= 32, turns <= 1
        assert torch.equal(f[fast], base[fast])
        assert torch.allclose(f[slow], base[slow] / 8, rtol=2.0 ** -22) and bool((f.diff() < 0).all())
        assert a == (pytest.approx(0.1 * np.log(8.0) + 1) if kind == "yarn" else 1.0)
    for bad in (dict(rotary_dim=7), dict(rotary_dim=8, scaling="what"), dict(rotary_dim=8, scaling="yarn", factor=2.0),
                dict(rotary_dim=8, scaling="linear", factor=0.5), dict(rotary_dim=8, base=0.5)):
        with pytest.raises(ValueError):
            pkv_lib.rope_inv_freq(**bad, device="cpu")
