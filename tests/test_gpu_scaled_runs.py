"""Block-scaled appends whose blocks' tokens are not one plain run: skipped tokens between them, slots out of order or
twice.  The runs of a block apply one after the other, in the call's order, bit for bit."""
import zlib

import numpy as np
import pytest
import torch

from tests import scaled_ref as ref
from tests import test_gpu_rope as rope

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture
def pkv(pkv_lib, cuda_device):
    pkv_lib.device_error(reset=True)
    yield pkv_lib
    assert pkv_lib.device_error(reset=True) == 0


def _slots(name, bs, n, g):
    """Slots of about n tokens in the manner `name`, every block's tokens neighbours but for skipped ones, and the
    pool's blocks."""
    ri = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    out, blk = [], 0
    while len(out) < n:
        first = ri(0, bs - 1) if blk % 3 else 0
        offs = list(range(first, ri(first, bs - 1) + 1))
        run = [blk * bs + o for o in offs]
        if name == "padding":  # skipped tokens anywhere
            run = [x for s in run for x in ([-1] * ri(0, 2) + [s])]
        elif name == "gaps":  # stored tokens left out
            run = [s for s in run if ri(0, 3)] or run[:1]
        elif name == "far":  # long stretches of skipped tokens, up to the most that may be
            run = [x for s in run for x in ([-1] * (ri(200, 255) if not ri(0, 5) else 0) + [s])]
        elif name == "order":  # any order, but for offset 0, and some twice
            rest = [s for s in run if s % bs]
            rest = [rest[i] for i in torch.randperm(len(rest), generator=g).tolist()]
            run = [s for s in run if s % bs == 0] + rest + (rest[:2] if not ri(0, 2) else [])
        out += run + [-1] * (ri(0, 40) if not ri(0, 7) else 0)
        blk += 1
    return np.asarray(out, np.int64), blk + 1


def _codes(g, *shape):
    c = torch.randint(0, 256, shape, dtype=torch.uint8, generator=g)
    c[(c & 0x7F) == 0x7F] = 0x30
    return c


CASES = [(name, n, act, hkv, D, bs) for name in ("padding", "gaps", "far", "order")
         for n, act, hkv, D, bs in ((30, "bf16", 40, 128, 16), (200, "f16", 8, 128, 16), (300, "bf16", 3, 80, 32),
                                    (700, "bf16", 2, 64, 5), (2500, "f16", 2, 64, 16), (3000, "bf16", 1, 128, 32),
                                    (1500, "f16", 5, 80, 64))]


def _pool(g, nb, hkv, bs, D):
    scales = lambda: torch.exp2(torch.randint(-12, -2, (nb, hkv), generator=g).float())  # noqa: E731
    return _codes(g, nb, hkv, bs, D), _codes(g, nb, hkv, bs, D), scales(), scales()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_append_of_split_runs(pkv, case):
    name, n, act, hkv, D, bs = case
    g = torch.Generator().manual_seed(zlib.crc32(repr(case).encode()))
    slots, nb = _slots(name, bs, n, g)
    T = len(slots)
    mag = torch.exp2(torch.randint(-12, 6, (T, hkv, 1), generator=g).float())
    k = (torch.randn(T, hkv, D, generator=g) * mag).to(DT[act])
    v = (torch.randn(T, hkv, D, generator=g) * mag.flip(0)).to(DT[act])
    pool = _pool(g, nb, hkv, bs, D)
    d = [t.cuda() for t in pool]
    pkv.paged_kv_append_scaled(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), *d)
    torch.cuda.synchronize()
    for x, codes, scales in ((k, 0, 2), (v, 1, 3)):
        wc, ws = ref.append_scaled(ref.f64(x), list(slots), pool[codes].numpy(), pool[scales].numpy(), bs)
        assert np.array_equal(d[scales].cpu().numpy(), ws), "scales"
        assert ref.same_codes(d[codes].cpu().numpy(), wc), "codes"


# (a call for each run: of the long ones, those whose runs are many are left out)
ROTATED = [c for c in CASES if c[1] <= 1000 or c[0] not in ("far", "order")]


@pytest.mark.parametrize("case", ROTATED, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("rot,interleaved", [(0, False), (24, False), (16, True)], ids=["whole", "apart", "next"])
def test_rotated_append_of_split_runs(pkv, case, rot, interleaved):
    """Rotated keys: the same bits as those of a rotation into a 16-bit row and one call for each run, where the runs
    are applied by calls of their own; padding by positions as well as by slots."""
    name, n, act, hkv, D, bs = case
    rot = rot or D
    g = torch.Generator().manual_seed(zlib.crc32(repr((case, rot)).encode()))
    slots, nb = _slots(name, bs, n, g)
    T = len(slots)
    k, v = (torch.randn(T, hkv, D, generator=g).to(DT[act]).cuda() for _ in range(2))
    positions = torch.randint(0, 5000, (T,), dtype=torch.int32, generator=g)
    hidden = torch.from_numpy(slots < 0) & (torch.rand(T, generator=g) < 0.5)  # padding by position, slots of others
    positions[hidden] = -1
    all_slots = torch.from_numpy(np.where(hidden.numpy(), 3, slots))
    freq, _ = pkv.rope_inv_freq(rot)
    pool = [t.cuda() for t in _pool(g, nb, hkv, bs, D)]
    one, many = [t.clone() for t in pool], [t.clone() for t in pool]
    pkv.paged_rope_append(None, k, v, positions.cuda(), all_slots.cuda(), freq, one[0], one[1], interleaved=interleaved,
                          k_scales=one[2], v_scales=one[3])
    d_slots, d_pos = torch.from_numpy(slots).cuda(), positions.cuda()
    for t, m in ref.runs(list(slots), bs):
        pkv.paged_rope_append(None, k[t:t + m], v[t:t + m], d_pos[t:t + m].clone(), d_slots[t:t + m].clone(), freq,
                              many[0], many[1], interleaved=interleaved, k_scales=many[2], v_scales=many[3])
    torch.cuda.synchronize()
    for a, b in zip(one, many):
        assert torch.equal(a, b)


LONG = [
    # act, tokens, Hq, Hkv, D, rotary_dim, interleaved, bs, positions below, packed
    ("bf16", 1400, 4, 2, 128, 128, False, 32, 9000, True),
    ("f16", 1400, 2, 2, 128, 128, True, 32, 9000, True),
    ("bf16", 1400, 2, 2, 128, 24, False, 32, 9000, True),
    ("f16", 1700, 2, 1, 128, 128, False, 64, 70000, True),
    ("bf16", 1700, 1, 1, 128, 64, True, 64, 70000, False),
    ("f16", 1700, 1, 1, 128, 40, False, 64, 70000, False),
    ("bf16", 1300, 2, 2, 128, 128, True, 16, 9000, True),
    ("f16", 1300, 2, 2, 128, 72, False, 16, 9000, True),
    ("bf16", 1300, 1, 1, 256, 256, False, 16, 9000, True),
    ("f16", 1300, 2, 2, 80, 20, True, 32, 9000, True),
    ("f16", 500, 4, 2, 128, 128, True, 16, 9000, True),
    ("bf16", 800, 2, 5, 128, 56, False, 32, 9000, True),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c)))
def test_rotated_prompts_in_every_layout(pkv, case):
    """Prompts whose runs stay in registers and those whose rows are read twice, with two warps a run (more than about
    1,200 tokens) and with one, for channels paired as neighbours, in whole chunks and apart."""
    rope.test_rope_append_e4m3(pkv, case, True)
