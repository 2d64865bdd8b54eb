"""The block-scaled E4M3 cache on the GPU: appends bit for bit, decode within a bound derived in
tests/scaled_ref.py, block copy and swap with their scales."""
import zlib

import numpy as np
import pytest
import torch

from tests import scaled_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture
def pkv(pkv_lib, cuda_device):
    pkv_lib.device_error(reset=True)
    prev = pkv_lib.set_kernel_path(pkv_lib.PATH_AUTO)
    yield pkv_lib
    pkv_lib.set_kernel_path(prev)
    assert pkv_lib.device_error(reset=True) == 0


def _gen(case):
    return torch.Generator().manual_seed(zlib.crc32(repr(case).encode()))


def _codes(g, *shape):
    c = torch.randint(0, 256, shape, dtype=torch.uint8, generator=g)
    c[(c & 0x7F) == 0x7F] = 0x30
    return c


def _append(pkv, k, v, slots, kc, vc, ks, vs):
    """Run on the GPU and check against the definition; returns the new (kc, vc, ks, vs) on the host."""
    d = [t.cuda() for t in (kc, vc, ks, vs)]
    pkv.paged_kv_append_scaled(k.cuda(), v.cuda(), torch.as_tensor(slots, dtype=torch.int64).cuda(), *d)
    torch.cuda.synchronize()
    got = [t.cpu() for t in d]
    bs = kc.shape[2]
    for x, codes, scales, gc, gs in ((k, kc, ks, got[0], got[2]), (v, vc, vs, got[1], got[3])):
        wc, ws = ref.append_scaled(ref.f64(x), list(np.asarray(slots)), codes.numpy(), scales.numpy(), bs)
        assert np.array_equal(gs.numpy(), ws), "scales"
        assert ref.same_codes(gc.numpy(), wc), "codes"
    return got


# ------------------------------------------------------------------ append ---
APPENDS = [
    # act, Hkv, D, bs, (tokens there, new tokens) of each request
    ("bf16", 8, 128, 16, [(0, 1), (3, 1), (15, 1), (16, 1), (31, 1), (100, 1)]),
    ("f16", 8, 64, 32, [(0, 1), (5, 1), (31, 1), (32, 1)]),
    ("bf16", 1, 128, 16, [(0, 1)]),
    ("bf16", 5, 80, 16, [(0, 37), (7, 2), (15, 18), (16, 16), (30, 4)]),
    ("f16", 2, 128, 32, [(0, 129), (1, 63), (31, 1), (33, 95)]),
    ("bf16", 3, 8, 5, [(0, 13), (4, 1), (2, 9)]),
    ("f16", 1, 256, 64, [(0, 200), (63, 2), (10, 100)]),
    ("bf16", 40, 128, 16, [(i, 1) for i in range(70)]),
    ("f16", 1, 40, 1, [(0, 40), (3, 5)]),
    # prompts: the kernel for runs of many tokens, whole blocks in registers or (64-token blocks) read twice
    ("bf16", 2, 64, 16, [(i % 19, 37 + i) for i in range(40)]),
    ("f16", 3, 128, 32, [(0, 1500), (7, 700), (31, 2), (33, 800)]),
    ("f16", 1, 128, 64, [(0, 900), (70, 650)]),
    ("bf16", 1, 80, 16, [(5, 1000), (0, 333)]),
]


def _requests(lens, bs, g):
    """Slots of the requests' new tokens over a shuffled pool, and the pool's size."""
    n_blk = [-(-(c + n) // bs) for c, n in lens]
    nb = sum(n_blk) + 3
    perm = torch.randperm(nb, generator=g).tolist()
    slots, at = [], 0
    for (c, n), k in zip(lens, n_blk):
        slots += [perm[at + p // bs] * bs + p % bs for p in range(c, c + n)]
        at += k
    return np.asarray(slots, np.int64), nb


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(map(str, c[:4])))
def test_append_scaled_bit_exact(pkv, case):
    act, Hkv, D, bs, lens = case
    g = _gen(case)
    slots, nb = _requests(lens, bs, g)
    T = len(slots)
    mag = torch.exp2(torch.randint(-12, 6, (T, Hkv, 1), generator=g).float())  # scales grow in some blocks
    k = (torch.randn(T, Hkv, D, generator=g) * mag).to(DT[act])
    v = (torch.randn(T, Hkv, D, generator=g) * mag.flip(0)).to(DT[act])
    kc, vc = _codes(g, nb, Hkv, bs, D), _codes(g, nb, Hkv, bs, D)
    ks = torch.exp2(torch.randint(-12, -2, (nb, Hkv), generator=g).float())
    vs = torch.exp2(torch.randint(-12, -2, (nb, Hkv), generator=g).float())
    _append(pkv, k, v, slots, kc, vc, ks, vs)


def test_append_scaled_borders_and_odd_values(pkv):
    """Largest elements at, just above and just below 448 * 2^e; zeros, infinities, NaN, the type's extremes."""
    g = _gen("odd")
    bs, D = 16, 64
    rows = []
    for top in (448.0, 450.0, 446.0, 3.5, 3.515625, 3.484375, 0.0, 2.0 ** -133, 2.0 ** -70, 3.3895e38):
        r = torch.randn(1, D, generator=g) * 0.01 * min(top, 1e30)
        r[0, 7] = -top
        rows.append(r)
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = torch.randn(1, D, generator=g)
        r[0, 3] = bad
        rows.append(r)
    rows.append(torch.full((1, D), float("nan")))
    k = torch.stack(rows).to(torch.bfloat16)
    T = len(rows)
    nb = T + 2
    slots = np.arange(T) * bs + np.where(np.arange(T) % 2, 4, 0)  # every second one into a block that has tokens
    kc = _codes(g, nb, 1, bs, D)
    s = torch.exp2(torch.randint(-9, 3, (nb, 1), generator=g).float())
    _append(pkv, k, k.flip(0).contiguous(), slots, kc, kc.flip(0).contiguous(), s, s.clone())


@pytest.mark.parametrize("act,bs", [("bf16", 16), ("f16", 32), ("bf16", 64)])
def test_append_scaled_odd_values_in_prompts(pkv, act, bs):
    """Infinities, NaN, zeros and tiny elements among the tokens of long runs."""
    g = _gen((act, bs))
    T, H, D = 1300, 2, 64
    k = (torch.randn(T, H, D, generator=g) * torch.exp2(torch.randint(-20, 8, (T, 1, 1), generator=g).float())).to(DT[act])
    at = torch.randint(0, T, (60,), generator=g)
    k[at[:20], :, 5] = float("inf")
    k[at[20:40], 0, 9] = float("nan")
    k[at[40:50]] = 0.0
    k[at[50:], 1] = -float("inf")
    k[200:200 + 2 * bs] = 0.0
    slots, nb = _requests([(3, T)], bs, g)
    kc, s = _codes(g, nb, H, bs, D), torch.exp2(torch.randint(-8, -4, (nb, H), generator=g).float())
    _append(pkv, k, k.flip(0).contiguous(), slots, kc, kc.clone(), s, s.clone())


def test_append_scaled_token_by_token_equals_the_values(pkv):
    """A block filled one token at a time while its scale grows: every element stays within what its own rounding
    and the later requantisations (exact, but for subnormal codes) allow."""
    g = _gen("grow")
    bs, D, H = 16, 128, 2
    x = torch.randn(bs, H, D, generator=g) * torch.exp2(torch.arange(bs).float() / 2)[:, None, None]
    x = x.to(torch.bfloat16)
    kc, vc = torch.zeros(2, H, bs, D, dtype=torch.uint8), torch.zeros(2, H, bs, D, dtype=torch.uint8)
    ks, vs = torch.zeros(2, H), torch.zeros(2, H)
    for t in range(bs):
        kc, vc, ks, vs = _append(pkv, x[t:t + 1], -x[t:t + 1], [bs + t], kc, vc, ks, vs)
    got = ref.VALUES[kc[1].numpy()] * ks[1].numpy()[:, None, None]
    want = ref.f64(x).transpose(1, 0, 2)
    # half a step of a normal code, 2^-4; of a subnormal one, 2^-10 of the scale, each time the scale grew (at most
    # doubling each token): the sum of 2^-10 s (1 + 1/2 + 1/4 ..) < 2^-9 s
    tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * ks[1].numpy()[:, None, None]
    assert np.all(np.abs(got - want) <= tol)


def test_append_scaled_keeps_other_slots(pkv):
    """Tokens behind a run keep their values too, and padding and bad slots write nothing."""
    g = _gen("behind")
    bs, D, H, nb = 16, 128, 2, 6
    k = torch.randn(5, H, D, generator=g).to(torch.float16) * 100
    slots = np.asarray([2 * bs + 5, 2 * bs + 6, -1, nb * bs + 3, 4 * bs + 15], np.int64)
    kc, s = _codes(g, nb, H, bs, D), torch.exp2(torch.randint(-8, -4, (nb, H), generator=g).float())
    got = _append(pkv, k, k.flip(0).contiguous(), slots, kc, kc.clone(), s, s.clone())
    assert pkv.device_error(reset=True) == pkv.DEV_BAD_SLOT
    for b in (0, 1, 3, 5):
        assert torch.equal(got[0][b], kc[b]) and torch.equal(got[2][b], s[b])


def test_append_scaled_other_scales(pkv):
    """Scales that are no powers of two, not positive or NaN in the cache before the call."""
    g = _gen("others")
    bs, D, H, nb = 16, 64, 1, 6
    k = torch.randn(nb, H, D, generator=g).to(torch.bfloat16)
    slots = np.arange(nb) * bs + 3
    kc = _codes(g, nb, H, bs, D)
    s = torch.tensor([[0.3], [0.001], [0.0], [-1.0], [float("nan")], [1e20]])
    with np.errstate(invalid="ignore"):
        _append(pkv, k, k, slots, kc, kc.clone(), s, s.clone())


def test_append_scaled_strided_rows(pkv):
    g = _gen("strided")
    bs, D, H, T, nb = 16, 128, 4, 50, 8
    qkv = torch.randn(T, 3, H, D, generator=g).to(torch.bfloat16).cuda()
    slots = torch.arange(T, dtype=torch.int64).cuda() + 16
    outs = []
    for k, v in ((qkv[:, 1], qkv[:, 2]), (qkv[:, 1].contiguous(), qkv[:, 2].contiguous())):
        d = [torch.zeros(nb, H, bs, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
        d += [torch.zeros(nb, H, device="cuda") for _ in range(2)]
        pkv.paged_kv_append_scaled(k, v, slots, *d)
        outs.append(d)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    # one row for every token (stride 0)
    one = qkv[:1, 1].expand(T, H, D)
    d = [torch.zeros(nb, H, bs, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    d += [torch.zeros(nb, H, device="cuda") for _ in range(2)]
    pkv.paged_kv_append_scaled(one, one, slots, *d)
    assert torch.equal(d[0][1, :, 0], d[0][2, :, 5])


# ------------------------------------------------------------------ decode ---
LENS = [1, 15, 16, 17, 33, 127, 128, 129, 0, 255, 511, 512, 513, 700, 1025]
DECODES = [
    # act, Hq, Hkv, D, bs, partition, scales
    ("bf16", 64, 8, 128, 16, -1, "narrow"),
    ("f16", 32, 8, 128, 32, -1, "wide"),
    ("bf16", 16, 2, 128, 16, 128, "wide"),
    ("bf16", 8, 1, 128, 16, 64, "odd"),
    ("bf16", 4, 2, 128, 16, -1, "wide"),
    ("f16", 4, 2, 128, 32, 64, "odd"),
    ("bf16", 8, 8, 128, 16, -1, "narrow"),
    ("f16", 3, 3, 128, 16, 96, "wide"),
    ("f16", 8, 8, 64, 16, -1, "wide"),
    ("bf16", 6, 3, 64, 32, 64, "odd"),
    ("bf16", 16, 4, 64, 16, -1, "wide"),
    ("f16", 64, 8, 64, 32, -1, "narrow"),
    ("bf16", 16, 2, 64, 16, 128, "odd"),
    ("f16", 24, 3, 64, 16, -1, "wide"),
    # partitions of several 512-token segments
    ("bf16", 16, 2, 128, 16, 1024, "wide"),
    ("f16", 16, 2, 64, 32, 608, "narrow"),
    ("bf16", 3, 3, 128, 16, 0, "odd"),
    ("f16", 8, 1, 128, 32, 0, "narrow"),
    ("bf16", 32, 4, 64, 16, 0, "wide"),
    ("f16", 4, 1, 128, 16, 1024, "odd"),
]


def _scales(g, kind, nb, hkv, values):
    if kind == "narrow":
        s = torch.exp2(torch.randint(-9, -4, (nb, hkv), generator=g).float())
    elif values:  # V scales over a wide range, whole blocks far below and above the others
        s = torch.exp2(torch.randint(-30, 20, (nb, hkv), generator=g).float())
    else:
        s = torch.exp2(torch.randint(-14, -5, (nb, hkv), generator=g).float())
    if kind == "odd":
        s = s * (0.5 + torch.rand(nb, hkv, generator=g))
        s[torch.rand(nb, hkv, generator=g) < 0.1] = 0.0
        s[torch.rand(nb, hkv, generator=g) < 0.1] *= -1.0
    return s


def _decode_case(case, lens, qmul=1.0):
    act, Hq, Hkv, D, bs, part, kind = case
    g = _gen(case)
    n_blk = [-(-n // bs) for n in lens]
    nb = sum(n_blk) + 5
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((len(lens), max(n_blk) + 1), 2 ** 31 - 1, dtype=torch.int32)  # never read past a length
    at = 0
    for i, n in enumerate(n_blk):
        tables[i, :n] = perm[at:at + n]
        at += n
    q = (torch.randn(len(lens), Hq, D, generator=g) * qmul).to(DT[act])
    kc, vc = _codes(g, nb, Hkv, bs, D), _codes(g, nb, Hkv, bs, D)
    ks, vs = _scales(g, kind, nb, Hkv, False), _scales(g, kind, nb, Hkv, True)
    for i, n in enumerate(lens):  # NaN codes behind the context, NaN scales in blocks nobody has
        if n % bs:
            kc[tables[i, n_blk[i] - 1].long(), :, n % bs:] = 0x7F
            vc[tables[i, n_blk[i] - 1].long(), :, n % bs:] = 0xFF
    for b in perm[at:].tolist():
        kc[b] = vc[b] = 0x7F
        ks[b] = vs[b] = float("nan")
    return q, kc, vc, ks, vs, tables, torch.tensor(lens, dtype=torch.int32)


def _check_decode(pkv, case, lens, qmul=1.0, **kw):
    bs, part = case[4], case[5]
    host = _decode_case(case, lens, qmul)
    q, kc, vc, ks, vs, tables, L = (t.cuda() for t in host)
    scale = case[3] ** -0.5
    out = pkv.paged_attention_decode_scaled(q, kc, vc, ks, vs, tables, L, scale, partition_size=part, **kw)
    torch.cuda.synchronize()
    want, bound = ref.decode_scaled(ref.f64(host[0]), host[1].numpy(), host[2].numpy(), host[3].numpy(),
                                    host[4].numpy(), host[5].numpy(), lens, scale, bs, host[0].dtype)
    got = ref.f64(out)
    top = torch.finfo(host[0].dtype).max  # values past the output type's range round to infinity
    ok = np.abs(got - want) <= bound
    ok |= (np.abs(want) >= top * 0.999) & (np.abs(got) >= top)
    worst = np.nanmax(np.where(ok, 0, np.abs(got - want) / bound)) if not ok.all() else 0
    assert ok.all(), f"{(~ok).sum()} elements off, worst {worst:.2f} of the bound, NaN {np.isnan(got).sum()}"
    return out


@pytest.mark.parametrize("case", DECODES, ids=lambda c: "-".join(map(str, c)))
def test_decode_scaled_matches_the_definition(pkv, case):
    if case[0] == "f16" and case[6] == "wide":
        case = case[:6] + ("narrow",)  # 2^20 * 448 passes binary16's range
    _check_decode(pkv, case, LENS)


@pytest.mark.parametrize("qmul", [2.0 ** -20, 30.0, 1e20])
def test_decode_scaled_query_magnitudes(pkv, qmul):
    """Tiny and huge bf16 queries (the CUDA-core kernel's float path), one-hot softmaxes."""
    for case in (("bf16", 16, 2, 128, 16, -1, "narrow"), ("bf16", 4, 4, 64, 16, -1, "narrow")):
        _check_decode(pkv, case, [1, 40, 513], qmul)


def test_decode_scaled_every_path(pkv):
    case = ("bf16", 32, 4, 128, 16, 256, "wide")
    for path in (pkv.PATH_CUDA_CORE, pkv.PATH_TENSOR, pkv.PATH_TENSOR_2CTA):
        pkv.set_kernel_path(path)
        _check_decode(pkv, case, LENS)


def test_decode_scaled_more_rows_than_one_launch(pkv):
    case = ("bf16", 8, 1, 128, 16, -1, "narrow")
    _check_decode(pkv, case, [(i * 7) % 41 for i in range(2100)])


def test_decode_scaled_long_context(pkv):
    _check_decode(pkv, ("bf16", 4, 1, 128, 16, -1, "wide"), [20011, 1])
    _check_decode(pkv, ("bf16", 2, 2, 128, 32, -1, "narrow"), [9001])
    _check_decode(pkv, ("bf16", 8, 1, 128, 16, 2048, "odd"), [20011, 2049, 7])
    _check_decode(pkv, ("f16", 8, 1, 64, 16, 0, "narrow"), [9001, 1])


@pytest.mark.parametrize("case", [("bf16", 16, 8, 128, 16, -1, "odd"), ("f16", 8, 8, 64, 32, -1, "narrow")],
                         ids=lambda c: "-".join(map(str, c)))
def test_decode_scaled_many_sequences(pkv, case):
    """Enough items for partitions of four segments; lengths at the segments' and the partitions' borders."""
    lens = [2049, 0, 512, 513, 1024, 1025, 1536, 1537, 2047, 2048, 1, 2100] + [(i * 37) % 200 for i in range(52)]
    _check_decode(pkv, case, lens)


def test_decode_scaled_all_rows_empty(pkv):
    for hq in (16, 2):
        out = _check_decode(pkv, ("bf16", hq, 2, 128, 16, -1, "narrow"), [0, 0, 0], out=None)
        assert out.count_nonzero() == 0


def test_decode_scaled_equals_one_scale(pkv):
    """With one scale everywhere the result is the per-tensor call's, within both kernels' bounds."""
    case = ("bf16", 32, 4, 128, 16, -1, "narrow")
    lens = [n for n in LENS if n]
    q, kc, vc, ks, vs, tables, L = (t.cuda() for t in _decode_case(case, lens))
    one = torch.tensor([0.01], device="cuda")
    a = pkv.paged_attention_decode(q, kc, vc, tables, L, 0.1, k_scale=one, v_scale=one)
    b = pkv.paged_attention_decode_scaled(q, kc, vc, one.expand(ks.shape).contiguous(),
                                          one.expand(vs.shape).contiguous(), tables, L, 0.1)
    assert torch.allclose(a.float(), b.float(), atol=2.0 ** -7 * 448 * 0.01, rtol=2.0 ** -7)


def test_decode_scaled_flags_and_skips(pkv):
    case = ("bf16", 16, 2, 128, 16, -1, "narrow")
    q, kc, vc, ks, vs, tables, L = (t.cuda() for t in _decode_case(case, [5, 40, 40]))
    L[0] = -3
    out = torch.full_like(q, 7.0)
    pkv.paged_attention_decode_scaled(q, kc, vc, ks, vs, tables, L, 0.1, out=out)
    assert pkv.device_error(reset=True) == pkv.DEV_BAD_CONTEXT_LEN
    assert bool((out[0] == 7.0).all()) and bool((out[1:] != 7.0).any())
    L[0] = 5
    tables[1, 1] = -1
    pkv.paged_attention_decode_scaled(q, kc, vc, ks, vs, tables, L, 0.1, out=out)
    assert pkv.device_error(reset=True) == pkv.DEV_BAD_BLOCK


def test_decode_scaled_plan_stream_and_graph(pkv):
    """A plan on a stream of its own, then captured and replayed with new lengths."""
    for case in (("bf16", 32, 4, 128, 16, -1, "wide"), ("bf16", 4, 4, 128, 16, 64, "wide")):
        q, kc, vc, ks, vs, tables, L = (t.cuda() for t in _decode_case(case, [200, 513, 77]))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ws = torch.empty(pkv.workspace_size(3, case[1], case[2], case[3], tables.shape[1], case[4], case[5],
                                            block_scales=True),
                         dtype=torch.uint8, device="cuda")
        plan = pkv.DecodePlan(q, kc, vc, tables, L, 0.1, k_scales=ks, v_scales=vs, partition_size=case[5],
                              workspace=ws, stream=s)
        plan.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan.run()
        for lens in ([200, 513, 77], [1, 64, 0], [199, 16, 76]):
            L.copy_(torch.tensor(lens, dtype=torch.int32))
            plan.out.fill_(9.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            want = pkv.paged_attention_decode_scaled(q, kc, vc, ks, vs, tables, L, 0.1, partition_size=case[5])
            assert torch.equal(plan.out, want)


# ----------------------------------------------------------- copy and swap ---
@pytest.mark.parametrize("hkv,bs,D", [(8, 16, 128), (3, 32, 64), (1, 16, 8)])
def test_block_copy_and_swap_take_scales_along(pkv, hkv, bs, D):
    g = _gen((hkv, bs, D))
    nb = 12
    kc, vc = _codes(g, nb, hkv, bs, D), _codes(g, nb, hkv, bs, D)
    ks, vs = torch.randn(nb, hkv, generator=g), torch.randn(nb, hkv, generator=g)
    d = [t.cuda() for t in (kc, vc, ks, vs)]
    pairs = torch.tensor([[3, 7], [0, 11], [5, 2]], dtype=torch.int32)
    pkv.paged_block_copy(d[0], d[1], pairs.cuda(), k_scales=d[2], v_scales=d[3])
    for host, dev in zip((kc, vc, ks, vs), d):
        want = host.clone()
        want[pairs[:, 1].long()] = host[pairs[:, 0].long()]
        assert torch.equal(dev.cpu(), want)
    ids = torch.tensor([7, 1, 9, 4], dtype=torch.int32).cuda()
    back = torch.tensor([0, 10, 6, 8], dtype=torch.int32).cuda()
    before = [t.clone() for t in d]
    block = hkv * bs * D
    for dev in ("cuda", "cpu"):
        st = torch.zeros(4, 2, block, dtype=torch.uint8, device=dev)
        sc = torch.zeros(4, 2, hkv, device=dev)
        if dev == "cpu":
            st, sc = st.pin_memory(), sc.pin_memory()
        pkv.paged_block_swap(d[0], d[1], ids, st, pkv.SWAP_OUT, k_scales=d[2], v_scales=d[3], scale_staging=sc)
        pkv.paged_block_swap(d[0], d[1], back, st, pkv.SWAP_IN, k_scales=d[2], v_scales=d[3], scale_staging=sc)
        torch.cuda.synchronize()
        for a, b in zip(before, d):
            want = a.clone()
            want[back.long()] = a[ids.long()]
            assert torch.equal(b, want)
    bad = torch.tensor([nb], dtype=torch.int32).cuda()
    pkv.paged_block_swap(d[0], d[1], bad, st, pkv.SWAP_OUT, k_scales=d[2], v_scales=d[3], scale_staging=sc)
    assert pkv.device_error(reset=True) == pkv.DEV_BAD_PAIR


# ------------------------------------------------------------- PagedKVCache ---
@pytest.mark.parametrize("D,hq,hkv", [(128, 16, 2), (64, 4, 4)])
def test_cache_with_block_scales_forks_and_rotates(pkv, D, hq, hkv):
    """PagedKVCache over block-scaled pools: rotary appends, a fork in the middle of a block, copy-on-write with the
    scales, decode against the definition over the cache as it is, and the shared tokens equal in both sequences."""
    from paged_kv_cache_102_gb300.cache import PagedKVCache
    g = _gen((D, hq, hkv))
    bs = 16
    cache = PagedKVCache(24, hkv, bs, D, block_scales=True)
    freq, factor = pkv.rope_inv_freq(D, scaling="yarn", factor=4.0, original_context=64)
    cache.add_sequence(0, 0)
    rand = lambda n, h: torch.randn(n, h, D, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    for _ in range(21):
        cache.rope_append([0], rand(1, hq), rand(1, hkv), rand(1, hkv), freq, attention_factor=factor)
    cache.fork(0, 1)
    shared = [t.clone() for t in (cache.k_cache, cache.v_cache, cache.k_scales, cache.v_scales)]
    for i in range(14):
        q = cache.rope_append([0, 1], rand(2, hq), rand(2, hkv) * 2.0 ** (i % 5), rand(2, hkv), freq,
                              attention_factor=factor)
        out = cache.decode([0, 1], q, 0.1)
    torch.cuda.synchronize()
    tables, lens = cache.blocks.tables([0, 1])
    assert lens.tolist() == [35, 35] and tables[0, 0] == tables[1, 0] and tables[0, 1] != tables[1, 1]
    want, bound = ref.decode_scaled(ref.f64(q), cache.k_cache.cpu().numpy(), cache.v_cache.cpu().numpy(),
                                    cache.k_scales.cpu().numpy(), cache.v_scales.cpu().numpy(), tables, lens, 0.1, bs,
                                    torch.bfloat16)
    assert np.all(np.abs(ref.f64(out) - want) <= bound)
    old_b = int(tables[0, 1]) if bool((shared[3][int(tables[0, 1])] > 0).any()) else int(tables[1, 1])
    was = ref.VALUES[shared[1][old_b, :, :5].cpu().numpy()] * shared[3][old_b].cpu().numpy()[:, None, None]
    for b in tables[:, 1]:  # the 5 tokens of the shared, partly filled block: values kept (V scales of N(0, 1) rows
        s = cache.v_scales[int(b)].cpu().numpy()[:, None, None]  # move by a doubling or two at most)
        now = ref.VALUES[cache.v_cache[int(b), :, :5].cpu().numpy()] * s
        assert np.all(np.abs(now - was) <= 2.0 ** -9 * s)
    # an appended token without rotation
    cache.append([1], rand(1, hkv), rand(1, hkv))
    assert cache.blocks.context_len(1) == 36


def test_two_streams_with_a_workspace_each(pkv):
    """Two decodes at once on streams of their own, default workspaces: each has its own."""
    case = ("bf16", 32, 4, 128, 16, -1, "wide")
    a, b = (_decode_case(case[:6] + (k,), LENS) for k in ("wide", "narrow"))
    da, db = [t.cuda() for t in a], [t.cuda() for t in b]
    run = lambda d: pkv.paged_attention_decode_scaled(d[0], d[1], d[2], d[3], d[4], d[5], d[6], 0.1)  # noqa: E731
    want = run(da), run(db)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        for s, d in ((s1, da), (s2, db)):
            with torch.cuda.stream(s):
                got.append(run(d))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])


def test_captured_calls_keep_a_workspace_of_their_own(pkv):
    """A captured call without a workspace, then eager calls that need a larger one on the same stream: the replay's
    result stays, and so does that of a second graph captured on it."""
    case = ("bf16", 32, 4, 128, 16, -1, "narrow")
    small, large = (_decode_case(case, lens) for lens in ([700, 1025], [1500] * 12))
    d, e = [t.cuda() for t in small], [t.cuda() for t in large]
    run = lambda t, out=None: pkv.paged_attention_decode_scaled(*t[:7], 0.1, out=out)  # noqa: E731
    want, out1, out2 = run(d), torch.empty_like(d[0]), torch.empty_like(d[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(d)
    torch.cuda.synchronize()
    graphs = []
    for out in (out1, out2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            run(d, out)
    with torch.cuda.stream(s):
        first = run(e)
        junk = [torch.full((1 << 20,), 77, dtype=torch.uint8, device="cuda") for _ in range(8)]
        graphs[0].replay()
        second = run(e)
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(out1, want) and torch.equal(out2, want) and torch.equal(first, second)
    assert all(bool((j == 77).all()) for j in junk)


def test_graphs_of_two_plans_at_once(pkv):
    """Two plans made on one stream, their graphs replayed on two: neither reads the other's partial results."""
    case = ("bf16", 32, 4, 128, 16, -1, "wide")
    s = torch.cuda.Stream()
    data, graphs, plans = [], [], []
    for kind in ("wide", "narrow"):
        d = [t.cuda() for t in _decode_case(case[:6] + (kind,), LENS)]
        torch.cuda.synchronize()
        plan = pkv.DecodePlan(d[0], d[1], d[2], d[5], d[6], 0.1, k_scales=d[3], v_scales=d[4], stream=s)
        plan.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan.run()
        data.append(d), graphs.append(graph), plans.append(plan)
    want = [pkv.paged_attention_decode_scaled(*d[:7], 0.1) for d in data]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p.out, w) for p, w in zip(plans, want))


@pytest.mark.parametrize("case", [("bf16", 16, 2, 128, 16, -1, "narrow"), ("f16", 8, 2, 128, 16, -1, "narrow"),
                                  ("bf16", 8, 1, 64, 16, -1, "narrow"), ("bf16", 4, 2, 128, 16, -1, "narrow")],
                         ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_decode_scaled_infinite_query(pkv, case, bad):
    """A head whose query holds an infinity or a NaN comes out NaN; the heads of its group are not touched."""
    lens = [256, 41, 200] if case[1] == 4 else [700, 41, 200]  # (at most 256: the CUDA-core kernel)
    host = _decode_case(case, lens)
    q, kc, vc, ks, vs, tables, L = (t.cuda() for t in host[:5] + (host[5][:, :-1].contiguous(), host[6]))
    run = lambda q: pkv.paged_attention_decode_scaled(q, kc, vc, ks, vs, tables, L, 0.1)  # noqa: E731
    want = run(q)
    q[0, 1, 3] = bad
    got = run(q)
    assert bool(torch.isnan(got[0, 1]).all())
    got[0, 1] = want[0, 1]
    if case[1] != 4:
        assert torch.equal(got, want)
    else:  # binary32 instead of binary16 products for this group: not the same bits
        exact, bound = ref.decode_scaled(*map(ref.f64, host[:1]), *(t.numpy() for t in host[1:6]), lens, 0.1, case[4],
                                         q.dtype)
        assert (np.abs(ref.f64(got) - exact) <= bound).all()


def test_decode_scaled_v_scales_far_apart(pkv):
    """V scales that fall by more than 2^118 over the blocks, and that rise by as much: the largest dominate."""
    for hq, hkv in ((2, 2), (16, 2)):
        for falling in (True, False):
            case = ("bf16", hq, hkv, 128, 16, -1, "narrow")
            q, kc, vc, ks, vs, tables, L = _decode_case(case, [96])
            steps = torch.exp2(torch.tensor([60., 60., -20., -20., -64., -64.]))
            vs[tables[0, :6].long()] = (steps if falling else steps.flip(0))[:, None].expand(6, hkv).contiguous()
            host = (q, kc, vc, ks, vs, tables, L)
            out = pkv.paged_attention_decode_scaled(*(t.cuda() for t in host), 128 ** -0.5)
            want, bound = ref.decode_scaled(ref.f64(q), kc.numpy(), vc.numpy(), ks.numpy(), vs.numpy(), tables.numpy(),
                                            [96], 128 ** -0.5, 16, q.dtype)
            assert (np.abs(ref.f64(out) - want) <= bound).all()


def test_empty_batches(pkv):
    z = dict(device="cuda")
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, **z)
    s = torch.zeros(4, 2, **z)
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, **z)
    slots, pos = torch.zeros(0, dtype=torch.int64, **z), torch.zeros(0, dtype=torch.int32, **z)
    pkv.paged_kv_append_scaled(k, k, slots, kc, kc.clone(), s, s.clone())
    assert pkv.paged_rope_append(k, k, k, pos, slots, torch.ones(32, **z), kc, kc.clone(), k_scales=s,
                                 v_scales=s.clone()).shape == k.shape
    out = pkv.paged_attention_decode_scaled(k, kc, kc.clone(), s, s.clone(), torch.zeros(0, 3, dtype=torch.int32, **z),
                                            pos, 0.1)
    assert out.shape == k.shape
    assert s.count_nonzero() == 0 and kc.count_nonzero() == 0


def test_large_offsets_in_a_pool_past_2_31_elements(pkv):
    """Blocks whose element offsets pass 32 bits: append and decode there equal those in a small pool."""
    H, bs, D = 8, 16, 128
    nb = (1 << 31) // (H * bs * D) + 9
    g = _gen("large")
    k = torch.randn(40, H, D, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(1, 32, D, generator=g).to(torch.bfloat16).cuda()
    got = []
    for blocks, n in (([nb - 1, nb - 2, nb - 5], nb), ([2, 0, 1], 4)):
        kc, vc = (torch.zeros(n, H, bs, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(n, H, device="cuda") for _ in range(2))
        at = torch.arange(40)
        slots = (torch.tensor(blocks)[at // bs] * bs + at % bs).cuda()
        pkv.paged_kv_append_scaled(k, -k, slots, kc, vc, ks, vs)
        tables = torch.tensor([blocks], dtype=torch.int32).cuda()
        got.append((kc[blocks].cpu(), ks[blocks].cpu(), vc[blocks].cpu(), pkv.paged_attention_decode_scaled(
            q, kc, vc, ks, vs, tables, torch.tensor([40], dtype=torch.int32).cuda(), 0.1).cpu()))
        del kc, vc
    assert all(torch.equal(a, b) for a, b in zip(*got))
