"""How many bits the block-scaled decode keeps: every output lies between the roundings of the exact value less and
plus what binary32 arithmetic and the parts of the weights may lose, so that a loss far below the output type's own
rounding shows wherever it moves a value across a border."""
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


def _exact(q, kcodes, vcodes, ks, vs, tables, lens, scale, bs, act, tensor_cores):
    """(out, slack) float64 [B, Hq, D].  slack is what an output may be off by before it is rounded:
      sums: a product's and the denominator's 512 binary32 additions, each less than 2^-15 of sum p |v| (CUDA cores:
      at most 64 tokens here, 2^-18 each);
      tensor cores: three E4M3 parts of a weight, 2^-14 of it, or half a step of the last one, 2^-20 where the largest
      weight is above 2^7: 2^-27 of that for every code;
      scores: 128 binary32 additions, 2^-17 of sum |q||k|; two and more parts of q, 2^-22 of the largest |q| (the least
      step of the second part) and, binary16, 2^-14 of each element; 2^-21 of the score and of the weight for the
      exponential.  A score off by d moves the weights by 2 d, relatively."""
    B, Hq, D = q.shape
    Hkv = kcodes.shape[1]
    out, slack = np.zeros(q.shape), np.zeros(q.shape)
    sums, parts = (2.0 ** -14, 2.0 ** -14) if tensor_cores else (2.0 ** -17, 0.0)
    elem = 2.0 ** -14 if tensor_cores and act == "f16" else 0.0
    for b in range(B):
        n = int(lens[b])
        nb = -(-n // bs)
        t = tables[b, :nb]
        vals = lambda c: ref.VALUES[c[t]].transpose(1, 0, 2, 3).reshape(Hkv, nb * bs, D)[:, :n]  # noqa: E731
        scal = lambda s: np.repeat(s.astype(np.float64)[t].T, bs, axis=1)[:, :n]  # noqa: E731
        kv, vv, ksc, vsc = vals(kcodes), vals(vcodes), scal(ks), scal(vs)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k, v = kv[g] * ksc[g][:, None], vv[g] * vsc[g][:, None]
            s = (k @ q[b, h]) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            aq, ak = np.abs(q[b, h]), np.abs(k)
            ds = scale * ((2.0 ** -17 + elem) * (ak @ aq) + 2.0 ** -22 * aq.max() * ak.sum(1)) + 2.0 ** -21 * (1 + abs(s))
            move = np.expm1(2.0 * ds[p > 1e-12].max())
            out[b, h] = p @ v
            slack[b, h] = (sums + parts + move) * (p @ np.abs(v))
            if tensor_cores:
                slack[b, h] += 2.0 ** -27 * (p * np.abs(vsc[g])).max() * np.abs(vv[g]).sum(0)
    return out, slack


def _check(pkv, host, bs, act, tensor_cores, scale):
    q, kc, vc, ks, vs, tables, lens = host
    pkv.set_kernel_path(pkv.PATH_TENSOR if tensor_cores else pkv.PATH_CUDA_CORE)
    out = pkv.paged_attention_decode_scaled(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), tables.cuda(),
                                            lens.cuda(), scale)
    torch.cuda.synchronize()
    want, slack = _exact(ref.f64(q), kc.numpy(), vc.numpy(), ks.numpy(), vs.numpy(), tables.numpy(), lens.numpy(), scale,
                         bs, act, tensor_cores)
    to = lambda x: ref.f64(torch.from_numpy(x).to(DT[act]))  # noqa: E731  (one rounding, from float64)
    got = ref.f64(out)
    ok = (to(want - slack) <= got) & (got <= to(want + slack))
    assert ok.all(), (f"{(~ok).sum()} of {ok.size} outputs off, worst "
                      f"{np.nanmax(np.abs(got - want) / np.maximum(np.abs(want), 1e-30)):.1e}, NaN {np.isnan(got).sum()}")


def _case(name, act, hq, hkv, D, bs, lens, spread):
    """Every query along one direction per kv head, so that scores are near what `spread` says of a sequence's tokens
    (natural logarithms), positive V codes."""
    g = torch.Generator().manual_seed(zlib.crc32(repr((name, act, hq, hkv, D, bs, lens)).encode()))
    n_blk = [-(-n // bs) for n in lens]
    nb = sum(n_blk) + 2
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.zeros(len(lens), max(n_blk), dtype=torch.int32)
    kc = torch.zeros(nb, hkv, bs, D, dtype=torch.uint8)
    vc = torch.randint(0x20, 0x78, (nb, hkv, bs, D), dtype=torch.uint8, generator=g)
    scale = D ** -0.5
    q = torch.rand(len(lens), hq, D, generator=g) * 0.5 + 0.75
    at = 0
    for b, n in enumerate(lens):
        t = perm[at:at + n_blk[b]]
        at += n_blk[b]
        tables[b, :n_blk[b]] = t
        s = spread(n, hkv, g)  # [n, hkv]
        x = (s / (D * scale))[..., None].expand(n, hkv, D) * 2.0 ** 6  # K scales are 2^-6
        pad = torch.zeros(n_blk[b] * bs, hkv, D)
        pad[:n] = x
        kc[t.long()] = (pad.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                        .view(n_blk[b], bs, hkv, D).transpose(1, 2))
    ks = torch.full((nb, hkv), 2.0 ** -6)
    vs = torch.full((nb, hkv), 2.0 ** -5)
    return [q.to(DT[act]), kc, vc, ks, vs, tables, torch.tensor(lens, dtype=torch.int32)], scale


def _sink(n, hkv, g):
    """One token with most of the weight, the rest spread about evenly."""
    s = torch.randn(n, hkv, generator=g) * 0.5 - 7.9 + np.log(512.0 / n)
    s[n // 3] = 0.0
    return s


SHAPES = [("f16", 16, 2, 128, 16), ("bf16", 16, 2, 128, 16), ("f16", 8, 2, 128, 32), ("bf16", 8, 2, 128, 16),
          ("bf16", 3, 3, 128, 32), ("f16", 16, 2, 64, 32), ("bf16", 16, 2, 64, 16), ("f16", 4, 2, 64, 16),
          ("bf16", 2, 2, 64, 32)]


@pytest.mark.parametrize("act,hq,hkv,D,bs", SHAPES)
@pytest.mark.parametrize("zero_v", [True, False])
def test_weights_beside_one_that_dominates(pkv, act, hq, hkv, D, bs, zero_v):
    """A token with 0.84 of the weight and (nearly) no values: the output is what the small weights keep."""
    lens = [512, 511, 300, 1]
    host, scale = _case("sink", act, hq, hkv, D, bs, lens, _sink)
    if zero_v:
        for b, n in enumerate(lens):
            at = n // 3
            host[2][host[5][b, at // bs].long(), :, at % bs] = 0x01
    _check(pkv, host, bs, act, True, scale)


@pytest.mark.parametrize("act,hq,hkv,D,bs", SHAPES)
def test_flat_weights_and_scales_apart(pkv, act, hq, hkv, D, bs):
    """Scores near one another; V scales that differ from block to block by up to 2^12, no powers of two."""
    host, scale = _case("flat", act, hq, hkv, D, bs, [512, 129, 33],
                        lambda n, h, g: torch.randn(n, h, generator=g) * 0.5)
    g = torch.Generator().manual_seed(5)
    host[4] = torch.exp2(torch.rand(host[4].shape, generator=g) * 12 - 10)
    _check(pkv, host, bs, act, True, scale)


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_with_channels_far_above_the_others(pkv, act, D):
    """A channel 2^9 times the others in q, over keys that are zero there: the scores hang on the small ones, which
    are equal in a head, so that what is cut off them adds up."""
    host, scale = _case("outlier", act, 8, 2, D, 16, [200, 64], lambda n, h, g: torch.randn(n, h, generator=g) * 2)
    host[0] = host[0][..., :1].expand(host[0].shape).contiguous()
    host[0][..., 3] = 2.0 ** 9
    host[1][..., 3] = 0
    _check(pkv, host, 16, act, True, scale)


@pytest.mark.parametrize("D,hq,hkv", [(128, 32, 32), (64, 32, 16), (128, 16, 4)])
@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_cuda_core_weights(pkv, act, D, hq, hkv):
    """Short contexts on the CUDA cores: few tokens, one of them without values, so that an output shows a weight."""
    host, scale = _case("short", act, hq, hkv, D, 16, [2] * 12 + [3, 9, 17, 40],
                        lambda n, h, g: torch.rand(n, h, generator=g))
    host[2][host[5][:, 0].long(), :, 0] = 0
    _check(pkv, host, 16, act, False, scale)


@pytest.mark.parametrize("D,hq,hkv", [(128, 2, 2), (64, 4, 2)])
@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_cuda_core_weight_times_scale_near_2_16(pkv, act, D, hq, hkv):
    """Scores just under 2^8 times the running reference's weight, on V scales just under 2^8 times the first ones."""
    host, _ = _case("gap", act, hq, hkv, D, 16, [64], lambda n, h, g: torch.zeros(n, h))
    host[0].fill_(1.0)
    late = host[5][0, 2:].long()
    host[1][late] = 0x38  # 1.0 in the last 32 tokens, 0 before
    host[4].fill_(2.0 ** -12)
    host[4][late] = 2.0 ** -12 * 2.0 ** 7 * 1.9999
    _check(pkv, host, 16, act, False, 7.9999 * np.log(2.0) / (D * 2.0 ** -6))


@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 8), (64, 8, 4)])
@pytest.mark.parametrize("tensor_cores", [False, True])
def test_tiny_bfloat16_queries_over_large_keys(pkv, D, hq, hkv, tensor_cores):
    """Queries near 2^-18, below what binary16 holds exactly, and K scales that make up for it."""
    host, scale = _case("tiny", "bf16", hq, hkv, D, 16, [40, 64, 3], lambda n, h, g: torch.randn(n, h, generator=g) * 2)
    host[0] = host[0][..., :1].expand(host[0].shape).contiguous() * 2.0 ** -18
    host[3].fill_(2.0 ** 12)
    _check(pkv, host, 16, "bf16", tensor_cores, scale)
