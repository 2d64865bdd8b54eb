"""The operators of one step over a paged cache held in 8 bits with a scale for each block and head.

Each case is one call that a serving program makes between the projections of a layer and its output
projection, or once per step before the first layer:

  extend  block tables, slots and positions of a step's tokens, made on the GPU from request lengths
  rope    rotary positions for queries and keys, the rotated keys and the values stored into the cache
  append  keys and values quantised into E4M3 blocks, one scale for each block and kv head
  decode  attention of one new token per sequence over such a cache, through its block table

Sizes follow the workloads of this repository (paged_kv_cache_102_gb300/workloads.py): 16- and 32-token
blocks, head_dim 64 and 128, 8 to 40 kv heads, 4 to 4096 sequences, contexts up to 32768 tokens.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3_MAX = 448.0
SCALE_MIN_EXP, SCALE_MAX_EXP = -64, 120  # block scales are powers of two within these


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a Llama-7B-shaped batch: a slot for each sequence, before the first layer runs
        dict(name="extend_decode_64", op="extend", batch=64, lens="uniform", lo=128, hi=2048, new_lo=1, new_hi=1,
             block_size=16, lens_seed=1),
        # 64 prompts of a batch enter at once: about 260 thousand tokens get their slots and positions
        dict(name="extend_prompts_64", op="extend", batch=64, lens="uniform", lo=0, hi=0, new_lo=129, new_hi=8190,
             block_size=32, lens_seed=2),
        # one decode step with grouped queries at far positions of a context that was stretched 8 times
        dict(name="rope_decode_gqa", op="rope", batch=128, prompt=False, hq=64, hkv=8, dim=128, rot=128,
             interleaved=False, act="bf16", cache="act", block_size=16, pos_hi=131071, stretch=8.0, lens_seed=3),
        # prompts, a quarter of each head rotated, neighbouring channels paired, binary16 cache
        dict(name="rope_prompt_partial", op="rope", batch=5, prompt=True, hq=32, hkv=32, dim=128, rot=32,
             interleaved=True, act="f16", cache="act", block_size=16, pos_hi=2048, stretch=1.0, lens_seed=4),
        # a batch of long prompts into the 8-bit cache with block scales
        dict(name="rope_prompt_scaled", op="rope", batch=9, prompt=True, hq=64, hkv=8, dim=128, rot=128,
             interleaved=False, act="bf16", cache="scaled", block_size=16, pos_hi=4096, stretch=1.0, lens_seed=5),
        # the new token of each of 256 sequences with 40 kv heads; most land in a block that has tokens already
        dict(name="append_decode_256", op="append", batch=256, prompt=False, hkv=40, dim=128, act="bf16",
             block_size=16, hi=4096, lens_seed=6),
        # prompts whose last blocks are partly filled, 32-token blocks, binary16 keys
        dict(name="append_prompt", op="append", batch=13, prompt=True, hkv=8, dim=128, act="f16", block_size=32,
             hi=4096, lens_seed=7),
        # the smallest call: four short sequences, 8 heads of 64
        dict(name="decode_tiny", op="decode", batch=4, lens="uniform", lo=2, hi=41, hq=8, hkv=8, dim=64,
             act="f16", block_size=16, lens_seed=8),
        # ragged lengths, 8 query heads for each kv head
        dict(name="decode_gqa", op="decode", batch=128, lens="lognormal", lo=16, hi=8192, hq=64, hkv=8, dim=128,
             act="bf16", block_size=16, lens_seed=9),
        # 13B-shaped: every query head has its own kv head
        dict(name="decode_mha", op="decode", batch=64, lens="uniform", lo=256, hi=4096, hq=40, hkv=40, dim=128,
             act="bf16", block_size=16, lens_seed=10),
        # few long contexts: the length has to be split over the GPU
        dict(name="decode_long", op="decode", batch=8, lens="uniform", lo=32768, hi=32768, hq=32, hkv=8, dim=128,
             act="bf16", block_size=16, lens_seed=11),
        # head_dim 64, 32-token blocks, binary16
        dict(name="decode_gqa_d64", op="decode", batch=96, lens="lognormal", lo=1, hi=8192, hq=64, hkv=8, dim=64,
             act="f16", block_size=32, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    seed = rng.randrange(1 << 30)
    op = rng.choice(["extend", "rope", "append", "decode", "decode"])
    bs = rng.choice([16, 32])
    if op == "extend":
        if rng.random() < 0.5:  # decode steps, among them wide batches and several tokens per sequence
            n = rng.choice([1, 1, 2, 5])
            return dict(op="extend", batch=_log_int(rng, 1, 4096), lens="uniform", lo=0, hi=_log_int(rng, 16, 2048),
                        new_lo=n if n == 1 else 0, new_hi=n, block_size=bs, lens_seed=seed)
        return dict(op="extend", batch=_log_int(rng, 1, 64), lens="uniform", lo=0, hi=_log_int(rng, 1, 2048),
                    new_lo=0, new_hi=_log_int(rng, 40, 4000), block_size=bs, lens_seed=seed)
    dim = rng.choice([64, 128])
    act = rng.choice(["f16", "bf16"])
    hkv = rng.choice([1, 2, 4, 5, 8, 16, 32, 40])
    if op == "rope":
        prompt = rng.random() < 0.5
        hq = min(64, hkv * rng.choice([1, 2, 4, 8]))
        hq = hq - hq % hkv
        return dict(op="rope", batch=_log_int(rng, 1, 6) if prompt else _log_int(rng, 1, 512), prompt=prompt, hq=hq,
                    hkv=hkv, dim=dim, rot=rng.choice([dim, dim, dim // 2, dim // 4, 24]),
                    interleaved=rng.random() < 0.5, act=act, cache=rng.choice(["act", "e4m3", "scaled"]),
                    block_size=bs, pos_hi=_log_int(rng, 20, 2048) if prompt else _log_int(rng, 100, 1000000),
                    stretch=rng.choice([1.0, 1.0, 4.0, 16.0]), lens_seed=seed)
    if op == "append":
        prompt = rng.random() < 0.5
        return dict(op="append", batch=_log_int(rng, 1, 8) if prompt else _log_int(rng, 1, 512), prompt=prompt, hkv=hkv,
                    dim=rng.choice([64, 128, 128, 80]), act=act, block_size=bs, hi=_log_int(rng, 10, 3000), lens_seed=seed)
    group = rng.choice([1, 2, 4, 8])
    hi = _log_int(rng, 20, 16000)
    batch = _log_int(rng, 1, max(1, min(512, 1000000 // (hi * hkv))))
    return dict(op="decode", batch=batch, lens=rng.choice(["uniform", "lognormal"]), lo=1, hi=hi, hq=hkv * group, hkv=hkv,
                dim=dim, act=act, block_size=bs, lens_seed=seed)


def _lens(case, kind, lo, hi, n, salt=0):
    """n lengths of a case: the same multiset for every seed of its values."""
    rng = random.Random(case["lens_seed"] * 7 + salt)
    if kind == "lognormal":
        return [max(lo, min(hi, int(math.exp(rng.gauss(math.log(min(1024, max(lo, hi // 2))), 1.0))))) for _ in range(n)]
    return [rng.randint(lo, hi) for _ in range(n)]


def _step_lens(case):
    """(tokens already there, new tokens) of each request of an append, rope or extend case."""
    n = case["batch"]
    if case["op"] == "extend":
        return (_lens(case, case["lens"], case["lo"], case["hi"], n),
                _lens(case, "uniform", case["new_lo"], case["new_hi"], n, salt=1))
    hi = case["pos_hi"] if case["op"] == "rope" else case["hi"]
    if case["prompt"]:  # prompts of many lengths
        return [0] * n, _lens(case, "uniform", max(1, hi // 4), hi, n, salt=1)
    return _lens(case, "uniform", 0, hi - 1, n), [1] * n


def _inv_freq(case):
    """Inverse frequencies of the rotated pairs, as a model keeps them (float32).  A stretched context divides the
    slow ones (fewer than one turn over the original length) by the stretch, keeps the fast ones (more than 32
    turns) and blends those between."""
    half = case["rot"] // 2
    f = torch.arange(half, dtype=torch.float64) * (2.0 / case["rot"])
    f = 10000.0 ** -f
    s = case["stretch"]
    if s != 1.0:
        turns = 4096.0 * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / s * (1 - keep)
    return f.to(torch.float32), (0.1 * math.log(s) + 1.0)


def _two_to(e, dtype):
    """2^e for whole e from -127 to 127, without a rounding."""
    return torch.tensor([2.0 ** i for i in range(-127, 128)], dtype=dtype, device=DEV)[e.long() + 127]


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _codes(g, *shape):
    """E4M3 codes of keys or values whose largest magnitude in a block is near the top of the type."""
    x = torch.empty(shape, dtype=torch.uint8, device=DEV)
    rows = x.view(shape[0], -1)
    step = max(1, (1 << 26) // rows.shape[1])
    for i in range(0, shape[0], step):
        part = rows[i:i + step]
        part.copy_((_randn(g, *part.shape) * 80).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8))
    return x


def _spread(g, heads, dim):
    """Channel magnitudes of keys: a few channels are several times the others."""
    return 1.0 + 5.0 * (torch.rand(heads, dim, generator=g, device=DEV) < 0.03).float()


def prepare(case, seed):
    g = _gen(seed)
    cpu = random.Random(seed)
    bs = case["block_size"]
    s = dict(case=case, bs=bs)
    if case["op"] in ("extend", "append", "rope"):
        ctx, new = _step_lens(case)
        order = list(range(len(ctx)))
        cpu.shuffle(order)
        ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    if case["op"] == "extend":
        max_blocks = max(-(-(c + n) // bs) for c, n in zip(ctx, new)) + 1
        have = [-(-c // bs) for c in ctx]
        take = sum(-(-(c + n) // bs) - h for c, n, h in zip(ctx, new, have))
        nb = (sum(have) + take) * 5 // 4 + 8
        perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
        col = torch.arange(max_blocks, device=DEV)
        h = torch.tensor(have, device=DEV)
        used = h.cumsum(0) - h
        tables = torch.where(col < h[:, None], perm[(used[:, None] + col).clamp(max=nb - 1)], 0).to(torch.int32)
        free = perm[sum(have):].contiguous()
        total = sum(new)
        i32 = dict(dtype=torch.int32, device=DEV)
        s.update(tables=tables.contiguous(), ctx=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32), free=free,
                 head=torch.tensor([cpu.randrange(0, free.numel() - take + 1)], **i32), num_blocks=nb,
                 slots=torch.empty(total + 7, dtype=torch.int64, device=DEV), positions=torch.empty(total + 7, **i32),
                 seq_starts=torch.empty(len(ctx) + 1, **i32), block_starts=torch.empty(len(ctx) + 1, **i32),
                 lens=torch.empty(len(ctx), **i32), head_out=torch.empty(1, **i32))
        return s
    act = DT[case["act"]]
    hkv, dim = case["hkv"], case["dim"]
    if case["op"] == "decode":
        lens = _lens(case, case["lens"], case["lo"], case["hi"], case["batch"])
        cpu.shuffle(lens)
        n_blk = [-(-n // bs) for n in lens]
        nb = sum(n_blk) * 5 // 4 + 1
        perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
        h = torch.tensor(n_blk, device=DEV)
        col = torch.arange(max(n_blk), device=DEV)
        idx = (h.cumsum(0) - h)[:, None] + col
        s["tables"] = torch.where(col < h[:, None], perm[idx.clamp(max=nb - 1)], 0).to(torch.int32).contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = _randn(g, case["batch"], case["hq"], dim).to(act)
        s["kc"], s["vc"] = _codes(g, nb, hkv, bs, dim), _codes(g, nb, hkv, bs, dim)
        # magnitudes differ from block to block and head to head
        for name in ("ks", "vs"):
            e = torch.randint(-9, -4, (nb, hkv), generator=g, device=DEV)
            s[name] = torch.exp2(e.float()).contiguous()
        s["scale"] = 1.0 / math.sqrt(dim)
        s["out"] = torch.empty_like(s["q"])
        return s
    # append and rope: each request has the block of its first new token and the blocks after it
    first = [c // bs for c in ctx]
    n_blk = [-(-(c + n) // bs) - f for c, n, f in zip(ctx, new, first)]
    nb = sum(n_blk) * 5 // 4 + 4
    perm = torch.randperm(nb, generator=g, device=DEV)
    t_seq = torch.repeat_interleave(torch.arange(len(ctx), device=DEV), torch.tensor(new, device=DEV))
    start = torch.tensor(new, device=DEV).cumsum(0) - torch.tensor(new, device=DEV)
    T = int(sum(new))
    pos = torch.tensor(ctx, device=DEV)[t_seq] + torch.arange(T, device=DEV) - start[t_seq]
    blk0 = torch.tensor(n_blk, device=DEV).cumsum(0) - torch.tensor(n_blk, device=DEV)
    phys = perm[blk0[t_seq] + pos // bs - torch.tensor(first, device=DEV)[t_seq]]
    s["slots"] = (phys * bs + pos % bs).to(torch.int64).contiguous()
    hq = case.get("hq", 0)
    qkv = _randn(g, T, (hq + 2 * hkv), dim)
    qkv[:, hq:hq + hkv] *= _spread(g, hkv, dim)
    qkv = qkv.to(act).reshape(T, -1)
    s["q"] = qkv[:, :hq * dim].unflatten(1, (hq, dim)) if hq else None
    s["k"] = qkv[:, hq * dim:(hq + hkv) * dim].unflatten(1, (hkv, dim))
    s["v"] = qkv[:, (hq + hkv) * dim:].unflatten(1, (hkv, dim))
    if case["op"] == "append":
        s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
    cache = case.get("cache", "scaled")
    if cache == "act":
        s["kc"], s["vc"] = (_randn(g, nb, hkv, bs, dim).to(act) for _ in range(2))
    else:
        s["kc"], s["vc"] = _codes(g, nb, hkv, bs, dim), _codes(g, nb, hkv, bs, dim)
    if cache == "e4m3":
        s["kt"], s["vt"] = (torch.tensor([x], device=DEV) for x in (0.06, 0.011))
    if cache == "scaled":  # about a quarter of the partly filled blocks get a larger value than they hold
        for name in ("ks", "vs"):
            s[name] = torch.exp2(torch.randint(-8, -4, (nb, hkv), generator=g, device=DEV).float()).contiguous()
    if case["op"] == "rope":
        f, factor = _inv_freq(case)
        s["inv_freq"], s["factor"] = f.to(DEV), factor
        s["positions"] = pos.to(torch.int32).contiguous()
        s["q_out"] = torch.empty(T, hq, dim, dtype=act, device=DEV)
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_extend(s):
    bs = s["bs"]
    ctx, new = s["ctx"].long(), s["new"].long()
    zero = ctx.new_zeros(1)
    have = (ctx + bs - 1) // bs
    need = (ctx + new + bs - 1) // bs
    starts = torch.cat([zero, new.cumsum(0)])
    blocks = torch.cat([zero, (need - have).cumsum(0)])
    col = torch.arange(s["tables"].shape[1], device=DEV)
    idx = s["head"].long() + blocks[:-1, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    taken = s["free"][idx.clamp(0, s["free"].numel() - 1)]
    s["tables"].copy_(torch.where(fresh, taken, s["tables"]))
    t = torch.arange(s["slots"].numel(), device=DEV)
    real = t < starts[-1]
    seq = torch.searchsorted(starts[1:], t, right=True).clamp(max=ctx.numel() - 1)
    pos = torch.where(real, ctx[seq] + t - starts[seq], 0)
    slot = s["tables"][seq, pos // bs].long() * bs + pos % bs
    s["slots"].copy_(torch.where(real, slot, -1))
    s["positions"].copy_(torch.where(real, pos, -1))
    s["seq_starts"].copy_(starts)
    s["block_starts"].copy_(blocks)
    s["lens"].copy_(ctx + new)
    s["head_out"].copy_(s["head"] + blocks[-1])


def _to_e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_store(x, slots, bs, cache, scales):
    """Quantise rows x [T, H, D] (float32) into the blocks of their slots, each block and head with one scale."""
    blk, off = slots // bs, slots % bs
    touched = torch.unique(blk)
    amax = x.abs().amax(-1)
    top = torch.zeros_like(scales).index_reduce_(0, blk, amax, "amax", include_self=True)[touched]
    fresh = torch.zeros(scales.shape[0], dtype=torch.bool, device=DEV)
    fresh[blk[off == 0]] = True
    fresh = fresh[touched][:, None]
    m, e = torch.frexp(top)
    # the least power of two whose 448-fold reaches the largest magnitude (448 = 0.875 * 2^9)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(top == 0, SCALE_MIN_EXP, e).clamp(SCALE_MIN_EXP, SCALE_MAX_EXP)
    need = _two_to(e, torch.float32)
    old = scales[touched]
    now = torch.where(fresh, need, torch.maximum(need, old))
    ratio = torch.where(fresh, 1.0, old / now)
    kept = cache[touched].view(torch.float8_e4m3fn).float() * ratio[:, :, None, None]
    cache[touched] = _to_e4m3(kept)
    scales[touched] = now
    cache[blk, :, off] = _to_e4m3(x / scales[blk][:, :, None])


def _plain_append(s):
    _plain_store(s["k"].float(), s["slots"], s["bs"], s["kc"], s["ks"])
    _plain_store(s["v"].float(), s["slots"], s["bs"], s["vc"], s["vs"])


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    ang = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = ((f(ang) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]))
    k, v = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"]), s["v"].float()
    blk, off = s["slots"] // s["bs"], s["slots"] % s["bs"]
    if c["cache"] == "act":
        s["kc"][blk, :, off] = k.to(s["kc"].dtype)
        s["vc"][blk, :, off] = s["v"]
    elif c["cache"] == "e4m3":
        s["kc"][blk, :, off] = _to_e4m3(k / s["kt"])
        s["vc"][blk, :, off] = _to_e4m3(v / s["vt"])
    else:
        _plain_store(k, s["slots"], s["bs"], s["kc"], s["ks"])
        _plain_store(v, s["slots"], s["bs"], s["vc"], s["vs"])


def _plain_decode(s):
    c = s["case"]
    b, hq, dim = s["q"].shape
    hkv, bs = c["hkv"], s["bs"]
    t = s["tables"].long()

    def gathered(cache, scales):  # [B, Hkv, L, D] in float32
        x = cache[t].view(torch.float8_e4m3fn).float() * scales[t][..., None, None]
        return x.transpose(1, 2).reshape(b, hkv, -1, dim)

    q = s["q"].float().view(b, hkv, hq // hkv, dim) * s["scale"]
    logits = q @ gathered(s["kc"], s["ks"]).transpose(-1, -2)
    live = torch.arange(t.shape[1] * bs, device=DEV) < s["lens"][:, None]
    logits = logits.masked_fill(~live[:, None, None], -math.inf)
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    o = (p @ gathered(s["vc"], s["vs"])) / p.sum(-1, keepdim=True)
    s["out"].copy_(o.reshape(b, hq, dim))


# --------------------------------------------------------------------------- one pass
def _outputs(s):
    op = s["case"]["op"]
    if op == "extend":
        return [s["slots"], s["positions"], s["seq_starts"], s["block_starts"], s["lens"], s["head_out"], s["tables"]]
    if op == "decode":
        return [s["out"]]
    cache = s["case"].get("cache", "scaled")
    kc, vc = s["kc"], s["vc"]
    out = [kc, vc] if cache == "act" else [kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)]
    if cache == "scaled":
        out += [s["ks"], s["vs"]]
    return out if op == "append" else [s["q_out"]] + out


def run(s):
    op = s["case"]["op"]
    if own:
        import paged_kv_cache_102_gb300 as pkv
        if op == "extend":
            pkv.paged_extend_tables(s["tables"], s["ctx"], s["new"], s["free"], s["head"], s["bs"], s["num_blocks"],
                                    slot_mapping=s["slots"], positions=s["positions"], seq_starts=s["seq_starts"],
                                    block_starts=s["block_starts"], context_lens_out=s["lens"],
                                    free_head_out=s["head_out"])
        elif op == "append":
            pkv.paged_kv_append_scaled(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
        elif op == "rope":
            pkv.paged_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["kc"], s["vc"],
                                  interleaved=s["case"]["interleaved"], attention_factor=s["factor"],
                                  q_out=s["q_out"], k_scale=s.get("kt"), v_scale=s.get("vt"), k_scales=s.get("ks"),
                                  v_scales=s.get("vs"))
        else:
            pkv.paged_attention_decode_scaled(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["tables"], s["lens"],
                                              s["scale"], out=s["out"])
    elif op == "extend":
        _plain_extend(s)
    elif op == "append":
        _plain_append(s)
    elif op == "rope":
        _plain_rope(s)
    else:
        _plain_decode(s)
    return _outputs(s)


def work(case):
    """Bytes that have to be read and written once, and the operations of the products."""
    bs = case["block_size"]
    if case["op"] == "decode":
        lens = _lens(case, case["lens"], case["lo"], case["hi"], case["batch"])
        tokens, blocks = sum(lens), sum(-(-n // bs) for n in lens)
        qo = 2 * 2 * case["batch"] * case["hq"] * case["dim"]
        return dict(bytes=2 * tokens * case["hkv"] * case["dim"] + 8 * blocks * case["hkv"] + 4 * blocks + qo
                    + 4 * len(lens), flops=4.0 * tokens * case["hq"] * case["dim"])
    ctx, new = _step_lens(case)
    T = sum(new)
    if case["op"] == "extend":
        taken = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in zip(ctx, new))
        olds = sum(1 for c, n in zip(ctx, new) if c % bs and n)
        return dict(bytes=12 * T + 8 * taken + 4 * olds + 20 * len(ctx), flops=0)
    hkv, dim, hq = case["hkv"], case["dim"], case.get("hq", 0)
    cache = case.get("cache", "scaled")
    kv = T * hkv * dim
    touched = sum(-(-(c + n) // bs) - c // bs for c, n in zip(ctx, new))
    b = 2 * kv * 2 + 2 * kv * (2 if cache == "act" else 1) + 8 * T
    if cache == "scaled":
        b += 2 * 4 * hkv * (touched + sum(1 for c in ctx if c % bs))
    if case["op"] == "rope":
        b += 2 * 2 * T * hq * dim + 4 * T + 2 * case["rot"]
    return dict(bytes=b, flops=3.0 * T * (hq + hkv) * case.get("rot", 0))


# --------------------------------------------------------------------------- the definition in 64 bits
def _e4m3_values(x):
    """float64 -> the nearest E4M3 values, ties to even, saturating."""
    a = x.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(a)  # a = m 2^e with m in [0.5, 1)
    step = _two_to((e - 4).clamp(min=-9), torch.float64)
    return torch.copysign((torch.round(a / step) * step).clamp(max=E4M3_MAX), x)


def _exact_store(x, slots, bs, cache, scales):
    """The block-scaled store, block by block of the call's tokens, in float64: (code values, scales)."""
    vals = cache.view(torch.float8_e4m3fn).double()
    sc = scales.double()
    blk, off = (slots // bs).cpu().tolist(), (slots % bs).cpu().tolist()
    i = 0
    while i < len(blk):
        j = i
        while j + 1 < len(blk) and blk[j + 1] == blk[i]:
            j += 1
        b, rows = blk[i], x[i:j + 1]  # [n, H, D]
        top = rows.abs().amax((0, 2)) / E4M3_MAX
        m, e = torch.frexp(top)  # the power of two at or above it: 0.5 is the mantissa of a power of two
        e = torch.where(top == 0, SCALE_MIN_EXP, torch.where(m == 0.5, e - 1, e)).clamp(SCALE_MIN_EXP, SCALE_MAX_EXP)
        need = _two_to(e, torch.float64)
        now = need if off[i] == 0 else torch.maximum(need, sc[b])
        if off[i] != 0:
            vals[b] = _e4m3_values(vals[b] * (sc[b] / now)[:, None, None])
        sc[b] = now
        vals[b, :, off[i]:off[j] + 1] = _e4m3_values(rows.transpose(0, 1) / now[:, None, None])
        i = j + 1
    return vals, sc


def _exact_rotate(x, ang, factor, rot, interleaved):
    z = x.double().clone()
    c, s = torch.cos(ang)[:, None] * factor, torch.sin(ang)[:, None] * factor
    i = torch.arange(rot // 2, device=DEV)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    za, zb = z[..., a], z[..., b]
    z[..., a], z[..., b] = za * c - zb * s, za * s + zb * c
    return z


def exact(case, seed):
    if case["op"] == "extend":  # whole numbers alone
        return None
    s = prepare(case, seed)
    bs = s["bs"]
    if case["op"] == "decode":
        hkv, dim = case["hkv"], case["dim"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lens"].tolist()):
            t = s["tables"][b, :-(-n // bs)].long()
            k, v = ((s[c][t].view(torch.float8_e4m3fn).double() * s[f][t].double()[..., None, None])
                    .transpose(0, 1).reshape(hkv, -1, dim)[:, :n] for c, f in (("kc", "ks"), ("vc", "vs")))
            logits = s["q"][b].double().view(hkv, -1, dim) @ k.transpose(1, 2) * s["scale"]
            out[b] = (torch.softmax(logits, -1) @ v).reshape(-1, dim)
        return [out]
    if case["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        got = [_exact_store(x, s["slots"], bs, s[c], s[f]) for x, c, f in ((k, "kc", "ks"), (v, "vc", "vs"))]
        return [got[0][0], got[1][0], got[0][1], got[1][1]]
    ang = s["positions"].double()[:, None] * s["inv_freq"].double()
    args = (ang, s["factor"], case["rot"], case["interleaved"])
    q, k, v = _exact_rotate(s["q"], *args), _exact_rotate(s["k"], *args), s["v"].double()
    if case["cache"] == "scaled":
        got = [_exact_store(x, s["slots"], bs, s[c], s[f]) for x, c, f in ((k, "kc", "ks"), (v, "vc", "vs"))]
        return [q, got[0][0], got[1][0], got[0][1], got[1][1]]
    out = [q]
    for x, c, f in ((k, "kc", "kt"), (v, "vc", "vt")):
        e4m3 = case["cache"] == "e4m3"
        vals = (s[c].view(torch.float8_e4m3fn) if e4m3 else s[c]).double()
        vals[s["slots"] // bs, :, s["slots"] % bs] = _e4m3_values(x / s[f].double()) if e4m3 else x
        out.append(vals)
    return out
