"""The operators that attend to, and keep, a part of a paged cache, and the ones that fill it in chunks.

Each case is one call that a serving program makes for a layer:

  chunk   attention of the new tokens of every sequence (prompts, parts of prompts, drafted tokens, batches of these
          and single tokens) over the paged cache that already holds them; causal, with or without a sliding window
          and first tokens that stay visible
  window  attention of one new token per sequence with a sliding window and first tokens that stay visible
  scored  attention of one new token per sequence that also adds up the weight that every cached token got
  evict   the tokens with the largest accumulated weight, the first and the latest ones moved to a smaller table

Sizes follow the workloads of this repository (paged_kv_cache_102_gb300/workloads.py): 16- and 32-token blocks,
head_dim 64 and 128, 8 to 40 kv heads, contexts up to 32768 tokens.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3_MAX = 448.0


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # five drafted tokens of each of 16 sequences are checked at once
        dict(name="chunk_drafts", op="chunk", batch=16, kind="fixed", new=5, lo=64, hi=4096, hq=32, hkv=8, dim=128,
             act="bf16", cache="act", block_size=16, window=0, sinks=0, pad=0, lens_seed=1),
        # four prompts enter at once, grouped queries
        dict(name="chunk_prompts", op="chunk", batch=4, kind="prompt", new=4096, lo=0, hi=0, hq=64, hkv=8, dim=128,
             act="bf16", cache="act", block_size=16, window=0, sinks=0, pad=0, lens_seed=2),
        # the last part of a long prompt that is taken in parts
        dict(name="chunk_long", op="chunk", batch=1, kind="fixed", new=509, lo=32768, hi=32768, hq=32, hkv=8, dim=128,
             act="f16", cache="act", block_size=32, window=0, sinks=0, pad=3, lens_seed=3),
        # long prompts of a layer with a sliding window
        dict(name="chunk_window_d64", op="chunk", batch=2, kind="prompt", new=8190, lo=0, hi=0, hq=32, hkv=32, dim=64,
             act="f16", cache="act", block_size=16, window=1024, sinks=4, pad=0, lens_seed=4),
        # a step of a busy server over the 8-bit cache with block scales: single tokens and three parts of prompts
        dict(name="chunk_mixed_scaled", op="chunk", batch=51, kind="mixed", new=512, lo=16, hi=4096, hq=32, hkv=8,
             dim=128, act="bf16", cache="scaled", block_size=16, window=0, sinks=0, pad=13, lens_seed=5),
        # the smallest call: four short sequences, 8 heads of 64
        dict(name="window_tiny", op="window", batch=4, lens="uniform", lo=2, hi=41, hq=8, hkv=8, dim=64, act="f16",
             cache="act", block_size=16, window=16, sinks=2, lens_seed=6),
        # ragged lengths, 8 query heads for each kv head
        dict(name="window_gqa", op="window", batch=128, lens="lognormal", lo=16, hi=8192, hq=64, hkv=8, dim=128,
             act="bf16", cache="act", block_size=16, window=1024, sinks=4, lens_seed=7),
        # every query head has its own kv head, 8-bit cache with block scales, a window that ends inside blocks
        dict(name="window_mha_scaled", op="window", batch=64, lens="uniform", lo=256, hi=4096, hq=40, hkv=40, dim=128,
             act="bf16", cache="scaled", block_size=16, window=500, sinks=20, lens_seed=8),
        # a decode step that keeps count of what its tokens are worth
        dict(name="scored_gqa", op="scored", batch=64, lens="uniform", lo=128, hi=4096, hq=64, hkv=8, dim=128,
             act="bf16", cache="act", block_size=16, lens_seed=9),
        # the same with a head of 64 and no shared kv heads, a few sequences
        dict(name="scored_mha_d64", op="scored", batch=5, lens="uniform", lo=100, hi=2048, hq=32, hkv=32, dim=64,
             act="f16", cache="act", block_size=32, lens_seed=10),
        # short caches that just outgrew their budget by a block
        dict(name="evict_step", op="evict", batch=4, lens="uniform", lo=257, hi=272, hkv=8, dim=64, act="f16",
             cache="act", block_size=16, budget=256, recent=64, sinks=4, lens_seed=11),
        # after long prompts: a quarter of the tokens stay
        dict(name="evict_long", op="evict", batch=16, lens="uniform", lo=4096, hi=8192, hkv=8, dim=128, act="bf16",
             cache="act", block_size=16, budget=2048, recent=512, sinks=0, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        c = _drawn(rng)
        w = work(c)
        if w["bytes"] <= 5.5e8 and w["flops"] <= 5e11:  # no more than the largest listed ones
            return c


def _drawn(rng):
    seed = rng.randrange(1 << 30)
    op = rng.choice(["chunk", "chunk", "window", "scored", "evict"])
    dim = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 5, 8, 16, 32, 40])
    c = dict(op=op, dim=dim, hkv=hkv, act=rng.choice(["f16", "bf16"]), block_size=rng.choice([16, 32]), lens_seed=seed)
    if op == "evict":
        hi = _log_int(rng, 20, 8192)
        budget = _log_int(rng, 8, max(9, hi))
        return dict(c, batch=_log_int(rng, 1, max(1, min(64, 500000 // (hi * hkv)))), lens="uniform", lo=1, hi=hi,
                    cache=rng.choice(["act", "e4m3"]), budget=budget, recent=rng.randint(0, budget // 2),
                    sinks=rng.choice([0, 0, 1, 4]))
    group = rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 64])
    window, sinks = _log_int(rng, 1, 4096), rng.choice([0, 1, 4, 16, 33, 128])
    if op == "chunk":
        kind = rng.choice(["fixed", "prompt", "mixed"])
        new = _log_int(rng, 2, 16) if kind == "fixed" and rng.random() < 0.5 else _log_int(rng, 16, 4096)
        hi = 0 if kind == "prompt" else _log_int(rng, 16, 16384)
        # logits of the plain form: batch * heads * new * (new + context)
        most = int(4e9 / (hkv * group * new * (new + hi)))
        hkv = hkv if most else 1
        most = int(4e9 / (hkv * group * new * (new + hi)))
        windowed = rng.random() < 0.4
        return dict(c, hkv=hkv, hq=hkv * group, batch=_log_int(rng, 1, max(1, min(64, most))), kind=kind, new=new, lo=0,
                    hi=hi, cache=rng.choice(["act", "act", "e4m3", "scaled"]), window=window if windowed else 0,
                    sinks=sinks if windowed else 0, pad=rng.choice([0, 0, 1, 9]))
    hi = _log_int(rng, 20, 16000)
    c.update(hq=hkv * group, batch=_log_int(rng, 1, max(1, min(512, 1000000 // (hi * hkv)))), lo=1, hi=hi,
             lens=rng.choice(["uniform", "lognormal"]))
    if op == "window":
        return dict(c, cache=rng.choice(["act", "e4m3", "scaled"]), window=window, sinks=sinks)
    return dict(c, cache=rng.choice(["act", "act", "e4m3"]))


def _lens(case, kind, lo, hi, n, salt=0):
    """n lengths of a case: the same multiset for every seed of its values."""
    rng = random.Random(case["lens_seed"] * 7 + salt)
    if kind == "lognormal":
        return [max(lo, min(hi, int(math.exp(rng.gauss(math.log(min(1024, max(lo, hi // 2))), 1.0))))) for _ in range(n)]
    return [rng.randint(lo, hi) for _ in range(n)]


def _chunk_lens(case):
    """(context length with the new tokens, new tokens) of each sequence of a chunk case."""
    n, new = case["batch"], case["new"]
    before = _lens(case, "uniform", case["lo"], case["hi"], n)
    if case["kind"] == "fixed":  # as many for each; lo and hi count them where they are long enough
        return [max(b, new) for b in before], [new] * n
    if case["kind"] == "prompt":
        many = _lens(case, "uniform", max(1, new // 4), new, n, salt=1)
        return many, many
    many = [new - i if i % 17 == 0 else 1 for i in range(n)]  # parts of prompts among single tokens
    many = [max(1, m) for m in many]
    return [b + m for b, m in zip(before, many)], many


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _pool(case, g, nb):
    """K and V pools, and their scales, of nb blocks: a few channels of the keys are several times the others."""
    hkv, bs, dim = case["hkv"], case["block_size"], case["dim"]
    spread = 1.0 + 3.0 * (torch.rand(hkv, 1, dim, generator=g, device=DEV) < 0.03).float()
    step = max(1, (1 << 26) // (hkv * bs * dim))
    dtype = DT[case["act"]] if case["cache"] == "act" else torch.uint8
    pools = [torch.empty(nb, hkv, bs, dim, dtype=dtype, device=DEV) for _ in range(2)]
    for pool, factor in zip(pools, (spread, torch.ones_like(spread))):
        for i in range(0, nb, step):
            x = _randn(g, min(step, nb - i), hkv, bs, dim) * factor
            if case["cache"] != "act":
                x = (x * 60).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            pool[i:i + step].copy_(x)
    s = dict(kc=pools[0], vc=pools[1])
    if case["cache"] == "e4m3":
        s["kt"], s["vt"] = (torch.tensor([x], device=DEV) for x in (0.016, 0.011))
    if case["cache"] == "scaled":  # magnitudes differ from block to block and head to head
        for name in ("ks", "vs"):
            s[name] = torch.exp2(torch.randint(-8, -4, (nb, hkv), generator=g, device=DEV).float()).contiguous()
    return s


def _tables(counts, perm, first=0):
    """Block tables of sequences with these numbers of blocks, taken from perm in turn."""
    h = torch.tensor(counts, device=DEV)
    col = torch.arange(max(1, max(counts)), device=DEV)
    idx = first + (h.cumsum(0) - h)[:, None] + col
    return torch.where(col < h[:, None], perm[idx.clamp(max=perm.numel() - 1)], 0).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    cpu = random.Random(seed)
    bs = case["block_size"]
    if case["op"] == "chunk":
        lens, new = _chunk_lens(case)
    else:
        lens = _lens(case, case["lens"], case["lo"], case["hi"], case["batch"])
        new = [1] * len(lens)
    order = list(range(len(lens)))
    cpu.shuffle(order)
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    n_blk = [-(-n // bs) for n in lens]
    n_dst = [-(-min(n, case["budget"]) // bs) for n in lens] if case["op"] == "evict" else [0]
    nb = (sum(n_blk) + sum(n_dst)) * 9 // 8 + 1
    perm = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    s = dict(case=case, bs=bs, **_pool(case, g, nb))
    s["tables"] = _tables(n_blk, perm)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    hkv, dim = case["hkv"], case["dim"]
    if case["op"] in ("scored", "evict"):  # accumulated weights: a few tokens have most, the newest none yet
        shape = (len(lens), hkv, max(n_blk) * bs)
        s["scores"] = torch.exp(2.0 * _randn(g, *shape))
        s["scores"][torch.rand(shape, generator=g, device=DEV) < 0.1] = 0.0
        s["scores"] *= torch.arange(shape[2], device=DEV) < s["lens"][:, None, None]
    if case["op"] == "evict":
        s["dst_tables"] = _tables(n_dst, perm, first=sum(n_blk))
        s["scores_out"] = torch.empty_like(s["scores"])
        s["lens_out"] = torch.empty_like(s["lens"])
        s["kept"] = torch.empty(len(lens), hkv, case["budget"], dtype=torch.int32, device=DEV)
        return s
    s["scale"] = 1.0 / math.sqrt(dim)
    rows = sum(new) + case.get("pad", 0)  # rows behind the last sequence belong to nobody
    s["q"] = _randn(g, rows, case["hq"], dim).to(DT[case["act"]])
    s["out"] = torch.zeros_like(s["q"])
    if case["op"] == "chunk":
        s["starts"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
        s["most_new"] = max(new)
    return s


# --------------------------------------------------------------------------- plain forms
def _gather(s, which, tables):
    """The blocks of tables [B, n] as float32 [B, Hkv, n * block_size, dim]."""
    c = s["case"]
    pool, t = s["kc" if which == "k" else "vc"], tables.long()
    x = pool[t]
    x = x.float() if c["cache"] == "act" else x.view(torch.float8_e4m3fn).float()
    if c["cache"] == "e4m3":
        x = x * s["kt" if which == "k" else "vt"]
    if c["cache"] == "scaled":
        x = x * s["ks" if which == "k" else "vs"][t][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _visible(j, pos, window, sinks):
    seen = (j <= pos) & (j >= 0)
    return seen & ((j > pos - window) | (j < sinks)) if window else seen


def _attend(q, k, v, seen):
    """Rows q [B, Hkv, R, D] (scaled), k, v [B, Hkv, L, D] and seen, which broadcasts to [B, Hkv, R, L]: the rows'
    outputs and weights."""
    w = (q @ k.transpose(-1, -2)).masked_fill_(~seen, -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    total = w.sum(-1, keepdim=True)
    return (w @ v) / total, w.div_(total)


def _plain_chunk(s):
    c = s["case"]
    hkv, dim, group = c["hkv"], c["dim"], c["hq"] // c["hkv"]
    starts, lens = s["starts"].long(), s["lens"].long()
    b, n = lens.numel(), s["most_new"]
    new = starts[1:] - starts[:-1]
    i = torch.arange(n, device=DEV)
    rows = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    real = i < new[:, None]
    q = s["q"][rows].float() * s["scale"]  # [B, n, Hq, D]
    q = q.view(b, n, hkv, group, dim).permute(0, 2, 1, 3, 4).reshape(b, hkv, n * group, dim)
    pos = torch.where(real, (lens - new)[:, None] + i, 0).repeat_interleave(group, dim=1)
    k, v = _gather(s, "k", s["tables"]), _gather(s, "v", s["tables"])
    j = torch.arange(k.shape[2], device=DEV)
    o, _ = _attend(q, k, v, _visible(j, pos[..., None], c["window"], c["sinks"])[:, None])
    o = o.view(b, hkv, n, group, dim).permute(0, 2, 1, 3, 4).reshape(b, n, c["hq"], dim)
    s["out"][rows[real]] = o[real].to(s["out"].dtype)


def _plain_window(s):
    c = s["case"]
    b, hkv, dim, bs = c["batch"], c["hkv"], c["dim"], s["bs"]
    lens = s["lens"].long()
    # the tokens that any sequence can see: the first ones and the last ones, none of them twice
    first = torch.arange(c["sinks"], device=DEV).expand(b, -1)
    last = lens[:, None] - c["window"] + torch.arange(c["window"], device=DEV)
    j = torch.cat([torch.where(first < lens[:, None] - c["window"], first, -1), last.clamp(min=-1)], 1)
    at, t = j.clamp(min=0), s["tables"].long()
    blk, off = t.gather(1, at // bs), at % bs

    def tokens(pool, tensor, scales):  # [B, Hkv, n, D]
        x = pool[blk, :, off]
        x = x.float() if c["cache"] == "act" else x.view(torch.float8_e4m3fn).float()
        x = x * s[tensor] if c["cache"] == "e4m3" else x * s[scales][blk][..., None] if c["cache"] == "scaled" else x
        return x.transpose(1, 2)

    q = s["q"].float().view(b, hkv, -1, dim) * s["scale"]
    o, _ = _attend(q, tokens(s["kc"], "kt", "ks"), tokens(s["vc"], "vt", "vs"), (j >= 0)[:, None, None])
    s["out"].copy_(o.reshape(b, c["hq"], dim))


def _plain_scored(s):
    c = s["case"]
    b, hkv, dim = c["batch"], c["hkv"], c["dim"]
    q = s["q"].float().view(b, hkv, -1, dim) * s["scale"]
    k, v = _gather(s, "k", s["tables"]), _gather(s, "v", s["tables"])
    j = torch.arange(k.shape[2], device=DEV)
    o, w = _attend(q, k, v, (j < s["lens"][:, None])[:, None, None])
    s["scores"] += w.sum(2)
    s["out"].copy_(o.reshape(b, c["hq"], dim))


def _plain_evict(s):
    c = s["case"]
    bs, budget, hkv = s["bs"], c["budget"], c["hkv"]
    lens = s["lens"].long()[:, None, None]
    n = s["scores"].shape[2]
    j = torch.arange(n, device=DEV)
    must = (j < min(c["sinks"], budget)) | (j >= lens - c["recent"])
    worth = torch.where(must, math.inf, s["scores"]).masked_fill(j >= lens, -1.0)
    best = torch.sort(worth, dim=-1, descending=True, stable=True)[1][..., :budget]  # ties: the earliest first
    stays = best < lens
    kept = torch.where(stays, best, n).sort(-1)[0]
    real = kept < n
    s["kept"].fill_(-1)[..., :kept.shape[-1]] = torch.where(real, kept, -1)
    s["lens_out"].copy_(s["lens"].clamp(max=budget))
    at = kept.clamp(max=n - 1)
    s["scores_out"].zero_()[..., :at.shape[-1]] = torch.where(real, s["scores"].gather(2, at), 0.0)
    to = torch.arange(at.shape[-1], device=DEV)
    b = torch.arange(lens.shape[0], device=DEV)[:, None, None]
    h = torch.arange(hkv, device=DEV)[:, None]
    src = s["tables"].long()[b, at // bs]
    dst = s["dst_tables"].long()[b, (to // bs).clamp(max=s["dst_tables"].shape[1] - 1)]
    b, h, to, at, src, dst = (x.expand(at.shape)[real] for x in (b, h, to, at, src, dst))
    s["kc"][dst, h, to % bs] = s["kc"][src, h, at % bs]
    s["vc"][dst, h, to % bs] = s["vc"][src, h, at % bs]


# --------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import paged_kv_cache_102_gb300 as pkv
        if op == "evict":
            pkv.paged_kv_evict(s["kc"], s["vc"], s["scores"], s["tables"], s["lens"], s["dst_tables"], c["budget"],
                               c["recent"], sinks=c["sinks"], scores_out=s["scores_out"], lens_out=s["lens_out"],
                               kept=s["kept"])
        else:
            scales = dict(k_scale=s.get("kt"), v_scale=s.get("vt"))
            if op != "scored":
                scales.update(k_scales=s.get("ks"), v_scales=s.get("vs"))
            if op == "chunk":
                pkv.paged_attention_chunk(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["starts"], s["scale"],
                                          window=c["window"] or None, sinks=c["sinks"], out=s["out"], **scales)
            elif op == "window":
                pkv.paged_attention_decode_window(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["scale"],
                                                  c["window"], sinks=c["sinks"], out=s["out"], **scales)
            else:
                pkv.paged_attention_decode_scored(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["scale"],
                                                  s["scores"], out=s["out"], **scales)
    elif op == "chunk":
        _plain_chunk(s)
    elif op == "window":
        _plain_window(s)
    elif op == "scored":
        _plain_scored(s)
    else:
        _plain_evict(s)
    if op == "evict":
        codes = (lambda x: x) if c["cache"] == "act" else (lambda x: x.view(torch.float8_e4m3fn))
        return [s["kept"], s["lens_out"], s["scores_out"], codes(s["kc"]), codes(s["vc"])]
    return [s["out"], s["scores"]] if op == "scored" else [s["out"]]


def _spans(case):
    """(tokens of K and V that some row sees, (row, token) pairs) of each sequence."""
    w, sinks = case.get("window", 0), case.get("sinks", 0)
    if case["op"] == "chunk":
        lens, new = _chunk_lens(case)
    else:
        lens = _lens(case, case["lens"], case["lo"], case["hi"], case["batch"])
        new = [1] * len(lens)
    out = []
    for n, m in zip(lens, new):
        if not w:
            out.append((n, m * n - m * (m - 1) // 2))
            continue
        first = n - m  # position of the first row
        lo = max(0, first - w + 1)
        out.append((n - lo + min(lo, sinks),
                    sum(min(p + 1, w) + min(max(0, p + 1 - w), sinks) for p in range(first, n))))
    return out


def work(case):
    """Bytes that have to be read and written once, and the operations of the products."""
    hkv, dim, bs = case["hkv"], case["dim"], case["block_size"]
    size = 2 if case["cache"] == "act" else 1
    if case["op"] == "evict":
        lens = _lens(case, case["lens"], case["lo"], case["hi"], case["batch"])
        kept = sum(min(n, case["budget"]) for n in lens)
        width = -(-max(lens) // bs) * bs
        return dict(bytes=4 * sum(lens) * hkv + 4 * kept * hkv * dim * size + 4 * case["batch"] * hkv * (case["budget"] + width)
                    + 4 * sum(-(-n // bs) for n in lens), flops=0)
    spans = _spans(case)
    tokens, pairs = sum(t for t, _ in spans), sum(p for _, p in spans)
    new = sum(_chunk_lens(case)[1]) if case["op"] == "chunk" else case["batch"]
    b = 2 * tokens * hkv * dim * size + 4 * new * case["hq"] * dim + 4 * (tokens // bs + len(spans)) + 8 * len(spans)
    if case["cache"] == "scaled":
        b += 8 * hkv * (tokens // bs)
    if case["op"] == "scored":
        b += 8 * tokens * hkv
    return dict(bytes=b, flops=4.0 * pairs * case["hq"] * dim)


# --------------------------------------------------------------------------- the definition in 64 bits
def _exact_tokens(s, b, n):
    """K and V of sequence b's n tokens in float64, [Hkv, n, D] each."""
    c = s["case"]
    t = s["tables"][b, :-(-n // s["bs"])].long()
    out = []
    for pool, one, many in (("kc", "kt", "ks"), ("vc", "vt", "vs")):
        x = s[pool][t]
        x = x.double() if c["cache"] == "act" else x.view(torch.float8_e4m3fn).double()
        if c["cache"] == "e4m3":
            x = x * s[one].double()
        elif c["cache"] == "scaled":
            x = x * s[many][t].double()[..., None, None]
        out.append(x.transpose(0, 1).reshape(c["hkv"], -1, c["dim"])[:, :n])
    return out


def _exact_evict(s):
    """Scores and pools after an eviction, one kv head of one sequence at a time; whole numbers have no such value."""
    c, bs = s["case"], s["bs"]
    pools = [(s[p] if c["cache"] == "act" else s[p].view(torch.float8_e4m3fn)).double() for p in ("kc", "vc")]
    out = torch.zeros_like(s["scores"], dtype=torch.float64)
    src, dst = s["tables"].long(), s["dst_tables"].long()
    for b, n in enumerate(s["lens"].tolist()):
        m = min(n, c["budget"])
        for h in range(c["hkv"]):
            if n <= c["budget"]:
                stay = torch.arange(n, device=DEV)
            else:
                first, last = c["sinks"], n - c["recent"]
                between = s["scores"][b, h, first:last]
                order = torch.argsort(between, descending=True, stable=True)[:m - first - c["recent"]]
                stay = torch.cat([torch.arange(first, device=DEV), first + order, torch.arange(last, n, device=DEV)])
                stay = stay.sort()[0]
            to = torch.arange(m, device=DEV)
            out[b, h, :m] = s["scores"][b, h, stay].double()
            for pool in pools:
                pool[dst[b, to // bs], h, to % bs] = pool[src[b, stay // bs], h, stay % bs]
    return [None, None, out, *pools]


def exact(case, seed):
    if case["op"] == "evict":
        return _exact_evict(prepare(case, seed))
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    hkv, dim, hq = case["hkv"], case["dim"], case["hq"]
    w, sinks = case.get("window", 0), case.get("sinks", 0)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    scores = s["scores"].double() if case["op"] == "scored" else None
    starts = s["starts"].tolist() if case["op"] == "chunk" else list(range(case["batch"] + 1))
    for b, n in enumerate(s["lens"].tolist()):
        k, v = _exact_tokens(s, b, n)
        first = n - (starts[b + 1] - starts[b])
        for r in range(starts[b], starts[b + 1], 512):  # rows r, r + 1, ... of the sequence
            e = min(r + 512, starts[b + 1])
            q = s["q"][r:e].double().view(e - r, hkv, hq // hkv, dim).permute(1, 2, 0, 3)
            logits = (q @ k.transpose(1, 2)[:, None]) * s["scale"]
            p = torch.arange(first + r - starts[b], first + e - starts[b], device=DEV)[:, None]
            j = torch.arange(n, device=DEV)
            hidden = j > p
            if w:
                hidden |= (j <= p - w) & (j >= sinks)
            weights = torch.softmax(logits.masked_fill(hidden, -math.inf), -1)
            out[r:e] = (weights @ v[:, None]).permute(2, 0, 1, 3).reshape(e - r, hq, dim)
            if scores is not None:
                scores[b, :, :n] += weights.sum((1, 2))
    return [out] if scores is None else [out, scores]
