"""Float64 statements of the block-scaled operators, written from their definitions: the oracle of
tests/test_gpu_scaled.py and tests/test_gpu_rope.py.  Nothing here runs the library."""
from __future__ import annotations

import numpy as np
import torch

import oracle

VALUES = oracle.decode_elements(np.arange(256, dtype=np.uint8), oracle.E4M3)  # code -> value, NaN at 0x7f, 0xff
_POS = VALUES[:127]  # 0 .. 448, ascending with the code


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy().astype(np.float64)


def encode(x) -> np.ndarray:
    """float64 -> the nearest E4M3 code, ties to the even code, saturating; NaN -> 0x7f with its sign dropped."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_POS, np.where(np.isnan(a), 0.0, a)), 0, 126)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 448.0, 126, code)
    code = np.where(np.isnan(x), 0x7F, code | (np.signbit(x).astype(np.int64) << 7))
    return code.astype(np.uint8)


def need_scale(rows: np.ndarray) -> np.ndarray:
    """Least power of two 2^e, -64 <= e <= 120, with max|x| <= 448 * 2^e over the finite x of [n, H, D]; [H]."""
    a = np.where(np.isfinite(rows), np.abs(rows), 0.0).max(axis=(0, 2))
    out = np.empty(a.shape)
    for h, top in enumerate(a):
        e = -64
        while top > 448.0 * 2.0 ** e and e < 120:
            e += 1
        out[h] = 2.0 ** e
    return out


def runs(slots, bs):
    """(first token, length) of each maximal stretch of neighbours with consecutive slots of one block."""
    out, t, T = [], 0, len(slots)
    while t < T:
        n = 1
        if slots[t] >= 0:
            while t + n < T and slots[t + n] == slots[t] + n and slots[t + n] % bs != 0:
                n += 1
            out.append((t, n))
        t += n
    return out


def append_scaled(x, slots, codes, scales, bs):
    """Rows x [T, H, D] (float64) into copies of codes uint8 [NB, H, bs, D] and scales float32 [NB, H]."""
    codes, scales = codes.copy(), scales.astype(np.float32).copy()
    limit = codes.shape[0] * bs
    slots = [s if s < limit else -1 for s in slots]
    for t, n in runs(slots, bs):
        b, off = divmod(int(slots[t]), bs)
        rows = x[t:t + n]
        need = need_scale(rows).astype(np.float32)
        for h in range(x.shape[1]):
            old = np.float32(0) if off == 0 else scales[b, h]
            new = old if old > need[h] else need[h]
            if old > 0 and new > old:
                ratio = np.float32(old) / np.float32(new)
                keep = [r for r in range(bs) if not off <= r < off + n]
                codes[b, h, keep] = encode(VALUES[codes[b, h, keep]].astype(np.float32) * ratio)
            scales[b, h] = new
            with np.errstate(invalid="ignore", over="ignore"):
                codes[b, h, off:off + n] = encode((rows[:, h].astype(np.float32) / new).astype(np.float64))
    return codes, scales


def same_codes(a, b) -> bool:
    """Equal codes, any NaN code equal to any other."""
    a, b = np.asarray(a), np.asarray(b)
    na, nb = (a & 0x7F) == 0x7F, (b & 0x7F) == 0x7F
    return bool(np.array_equal(na, nb) and np.array_equal(a[~na], b[~nb]))


def rotate(x, positions, inv_freq, interleaved, factor):
    """(rotated x, |a| + |b| of each channel's pair times the factor) in float64; inv_freq float32."""
    f = np.asarray(inv_freq, np.float64)
    half = len(f)
    t = np.asarray(positions, np.float64)[:, None] * f
    c, s = np.cos(t)[:, None] * factor, np.sin(t)[:, None] * factor
    y = x.copy()
    mag = np.zeros_like(x)
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (np.abs(a) + np.abs(b)) * abs(factor)
    return y, mag


def decode_scaled(q, kcodes, vcodes, ks, vs, tables, lens, scale, bs, out_dtype):
    """(out, bound) float64 [B, Hq, D] of attention over a block-scaled cache.

    bound is what the kernels' arithmetic may be off by, element by element:
      half a step of the output type, relative to the value;
      2^-8 (bf16) or 2^-11 (fp16) of sum_j p_j |v_j|: a weight enters the tensor-core product as two or three E4M3
      parts (each leaves at most 2^-4 of what it rounds), the CUDA-core product as a binary16 (2^-11) or float32 value;
      2^-17 of the largest p_j |vs_j| for every code: what the last part cannot hold (its least step is 2^-9, half
      of it lost, where the largest weight is between 2^7 and 2^8);
      the scores: q enters as two (bf16) or three (fp16) E4M3 parts, 2^-12 of each element at most or 2^-17 of the
      largest, and 128 float32 additions, 2^-17 of sum |q||k|; a score off by d moves the weights by 2 d relative."""
    B, Hq, D = q.shape
    Hkv = kcodes.shape[1]
    G = Hq // Hkv
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        L = int(lens[b])
        if L <= 0:
            continue
        nb = -(-L // bs)
        t = tables[b, :nb]
        def rows(codes, sc):  # noqa: E306  [Hkv, L, D] values, [Hkv, L] scales
            v = VALUES[codes[t]].transpose(1, 0, 2, 3).reshape(Hkv, nb * bs, D)[:, :L]
            s = np.repeat(np.asarray(sc, np.float64)[t].T, bs, axis=1)[:, :L]
            return v, s
        (kv, ksc), (vv, vsc) = rows(kcodes, ks), rows(vcodes, vs)
        for h in range(Hq):
            kh = h // G
            k, v = kv[kh] * ksc[kh][:, None], vv[kh] * vsc[kh][:, None]
            s = (k @ q[b, h]) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h] = p @ v
            aq, ak = np.abs(q[b, h]), np.abs(k)
            ds = abs(scale) * (2.0 ** -12 * (ak @ aq) + 2.0 ** -17 * aq.max() * ak.sum(1) + 2.0 ** -17 * (ak @ aq))
            live = p > 1e-12  # a token without weight has no say, however large its score's error
            move = min(1.0, 2.0 * ds[live].max())
            spread = p @ np.abs(v)
            wmax = (p * np.abs(vsc[kh])).max()
            parts = 2.0 ** -11 if out_dtype == torch.float16 else 2.0 ** -8
            bound[b, h] = (torch.finfo(out_dtype).eps / 2 * np.abs(out[b, h]) + (parts + move) * spread
                           + 2.0 ** -17 * wmax * np.abs(vv[kh]).sum(0) + 2.0 ** -25)
    return out, bound
