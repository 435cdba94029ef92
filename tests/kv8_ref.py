"""Plain 64-bit forms of the 8-bit key/value cache, on the CPU, written from the
definitions: a cache as row-major codes and scales, sequences one at a time."""
from __future__ import annotations

import math

import numpy as np
import torch


def k_tiles(q):
    """Row-major codes [pages][heads][page][d] in the order of k_codes."""
    n, h, p, d = q.shape
    return q.reshape(n, h, p // 16, 16, d // 16, 16).swapaxes(3, 4).reshape(n, h, p, d)


def v_tiles(q):
    n, h, p, d = q.shape
    return q.reshape(n, h, p // 4, 4, d).swapaxes(3, 4).reshape(n, h, p, d)


def k_rows(c):
    n, h, p, d = c.shape
    return c.reshape(n, h, p // 16, d // 16, 16, 16).swapaxes(3, 4).reshape(n, h, p, d)


def v_rows(c):
    n, h, p, d = c.shape
    return c.reshape(n, h, p // 4, d, 4).swapaxes(3, 4).reshape(n, h, p, d)


def rne(x):
    """Nearest integer, ties to even (numpy's rint is)."""
    return np.rint(x)


def write(codes, scales, table, lens, starts, x):
    """Rows x (float64 [n_tok][heads][d]) into row-major int8 codes and float32 scales
    [pages][heads][blocks], in place."""
    pages, heads, p, d = codes.shape
    b = p // scales.shape[2]
    for s in range(len(lens)):
        n = starts[s + 1] - starts[s]
        pos = np.arange(lens[s] - n, lens[s])
        for blk in sorted({int(q) // b for q in pos if q >= 0}):
            mine = [i for i, q in enumerate(pos) if q >= 0 and q // b == blk]
            page = int(table[s][blk * b // p])
            if not 0 <= page < pages:
                continue
            at = blk * b % p
            old = int(pos[mine[0]]) - blk * b  # older tokens of the block
            for h in range(heads):
                new = x[starts[s] + mine[0]:starts[s] + mine[-1] + 1, h]
                s0 = scales[page, h, at // b]
                with np.errstate(all="ignore"):
                    s1 = np.float32(np.float32(np.abs(new).max()) / np.float32(127.0))
                if old and s0 > s1:
                    s1 = s0
                if not np.isfinite(new).all() or (old and np.isnan(s0)):
                    s1 = np.float32(np.nan)
                rows = codes[page, h, at:at + b]
                if old and s1 > s0:
                    rows[:old] = rne(rows[:old].astype(np.float64) * np.float64(s0) / np.float64(s1))
                if np.isnan(s1) or s1 == 0:
                    rows[old:old + len(mine)] = 0
                else:
                    rows[old:old + len(mine)] = np.clip(rne(new / np.float64(s1)), -127, 127)
                scales[page, h, at // b] = s1


def sequence(codes, scales, table_row, length):
    """Values [length][heads][d] in float64 of one sequence; NaN where the page is none of the pool."""
    pages, heads, p, d = codes.shape
    b = p // scales.shape[2]
    out = np.full((length, heads, d), np.nan)
    for at in range(0, length, p):
        page = int(table_row[at // p])
        n = min(p, length - at)
        if 0 <= page < pages:
            v = codes[page].astype(np.float64) * np.repeat(scales[page].astype(np.float64), b, 1)[..., None]
            out[at:at + n] = v[:, :n].swapaxes(0, 1)
    return out


def attention(kcodes, kscales, vcodes, vscales, table, lens, starts, q, scale, window=0, sinks=None):
    """(out, lse, mag, smag, n) in float64: mag = sum w |v| / sum w of each output, smag the largest
    sum |q k| scale of a row's keys, n its keys."""
    n_tok, hq, d = q.shape
    hkv = kcodes.shape[1]
    g = hq // hkv
    out, mag = np.zeros((n_tok, hq, d)), np.zeros((n_tok, hq, d))
    lse, smag = np.full((n_tok, hq), -np.inf), np.zeros((n_tok, hq))
    keys = np.zeros((n_tok, 1))
    if sinks is not None:
        lse[:] = sinks
    for s in range(len(lens)):
        n, length = starts[s + 1] - starts[s], lens[s]
        k = sequence(kcodes, kscales, table[s], length)
        v = sequence(vcodes, vscales, table[s], length)
        for i in range(n):
            pos = length - n + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < lo:
                continue
            t = starts[s] + i
            keys[t] = pos + 1 - lo
            for h in range(hq):
                kh, vh = k[lo:pos + 1, h // g], v[lo:pos + 1, h // g]
                with np.errstate(all="ignore"):
                    z = kh @ q[t, h] * scale
                    smag[t, h] = (np.abs(kh) @ np.abs(q[t, h])).max() * abs(scale)
                    top = max(z.max(), -np.inf if sinks is None else sinks[h])
                    w = np.exp(z - top)
                    total = w.sum() + (0.0 if sinks is None else math.exp(sinks[h] - top))
                    out[t, h] = w @ vh / total
                    mag[t, h] = w @ np.abs(vh) / total
                    lse[t, h] = top + np.log(total)
    return out, lse, mag, smag, keys


def attention_tolerance(out, mag, smag, keys, d, vmax, dtype, halves):
    """How far an output may be from the exact one.  A weight's relative error has three parts.
    (1) Its rounding to fp16, half a step of 2^-11, or 2^-22 in two halves, and, for weights
    below fp16's normal numbers, 2^-25 of a weight of 2^7 or more (the largest one's least size).
    (2) Its score: d products summed in fp32 in any order, d 2^-24 sum|q k|, 2^-22 for a query in two
    halves, and a few roundings more of the score; twice, as the denominator has it too.
    (3) exp2 and log2 of the hardware, the rescalings and the sums over the keys: n 2^-24, and
    2^-19 for some dozens of single roundings.  At last the output's own rounding: half a step of
    the value, and below the type's normal numbers half of their one step, smallest_normal * eps / 2
    (fp16 2^-25)."""
    p = 2.0 ** -22 if halves else 2.0 ** -11
    rel = p + 2 * smag[..., None] * ((d + 16) * 2.0 ** -24 + 2.0 ** -22) + 2 * keys[..., None] * 2.0 ** -24 + 2.0 ** -19
    tiny = 2 * vmax * keys[..., None] * 2.0 ** (-43 if halves else -32)
    info = torch.finfo(dtype)
    return mag * rel + tiny + np.abs(out) * info.eps / 2 + max(info.smallest_normal * info.eps / 2, 1e-40)


def lse_tolerance(lse, smag, keys, d):
    with np.errstate(invalid="ignore"):
        return (np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22 + smag * ((d + 16) * 2.0 ** -24 + 2.0 ** -22)
                + keys * 2.0 ** -24 + 2.0 ** -19)
