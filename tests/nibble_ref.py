"""Plain restatement of the 4-bit cache in 64 bits (numpy / torch on the CPU): codec, storage
layout, tables and attention, from the definitions in include/dwkv.h.  Tests compare with it."""
from __future__ import annotations

import math

import numpy as np
import torch

S_MAX = 7680.0


# ------------------------------------------------------------------------------ codec
def scale_of(amax):
    """s: amax / 7 rounded to nearest even to 4 significant bits, at most 7680 (numpy fp64)."""
    y = np.asarray(amax, np.float64) / 7.0
    out = np.zeros_like(y)
    for i, v in np.ndenumerate(y):
        if v > 0:
            step = 2.0 ** (max(math.frexp(v)[1] - 1, -14) - 3)
            out[i] = min(np.rint(v / step) * step, S_MAX)
    return out


def scale_byte(s):
    return (np.asarray(s, np.float16).view(np.uint16) >> 7).astype(np.uint8)


def byte_scale(b):
    return (np.asarray(b, np.uint16) << 7).view(np.float16).astype(np.float64)


def quantise(x):
    """x fp64 [..][d] -> (codes int [..][d], scale bytes [..][d/16])."""
    x = np.where(np.isnan(x), 0.0, np.clip(x, -7 * S_MAX, 7 * S_MAX))
    g = x.reshape(*x.shape[:-1], -1, 16)
    s = scale_of(np.abs(g).max(-1))
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, np.clip(np.rint(g / s[..., None]), -7, 7), 0)
    return c.reshape(x.shape).astype(np.int64), scale_byte(s)


def values(codes, sbytes):
    return (codes.reshape(*codes.shape[:-1], -1, 16) * byte_scale(sbytes)[..., None]).reshape(codes.shape)


# ------------------------------------------------------------------------------ storage
def unit_of(c4):
    w = sum((int(c) + 8) << (4 * j) for j, c in enumerate(c4))
    return ((w << 2) | (w >> 14)) & 0xFFFF


def codes_of(unit):
    w = ((unit >> 2) | (unit << 14)) & 0xFFFF
    return [((w >> (4 * j)) & 15) - 8 for j in range(4)]


def block_offset(hkv, page_tokens, d, page, head, tok):
    per = page_tokens // 16
    return ((page * hkv + head) * per + tok // 16) * 18 * d


def put(pool, hkv, page_tokens, d, slot, head, z, codes, sbytes):
    """Store one vector (numpy uint8 pool)."""
    tok = slot % page_tokens
    base, t = block_offset(hkv, page_tokens, d, slot // page_tokens, head, tok), tok % 16
    for u in range(d // 4):
        w = unit_of(codes[4 * u:4 * u + 4])
        if z == 0:
            at = base + t * (d // 2) + 2 * u
        else:
            turn = (t >> 1) & 3 if d == 128 else (t >> 2) & 1
            at = base + 9 * d + t * (d // 2) + ((u // 8) ^ turn) * 16 + 2 * (u % 8)
        pool[at], pool[at + 1] = w & 255, w >> 8
    for g in range(d // 16):
        if z == 0:
            at = base + 8 * d + t * (d // 16) + g
        else:
            at = base + 17 * d + ((4 * (g & 1) + (t & 7) // 2) * (d // 32) + g // 2) * 4 + (t & 1) + 2 * (t // 8)
        pool[at] = sbytes[g]


_MAPS = {}


def _maps(d):
    """Byte offsets in a block: units [2][16][d/4] (low byte), scales [2][16][d/16]."""
    if d not in _MAPS:
        un, sc = np.zeros((2, 16, d // 4), int), np.zeros((2, 16, d // 16), int)
        for t in range(16):
            for u in range(d // 4):
                turn = (t >> 1) & 3 if d == 128 else (t >> 2) & 1
                un[0, t, u] = t * (d // 2) + 2 * u
                un[1, t, u] = 9 * d + t * (d // 2) + ((u // 8) ^ turn) * 16 + 2 * (u % 8)
            for g in range(d // 16):
                sc[0, t, g] = 8 * d + t * (d // 16) + g
                sc[1, t, g] = 17 * d + ((4 * (g & 1) + (t & 7) // 2) * (d // 32) + g // 2) * 4 + (t & 1) + 2 * (t // 8)
        _MAPS[d] = un, sc
    return _MAPS[d]


def get(pool, hkv, page_tokens, d, slots, head, z):
    """Values fp64 [n][d] of the given slots of one head (numpy uint8 pool)."""
    slots = np.asarray(slots, np.int64)
    un, sc = _maps(d)
    tok = slots % page_tokens
    base = ((slots // page_tokens * hkv + head) * (page_tokens // 16) + tok // 16) * 18 * d
    t = tok % 16
    at = base[:, None] + un[z][t]
    w = pool[at].astype(np.int64) | pool[at + 1].astype(np.int64) << 8
    w = ((w >> 2) | (w << 14)) & 0xFFFF
    c = np.stack([((w >> (4 * j)) & 15) - 8 for j in range(4)], -1).reshape(len(slots), d)
    return values(c, pool[base[:, None] + sc[z][t]])


# ------------------------------------------------------------------------------ tables
def tables(lens, new, release, table, free, count, page_tokens, max_rows):
    """One step of dwkv_nibble_tables on Python lists; returns the outputs as a dict."""
    n, p, width = len(lens), page_tokens, len(table[0]) if table else 0
    lens, table, free = list(lens), [list(r) for r in table], list(free)
    bad = [not 0 <= lens[b] <= width * p or new[b] < 0 for b in range(n)]
    for b in range(n):
        if release[b] and not bad[b]:
            for j in range(-(-lens[b] // p)):
                free[count] = table[b][j]
                count += 1
            lens[b] = 0
    cu, pos, slots = [0], [-1] * max_rows, [-1] * max_rows
    running, taken = 0, 0
    for b in range(n):
        m = 0 if bad[b] else new[b]
        cu.append(min(cu[-1] + m, 1 << 30))
        if bad[b]:
            continue
        if lens[b] + m > width * p:
            continue
        had = -(-lens[b] // p)
        need = -(-(lens[b] + m) // p) - had
        first, running = running, running + need
        if (need and running > count) or cu[-1] > max_rows:
            continue
        for j in range(need):
            table[b][had + j] = free[count - 1 - first - j]
        taken += need
        for j in range(m):
            pos[cu[b] + j] = lens[b] + j
            slots[cu[b] + j] = table[b][(lens[b] + j) // p] * p + (lens[b] + j) % p
        lens[b] += m
    return dict(seq_lens=lens, block_tables=table, free_list=free, free_count=[count - taken], cu_rows=cu,
                positions=pos, slots=slots)


# ------------------------------------------------------------------------------ attention
def attention(q, cu, lens, table, pool, hkv, page_tokens, window=0, scale=0.0):
    """q: torch [rows][Hq][d].  (o, lse, mag, span) in fp64: o and lse of the definition, mag the
    sum of weights times |v| per output, span the largest sum of |q_i k_i| scale of a row."""
    rows, hq, d = q.shape
    g = hq // hkv
    tau = scale if scale > 0 else 1.0 / math.sqrt(d)
    x = q.double().numpy()
    o, mag = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    lse, span = np.full((rows, hq), -np.inf), np.zeros((rows, hq))
    for b in range(len(lens)):
        a, m = cu[b], cu[b + 1] - cu[b]
        if m <= 0 or lens[b] == 0:
            continue
        t = np.arange(lens[b])
        slots = np.asarray(table[b], np.int64)[t // page_tokens] * page_tokens + t % page_tokens
        pos = lens[b] - m + np.arange(m)
        seen = t[None] <= pos[:, None]
        if window > 0:
            seen &= t[None] > pos[:, None] - window
        for h in range(hkv):
            k, v = (get(pool, hkv, page_tokens, d, slots, h, z) for z in (0, 1))
            k, v = (np.where(seen.any(0)[:, None], y, 0.0) for y in (k, v))
            for head in range(h * g, (h + 1) * g):
                s = tau * (x[a:a + m, head] @ k.T)
                ab = tau * (np.abs(x[a:a + m, head]) @ np.abs(k).T)
                s = np.where(seen, s, -np.inf)
                top = s.max(1, keepdims=True)
                top = np.where(np.isinf(top), 0.0, top)
                w = np.exp(s - top)
                tot = w.sum(1, keepdims=True)
                with np.errstate(divide="ignore"):
                    lse[a:a + m, head] = (top + np.log(tot))[:, 0]
                w = w / np.where(tot > 0, tot, 1.0)
                o[a:a + m, head] = w @ v
                mag[a:a + m, head] = w @ np.abs(v)
                span[a:a + m, head] = np.where(seen, ab, 0.0).max(1)
    return o, lse, mag, span


def tolerances(o, lse, mag, span, d, dtype):
    """Elementwise bounds of the kernels' outputs against attention().
    Scores: products of a 16-bit query with 8-bit-significand keys are exact; adding d of them in
    fp32, each addition off by at most 2^-23 of the running magnitude, errs by d 2^-23 span; a
    query below 2^-17 of its row's largest may lose its tail in fp16, another d 2^-25 span; scaling
    and exponential 2^-21 of the score's size and 2^-21 relative.  A relative error e of every
    weight moves o by at most 2 e mag (numerator and sum).  Weights are rounded to fp16 for the
    value product (half a step: 2^-11 mag, once), sums are fp32 (2^-20 mag allows for thousands of
    additions of either sign).  The output is rounded once: eps / 2 of itself, and at most half of the
    smallest subnormal of fp16 (2^-25)."""
    es = span * (d * 2.0 ** -23 + d * 2.0 ** -25 + 2.0 ** -21) + 2.0 ** -21
    half = torch.finfo(dtype).eps / 2
    to = mag * (2.0 ** -11 + 2.0 ** -20 + 2 * es[..., None]) + half * np.abs(o) * (1 + 2.0 ** -8) + 2.0 ** -25
    tl = es + 2.0 ** -20 + np.where(np.isfinite(lse), np.abs(lse), 0.0) * 2.0 ** -22
    return to, tl
