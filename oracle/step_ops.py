"""fp64 / integer definitions of the serving-step operators -- TEST INFRASTRUCTURE ONLY.

Plain numpy, one sequence, block and token at a time: the 8-bit cache with a scale per
(block, kv head) (append, decode), the step plan and the packed causal attention.
bf16 data is carried as float64 arrays holding bf16 values; codes as float64 arrays
holding the numbers the codes stand for (e4m3 NaN as NaN).
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16
TOP = {"e4m3": 448.0, "int8": 127.0}
MIN_SCALE = 2.0 ** -64


def round_code(y, code):
    """The code value nearest to y (ties to even), saturated; NaN: e4m3 NaN, int8 0."""
    y = np.asarray(y, np.float64)
    top = TOP[code]
    c = np.clip(y, -top, top)
    if code == "int8":
        return np.where(np.isnan(y), 0.0, np.rint(c))
    with np.errstate(invalid="ignore"):
        mag = np.maximum(np.abs(c), 2.0 ** -6)
        step = 2.0 ** (np.floor(np.log2(np.where(np.isnan(mag), 1.0, mag))) - 3)
    return np.where(np.isnan(y), np.nan, np.rint(c / step) * step)


def need_scale(amax, code):
    """The smallest power of two s >= 2^-64 with amax <= s * top."""
    s = MIN_SCALE
    if amax <= s * TOP[code]:
        return s
    s = 2.0 ** (math.frexp(amax / TOP[code])[1] - 2)
    while amax > s * TOP[code]:
        s *= 2.0
    return s


def cache_write_scaled(x, slots, pool, scales, code):
    """Append x [T, H, d] at slots [T]: pool [NB, H, 16, d] (code values) and scales [NB, H]
    are changed in place."""
    nb, H = scales.shape
    by_block = {}
    for i, s in enumerate(np.asarray(slots).tolist()):
        if 0 <= s < nb * BLOCK:
            by_block.setdefault(s // BLOCK, []).append((s % BLOCK, i))
    for b, items in by_block.items():
        written = {o for o, _ in items}
        for h in range(H):
            rows = np.stack([x[i, h] for _, i in items])
            fin = np.abs(rows[np.isfinite(rows)])
            need = need_scale(float(fin.max()) if fin.size else 0.0, code)
            old = float(scales[b, h])
            sigma = need
            if 0 not in written and math.isfinite(old) and old > 0:
                sigma = max(old, need)
                if sigma > old:
                    for o in range(max(written)):
                        if o not in written:
                            pool[b, h, o] = round_code(pool[b, h, o] * old / sigma, code)
            for (o, _), r in zip(items, rows):
                pool[b, h, o] = round_code(r / sigma, code)
            scales[b, h] = sigma


def decode_scaled(q, kpool, vpool, kscales, vscales, tables, lens, scale):
    """Returns (out [S, Hq, d], bound [S, Hq, d]): the attention, and the sum of absolute
    contributions sum_t p_t |v_t| with the largest sum_i |q_i k_i| * scale of each row."""
    S, hq, d = q.shape
    g = hq // kpool.shape[1]
    out, mass, reach = np.zeros((S, hq, d)), np.zeros((S, hq, d)), np.zeros((S, hq, 1))
    for s in range(S):
        n = int(lens[s])
        if n <= 0:
            continue
        blocks = [int(b) for b in tables[s][:-(-n // BLOCK)]]
        for h in range(kpool.shape[1]):
            k = np.concatenate([kpool[b, h] * float(kscales[b, h]) for b in blocks])[:n]
            v = np.concatenate([vpool[b, h] * float(vscales[b, h]) for b in blocks])[:n]
            for j in range(h * g, (h + 1) * g):
                x = scale * (k @ q[s, j])
                p = np.exp(x - x.max())
                p /= p.sum()
                out[s, j], mass[s, j] = p @ v, p @ np.abs(v)
                reach[s, j] = abs(scale) * (np.abs(k) @ np.abs(q[s, j])).max()
    return out, mass, reach


def largest_weight(q, kpool, kscales, vscales, tables, lens, scale):
    """[S, Hq, 1]: the largest p_t * value scale over a row's tokens, p being the probabilities of
    decode_scaled -- what its 16-bit weights are relative to."""
    S, hq, _ = q.shape
    g = hq // kpool.shape[1]
    top = np.zeros((S, hq, 1))
    for s in range(S):
        n = int(lens[s])
        blocks = [int(b) for b in tables[s][:-(-n // BLOCK)]]
        for j in range(hq if n > 0 else 0):
            h = j // g
            k = np.concatenate([kpool[b, h] * float(kscales[b, h]) for b in blocks])[:n]
            x = scale * (k @ q[s, j])
            p = np.exp(x - x.max())
            top[s, j] = (p / p.sum() * np.repeat([float(vscales[b, h]) for b in blocks], BLOCK)[:n]).max()
    return top


def packed_attention(q, k, v, starts, scale):
    """Causal attention of every packed sequence; rows outside them are NaN."""
    T, hq, d = q.shape
    g = hq // k.shape[1]
    out, mass, reach = np.full((T, hq, d), np.nan), np.zeros((T, hq, d)), np.zeros((T, hq, 1))
    for a, b in zip(starts[:-1], starts[1:]):
        a, b = int(a), int(b)
        for h in range(hq):
            kk, vv, qq = k[a:b, h // g], v[a:b, h // g], q[a:b, h]
            x = scale * (qq @ kk.T)
            dead = np.triu(np.ones((b - a, b - a), bool), 1)
            x[dead] = -np.inf
            p = np.exp(x - x.max(1, keepdims=True, initial=-np.inf))
            p /= p.sum(1, keepdims=True)
            out[a:b, h], mass[a:b, h] = p @ vv, p @ np.abs(vv)
            reach[a:b, h] = abs(scale) * np.where(dead, 0.0, np.abs(qq) @ np.abs(kk).T).max(1, keepdims=True, initial=0)
    return out, mass, reach


def attention_bound(out, mass, reach, tokens):
    """How far a bf16 output may be from the fp64 one.

    out is rounded once to bf16: 2^-8 |out|.  Each probability is rounded to 16 bits (f16
    2^-11, bf16 2^-8: the caller's `tokens` tuple says which) in the numerator, so a row
    is off by at most that share of sum p |v|.  The scores are fp32 sums of d <= 128
    products in 8 chained tensor-core steps and at most 8 roundings after them: 16 * 2^-22
    of scale * sum |q k| in natural units, in the numerator and in the denominator; the
    exponential is off by 2^-21 more in both.  f16 probabilities below 2^-14 of the
    reference lose 2^-25 each, against a denominator of at least one.
    """
    n, half_step, vmax = tokens
    return (2.0 ** -8 * np.abs(out) + mass * (half_step + 2 * (16 * 2.0 ** -22 * reach + 2.0 ** -21)) * (1 + 2.0 ** -7)
            + n * 2.0 ** -25 * vmax + 1e-30)


def step_plan(counts, lens, tables, free, num_free, capacity):
    """(tables, slots, starts, lens, num_free) of one step, or None when it does not fit."""
    tables = np.array(tables, np.int32)
    slots, starts, new, height = [], [0], [], int(num_free)
    if not 0 <= height <= len(free):
        return None
    for s, (c, n) in enumerate(zip(counts.tolist(), lens.tolist())):
        if c < 0 or n < 0 or n + c > tables.shape[1] * BLOCK:
            return None
        for at in range(n, n + c):
            if at % BLOCK == 0:
                if height == 0:
                    return None
                height -= 1
                tables[s, at // BLOCK] = free[height]
            slots.append(int(tables[s, at // BLOCK]) * BLOCK + at % BLOCK)
        starts.append(len(slots))
        new.append(n + c)
    if len(slots) > capacity:
        return None
    return (tables, np.array(slots + [-1] * (capacity - len(slots)), np.int64), np.array(starts, np.int32),
            np.array(new, np.int32), height)
