"""CPU oracle of a paged cache held in 4 bits -- TEST INFRASTRUCTURE.

Only the test suite may import this module; the CUDA path never does, and the two share no
code. fp64 on the exact input values, and byte addresses formed one by one.
"""
from __future__ import annotations

import numpy as np

from oracle import cache_ops as O


def page_bytes(page, d, group):
    return page * (d + 8 * (d // group))


def nearest(x, bits):
    """x rounded to so many significant bits, ties to even."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def floor_bf16(x):
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.floor(np.ldexp(m, 8)), e - 8)


def bits16(x):
    """Numbers that are exact in bf16, as their 16 bits."""
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def from16(u):
    return (np.asarray(u, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x, group):
    """One head's row x [d]: codes [d], step and lowest [d / group]."""
    x = np.asarray(x, np.float64)
    codes, steps, lows = [], [], []
    for y in x.reshape(-1, group):
        if not np.all(np.isfinite(y)):
            codes.append(np.zeros(group, int)), steps.append(0.0), lows.append(np.nan)
            continue
        low = float(floor_bf16(y.min()))
        span = y.max() - low
        if not span < 15 * 2.0 ** 100:
            codes.append(np.zeros(group, int)), steps.append(0.0), lows.append(np.nan)
            continue
        step = float(nearest(span / 15.0, 8))
        if step < 2.0 ** -100:
            step = 0.0
        c = np.zeros(group, int) if step == 0 else np.minimum(np.rint((y - low) / step), 15).astype(int)
        codes.append(c), steps.append(step), lows.append(low)
    return np.concatenate(codes), np.array(steps), np.array(lows)


def addresses(page, d, group, place):
    """Byte offsets inside a head's page of a token: of its column's codes [2][d] (keys, values), and of its
    scales [2][d / group]."""
    n, slab = d // group, min(page, 64)
    base, u = place // slab * slab * (d + 8 * n), place % slab
    e, g = np.arange(d), np.arange(n)
    code = base + ((u // 8 * (d // 32) + e // 32) * 8 + u % 8) * 16 + e % 32 // 2
    scale = base + slab * d + ((u // 8 * n + g) * 8 + u % 8) * 4
    return (code, code + slab * d // 2), (scale, scale + 4 * slab * n)


def put(cache, page, d, group, pg, g, place, kv, x):
    """Quantises row x into a cache [pages, heads, bytes] of uint8."""
    code, step, low = quantise(x, group)
    at, sc = addresses(page, d, group, place)
    row = cache[pg, g]
    row[at[kv][0::2]] = (code[0::2] | code[1::2] << 4).astype(np.uint8)
    u = np.stack([bits16(step), bits16(low)], 1)
    u[np.isnan(low)] = (0, 0x7fc0)
    for k in range(4):
        row[sc[kv] + k] = (u[:, k // 2] >> (8 * (k % 2)) & 255).astype(np.uint8)


def get(cache, page, d, group, pg, g, place, kv):
    """codes [d], step and lowest by column [d], of a token."""
    at, sc = addresses(page, d, group, place)
    row = cache[pg, g]
    code = row[at[kv]] >> (4 * (np.arange(d) % 2)) & 15
    step = from16(row[sc[kv]] + 256 * row[sc[kv] + 1].astype(int))
    low = from16(row[sc[kv] + 2] + 256 * row[sc[kv] + 3].astype(int))
    return code.astype(np.float64), np.repeat(step, group), np.repeat(low, group)


def held(cache, row, n, g, page, d, group, kv):
    """The first n tokens behind a block-table row: codes, step, lowest [n][d]."""
    out = [get(cache, page, d, group, int(row[t // page]), g, t % page, kv) for t in range(n)]
    return tuple(np.array([o[i] for o in out]).reshape(n, d) for i in range(3))


def turned(x, pos, inv_freq, rot, interleaved, scale, dtype):
    return nearest(O.rotate(x, pos, inv_freq, rot, interleaved, scale), 8 if dtype == "bf16" else 24)


def append(k, v, offsets, positions, table, seq_lens, inv_freq, rot, interleaved, scale, cache, page, group, dtype):
    """The cache after the append."""
    cache = cache.copy()
    d = k.shape[2]
    for b in range(len(seq_lens)):
        lo, hi, n = int(offsets[b]), int(offsets[b + 1]), int(seq_lens[b])
        if n < hi - lo or n > table.shape[1] * page:
            continue
        for t in range(lo, hi):
            place = n - (hi - lo) + (t - lo)
            pos = place if positions is None else int(positions[t])
            pg = int(table[b, place // page])
            if not 0 <= pg < cache.shape[0]:
                continue
            for g in range(k.shape[1]):
                put(cache, page, d, group, pg, g, place % page, 0,
                    turned(k[t, g], pos, inv_freq, rot, interleaved, scale, dtype))
                put(cache, page, d, group, pg, g, place % page, 1, v[t, g])
    return cache


def extend(q, cache, table, seq_lens, offsets, causal, page, group, skip=()):
    """(out, terms): out as cache_ops.extend; terms [T, hq, 4]: for the tolerances, the largest sum of |q| (step
    code + |lowest|) / sqrt(d) over the keys, attention over step * code at its largest column, the largest step * 15 +
    |lowest| and the number of keys."""
    T, hq, d = q.shape
    hkv = cache.shape[1]
    out, terms = np.full(q.shape, np.nan), np.zeros((T, hq, 4))
    for b in range(len(seq_lens)):
        lo, hi, n = int(offsets[b]), int(offsets[b + 1]), int(seq_lens[b])
        if b in skip:
            out[lo:hi] = 0.0
            continue
        for g in range(hkv if hi > lo else 0):
            (kc, ks, kl), (vc, vs, vl) = (held(cache, table[b], n, g, page, d, group, kv) for kv in (0, 1))
            k, v = kl + ks * kc, vl + vs * vc
            for t in range(lo, hi):
                seen = max(0, n - (hi - lo) + (t - lo) + 1) if causal else n
                for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                    out[t, h] = O.attend(q[t, h], k[:seen], v[:seen])
                    if seen and np.all(np.isfinite(out[t, h])):
                        s = k[:seen] @ q[t, h] / np.sqrt(d)
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        terms[t, h] = ((ks * kc + np.abs(kl))[:seen] @ np.abs(q[t, h])).max() / np.sqrt(d), \
                            (p @ (vs * vc)[:seen]).max(), (15 * vs + np.abs(vl))[:seen].max(), seen
    return out, terms


def column_terms(q, cache, table, seq_lens, offsets, causal, page, group):
    """(out, score, mean, most, n): out as extend; score [T, hq] the largest sum of |q| (step 15 + |lowest|) / sqrt(d) over
    the keys; by column [T, hq, d], of the values seen: mean attention over their steps, largest 15 step + |lowest|; n [T]
    keys seen."""
    T, hq, d = q.shape
    out, score = np.full(q.shape, np.nan), np.zeros((T, hq))
    mean, most, n = np.zeros(q.shape), np.zeros(q.shape), np.zeros(T)
    per = hq // cache.shape[1]
    for b in range(len(seq_lens)):
        lo, hi, size = int(offsets[b]), int(offsets[b + 1]), int(seq_lens[b])
        for g in range(cache.shape[1] if hi > lo else 0):
            (kc, ks, kl), (vc, vs, vl) = (held(cache, table[b], size, g, page, d, group, kv) for kv in (0, 1))
            k, v = kl + ks * kc, vl + vs * vc
            for t in range(lo, hi):
                seen = max(0, size - (hi - lo) + (t - lo) + 1) if causal else size
                n[t] = seen
                for h in range(g * per, (g + 1) * per):
                    if seen == 0:
                        out[t, h] = 0.0
                        continue
                    s = k[:seen] @ q[t, h] / np.sqrt(d)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[t, h] = p @ v[:seen]
                    score[t, h] = ((15 * ks + np.abs(kl))[:seen] @ np.abs(q[t, h])).max() / np.sqrt(d)
                    mean[t, h] = p @ vs[:seen]
                    most[t, h] = (15 * vs + np.abs(vl))[:seen].max(0)
    return out, score, mean, most, n
