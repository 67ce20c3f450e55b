"""CPU oracle of writing the paged cache and of attention over it -- TEST
INFRASTRUCTURE.

Only the test suite may import this module; the CUDA path never does, and the
two share no code. Everything is fp64 on the exact input values (float arrays
holding bf16 or fp32 numbers), token by token and head by head.
"""
from __future__ import annotations

import math

import numpy as np


def rotate(x, pos, inv_freq, rot_dim, interleaved, scale=1.0):
    """One head's row x [d] turned to position pos."""
    y = np.array(x, np.float64)
    for j in range(rot_dim // 2):
        i, k = (2 * j, 2 * j + 1) if interleaved else (j, j + rot_dim // 2)
        c, s = math.cos(pos * float(inv_freq[j])), math.sin(pos * float(inv_freq[j]))
        a, b = float(x[i]), float(x[k])
        y[i], y[k] = scale * (a * c - b * s), scale * (b * c + a * s)
    return y


def append(q, k, v, offsets, positions, table, seq_lens, inv_freq, rot_dim, interleaved, scale, k_cache, v_cache,
           num_pages):
    """q_out, k_cache, v_cache (fp64 copies) after the append. Sequences with bad
    lengths append nothing and have zero queries; bad pages are skipped. Rows of
    q_out that no sequence holds are NaN here (never written)."""
    q_out = np.full(q.shape, np.nan)
    kc, vc = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    ps = kc.shape[2]
    for b in range(len(seq_lens)):
        lo, hi, n = int(offsets[b]), int(offsets[b + 1]), int(seq_lens[b])
        if n < hi - lo or n > table.shape[1] * ps:
            q_out[lo:hi] = 0.0
            continue
        for t in range(lo, hi):
            place = n - (hi - lo) + (t - lo)
            pos = place if positions is None else int(positions[t])
            for h in range(q.shape[1]):
                q_out[t, h] = rotate(q[t, h], pos, inv_freq, rot_dim, interleaved, scale)
            page = int(table[b, place // ps])
            if not 0 <= page < num_pages:
                continue
            for g in range(k.shape[1]):
                kc[page, g, place % ps] = rotate(k[t, g], pos, inv_freq, rot_dim, interleaved, scale)
                vc[page, g, place % ps] = v[t, g]
    return q_out, kc, vc


def gather(cache, row, n, g):
    """The first n cached rows of KV head g behind one block-table row: [n, d] fp64."""
    ps = cache.shape[2]
    out = np.zeros((n, cache.shape[3]))
    for t in range(n):
        out[t] = cache[int(row[t // ps]), g, t % ps]
    return out


def attend(q, k, v):
    """softmax(q k^T / sqrt(d)) v of one row; no keys: zero."""
    if len(k) == 0:
        return np.zeros(q.shape[-1])
    s = k @ np.asarray(q, np.float64) / math.sqrt(q.shape[-1])
    p = np.exp(s - s.max())
    return (p / p.sum()) @ v


def extend(q, k_cache, v_cache, table, seq_lens, offsets, causal, skip=()):
    """dense_extend; sequences in `skip` (bad ones) are zero, rows of no sequence NaN."""
    T, hq, d = q.shape
    hkv = k_cache.shape[1]
    out = np.full(q.shape, np.nan)
    for b in range(len(seq_lens)):
        lo, hi, n = int(offsets[b]), int(offsets[b + 1]), int(seq_lens[b])
        if b in skip:
            out[lo:hi] = 0.0
            continue
        for g in range(hkv if hi > lo else 0):
            k, v = gather(k_cache, table[b], n, g), gather(v_cache, table[b], n, g)
            for t in range(lo, hi):
                seen = n - (hi - lo) + (t - lo) + 1 if causal else n
                for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                    out[t, h] = attend(q[t, h], k[:seen], v[:seen])
    return out


def decode_shared(q, k_cache, v_cache, table, seq_lens, group_offsets, prefix_lens, skip=()):
    """dense_decode_shared; sequences in `skip` are zero."""
    B, hq, d = q.shape
    hkv, ps = k_cache.shape[1], k_cache.shape[2]
    out = np.zeros(q.shape)
    for b in range(B):
        if b in skip:
            continue
        n, lead, pre = int(seq_lens[b]), b, 0
        for j in range(len(prefix_lens)):
            if group_offsets[j] <= b < group_offsets[j + 1]:
                lead, pre = int(group_offsets[j]), int(prefix_lens[j])
        for g in range(hkv):
            rows = []
            for cache in (k_cache, v_cache):
                r = np.zeros((n, d))
                for t in range(n):
                    r[t] = cache[int(table[lead if t < pre else b, t // ps]), g, t % ps]
                rows.append(r)
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                out[b, h] = attend(q[b, h], rows[0], rows[1])
    return out
