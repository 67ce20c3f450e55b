"""Inputs and tolerances of the tests of art_append_kv4, art_read_kv4 and dense_extend_kv4.

What is written into the cache, and what is read back from it, is compared bit by bit (rotated keys:
the kernel's angles are within 1e-11, and a key whose exact value lies so near a rounding border is
met about once in 10^8).

Attention, elementwise, from the arithmetic (u = half a step of the type, 2^-8 for bf16 and 2^-24 for
fp32; A, C, V, n as in oracle.kv4.extend's terms):
  the output's own rounding        u |ref|
  weights times step               2^-12 C (bf16: once to fp16's 11 bits), 2^-23 C (fp32: two such parts);
                                   below 2^-14 of fp16's range a weight is off by 2^-25 at most, the
                                   largest being at least 2^4: n 2^-29 15 step < n 2^-29 V
  fp32 queries in two parts        2^-22 A in the exponent, on both sides of the quotient: 2 2^-22 A V
  bf16 products with keys' codes   a code is a denormal there, and a step of the product (16 columns and the sum so far)
                                   is cut at 2^-24 of the largest query times 2^-14, 2^-14 of that query in units of a
                                   code: 17 d / 16 such cuts, uniform, as random at 4 sigma (0.29 each), times the
                                   keys' largest step, on both sides of the quotient; only where queries have columns
                                   far larger than the others is this seen beside the terms above
  fp32 sums                        as for dense_extend: 2^-24 (8 sqrt(d) A + 8 sqrt(n) + 16) V
"""
import math

import numpy as np

from cache_ops_harness import E24, U, rounded
from oracle import kv4 as Q


class Pool4:
    """A cache of random bytes (codes, scales: whatever they mean) behind a block table; tokens are put by `fill`.
    Table entries that must not be read lie far out of range."""

    def __init__(self, rng, dtype, hkv, d, page, group, seq_lens, extra=3):
        self.dtype, self.page, self.d, self.hkv, self.group = dtype, page, d, hkv, group
        self.seq_lens = np.asarray(seq_lens, np.int32)
        need = [-(-int(n) // page) for n in seq_lens]
        self.num_pages = sum(need) + extra
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(need), max(1, max(need)) + 1), -12345, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.bytes = rng.integers(0, 256, (self.num_pages, hkv, Q.page_bytes(page, d, group))).astype(np.uint8)

    def fill(self, rng, scale=1.0, kscale=1.0):
        """Random tokens in every place below the lengths. scale, kscale: factors of a value's or a key's row, or
        functions of (sequence, token)."""
        for b, n in enumerate(self.seq_lens):
            for t in range(int(n)):
                for g in range(self.hkv):
                    for kv, s in ((0, kscale), (1, scale)):
                        f = s(b, t) if callable(s) else s
                        self.put(b, t, g, kv, rounded(rng.standard_normal(self.d) * f, self.dtype))
        return self

    def put(self, b, t, g, kv, x):
        Q.put(self.bytes, self.page, self.d, self.group, int(self.table[b, t // self.page]), g, t % self.page, kv, x)

    def shape(self, hq, **kw):
        return dict(dict(batch=len(self.seq_lens), num_q_heads=hq, num_kv_heads=self.hkv, head_dim=self.d,
                         page_size=self.page, block_size=64, max_pages_per_seq=self.table.shape[1], max_visit=1,
                         num_probe=1, num_pages_total=self.num_pages, dtype=0 if self.dtype == "bf16" else 1), **kw)


def cuts(top, step, v, d):
    """The tolerance's part for the cuts in the products with keys' codes (top: a query's largest column)."""
    return 2 * 4 * 0.29 * math.sqrt(17 * d / 16) * 2.0 ** -14 * top * step / math.sqrt(d) * v


def attend_tol(ref, terms, d, dtype):
    a, c, v, n = (terms[..., i][..., None] for i in range(4))
    tol = U[dtype] * np.abs(ref) + (2.0 ** -12 if dtype == "bf16" else 2.0 ** -23) * c + n * 2.0 ** -29 * v
    if dtype == "f32":
        tol = tol + 2.0 ** -21 * a * v
    return tol + E24 * (8 * math.sqrt(d) * a + 8 * np.sqrt(np.maximum(n, 1)) + 16) * v


def column_tol(terms, q, key_step, d, dtype):
    """By column, so that a group of small values is held to its own size. S: attention over the column's steps, V: the
    largest 15 step + |lowest| seen there, A: score's terms, n: keys (oracle.kv4.column_terms); key_step: the keys' largest.
      the output's own rounding         u |ref|
      weights times step, with codes less 8 (8 at most)
                                        8 S 2^-11 (bf16: fp16's rounding, 2^-11) or 8 S 2^-22 (fp32: two parts), and below
                                        2^-14 off by 2^-25 at most where the largest W is at least 2^4: 8 n 2^-29 S
      fp32 queries in two parts         2^-22 A in the exponent, on both sides of the quotient: 2 2^-22 A V
      bf16 products with keys' codes    `cuts`
      fp32 sums                         2^-24 (8 sqrt(d) A + 8 sqrt(n) + 16) V
    and 2^-120 where a step is so small that its weights reach beyond fp32's range."""
    ref, score, mean, most, n = terms
    a, n = score[..., None], n[:, None, None]
    tol = U[dtype] * np.abs(ref) + 8 * mean * ((2.0 ** -11 if dtype == "bf16" else 2.0 ** -22) + n * 2.0 ** -29) + 2.0 ** -120
    tol = tol + (cuts(np.abs(q).max(-1)[..., None], key_step, most, d) if dtype == "bf16" else 2.0 ** -21 * a * most)
    return tol + E24 * (8 * math.sqrt(d) * a + 8 * np.sqrt(np.maximum(n, 1)) + 16) * most
