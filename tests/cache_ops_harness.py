"""Inputs and tolerances of the tests of art_append_kv, dense_extend and
dense_decode_shared.

Tolerances, elementwise, from the arithmetic (u = half a step of the type:
2^-8 for bf16, 2^-24 for fp32):
  append  the angle is rounded to 32 bits inside [-pi, pi] (pi 2^-24), sine and
          cosine are within 2 ulp (2^-23), the rotation has 3 roundings:
          (pi 2^-24 + 2^-23 + 3 2^-24) (|x| + |y|) scale < 8.2 2^-24 (...), then
          one rounding to the type, u |ref|.
  attend  one rounding of the output, u |ref|; for bf16 every weight p is rounded
          once for the matrix product, u sum(p |v|); fp32 sums of d products (scores,
          in the exponent: the error is multiplied by the score's own terms A) and
          of n weights, taken as random walks at 4 sigma:
          2^-24 (8 sqrt(d) A + 8 sqrt(n) + 16) max|v|, A = max sum|q k| / sqrt(d).
"""
import math

import numpy as np

import workloads as W

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
E24 = 2.0 ** -24


def rounded(x, dtype):
    """fp32 values exactly representable in the dtype."""
    x = np.asarray(x, np.float32)
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(x)) if dtype == "bf16" else x


class Pool:
    """A paged cache for the given lengths: pages in random order, NaN wherever no
    token is (unless poison is False), table entries that must not be read far out
    of range."""

    def __init__(self, rng, dtype, hkv, d, page, seq_lens, fill=True, poison=True, extra=3):
        self.dtype, self.page, self.d, self.hkv = dtype, page, d, hkv
        self.seq_lens = np.asarray(seq_lens, np.int32)
        need = [-(-int(n) // page) for n in seq_lens]
        cols = max(1, max(need)) + 1
        self.num_pages = sum(need) + extra
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(need), cols), -12345, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.num_pages, hkv, page, d)
        self.k = np.full(shape, np.nan if poison else 0.0, np.float32)
        self.v = self.k.copy()
        if fill:
            for b, n in enumerate(seq_lens):
                for t in range(int(n)):
                    self.put(b, t, rounded(rng.standard_normal((hkv, d)), dtype),
                             rounded(rng.standard_normal((hkv, d)), dtype))

    def put(self, b, t, k, v):
        pg = self.table[b, t // self.page]
        self.k[pg, :, t % self.page] = k
        self.v[pg, :, t % self.page] = v

    def shape(self, hq, **kw):
        return dict(dict(batch=len(self.seq_lens), num_q_heads=hq, num_kv_heads=self.hkv, head_dim=self.d,
                         page_size=self.page, block_size=64, max_pages_per_seq=self.table.shape[1], max_visit=1,
                         num_probe=1, num_pages_total=self.num_pages, dtype=0 if self.dtype == "bf16" else 1), **kw)


def attend_tol(ref, ref_abs, score_abs, n, d, vmax, dtype):
    """See the module's text; ref_abs: attention over |v|, score_abs: A."""
    tol = U[dtype] * np.abs(ref) + E24 * (8 * math.sqrt(d) * score_abs + 8 * math.sqrt(max(n, 1)) + 16) * vmax
    return tol + (U[dtype] * ref_abs if dtype == "bf16" else 0.0)
