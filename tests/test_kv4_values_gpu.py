"""GPU tests of dense_extend_kv4 over values of unequal and extreme sizes, against the fp64 oracle column by column
(kv4_harness.column_tol): flat groups, of step 0, of any size; groups of a head that differ."""
import numpy as np
import pytest

from cache_ops_harness import rounded
from kv4_harness import Pool4, column_tol
from oracle import kv4 as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv_cache_early_gb300 as K  # noqa: E402


def run(pool, q, off, causal, hq):
    shape = K.make_shape(**pool.shape(hq))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    tq = dev(q).to(torch.bfloat16 if pool.dtype == "bf16" else torch.float32)
    out = torch.full_like(tq, 7.75)
    ws = torch.full((K.dense_extend_kv4_min_workspace_bytes(shape, len(q), pool.group),), 0xA5, dtype=torch.uint8, device="cuda")
    K.dense_extend_kv4(tq, dev(pool.bytes), dev(pool.table), dev(pool.seq_lens), None if off is None else dev(off), out, shape,
                       ws, group=pool.group, causal=causal)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    return out.double().cpu().numpy()


def case(seed, dtype, d, group, lens, value, new=None, key=None, hq=4, page=16):
    """value, key: rows of (rng, sequence, token); new None: a decode step."""
    rng = np.random.default_rng(seed)
    pool = Pool4(rng, dtype, 1, d, page, group, lens)
    for b, n in enumerate(lens):
        for t in range(n):
            pool.put(b, t, 0, 0, rounded(rng.standard_normal(d) if key is None else key(rng, b, t), dtype))
            pool.put(b, t, 0, 1, rounded(np.broadcast_to(value(rng, b, t), d), dtype))
    off = np.concatenate([[0], np.cumsum([1] * len(lens) if new is None else new)]).astype(np.int32)
    q = rounded(rng.standard_normal((off[-1], hq, d)) if key is None else np.ones((off[-1], hq, d)), dtype)
    got = run(pool, q, None if new is None else off, new is not None, hq)
    terms = Q.column_terms(q, pool.bytes, pool.table, pool.seq_lens, off, new is not None, page, group)
    step = max(Q.held(pool.bytes, pool.table[b], n, 0, page, d, group, 0)[1].max() for b, n in enumerate(lens) if n)
    tol = column_tol(terms, q, step, d, dtype)
    err = np.abs(got - terms[0])
    assert np.all(err <= tol), (np.nanmax(err / tol), np.argwhere(~(err <= tol))[:4])


BOTH = pytest.mark.parametrize("dtype", ["bf16", "f32"])


def rising(by):
    """Keys whose scores against a query of ones rise by `by` (in log2) from token to token; flat, so that they are held
    exactly enough."""
    def key(rng, b, t):
        return np.full(64, by * t / 64 ** 0.5 / 1.4426950408889634)
    return key


@BOTH
@pytest.mark.parametrize("size", [2.0 ** 26, 2.0 ** 44, -2.0 ** 44, 2.0 ** 100, -2.0 ** 126])
def test_flat_rows_of_any_size(dtype, size):
    """Values of one number: attention over them is that number, however large."""
    case(1, dtype, 64, 32, [1, 40, 300], lambda rng, b, t: size)
    case(2, dtype, 64, 64, [700], lambda rng, b, t: size * (0.5 + (t % 2) / 2))
    case(3, dtype, 128, 32, [9, 150], lambda rng, b, t: size, new=[9, 5])
    case(4, dtype, 64, 32, [600], lambda rng, b, t: size, key=rising(0.1))
    case(5, dtype, 64, 32, [40], lambda rng, b, t: size, key=rising(14.0))


@BOTH
def test_flat_rows_beside_small_steps(dtype):
    """A large group without steps, beside one whose steps are very small, and rows of both kinds in turn."""
    half = np.arange(64) < 32
    case(6, dtype, 64, 32, [1, 200], lambda rng, b, t: np.where(half, 2.0 ** 60, rng.standard_normal(64) * 2.0 ** -80))
    case(7, dtype, 64, 32, [1, 200], lambda rng, b, t: np.where(half, 2.0 ** 100, rng.standard_normal(64) * 2.0 ** -92),
         new=[1, 4])
    case(8, dtype, 64, 32, [300], lambda rng, b, t: 2.0 ** 44 if t % 3 else rng.standard_normal(64))


def sized(ratio, d, group):
    """Sizes by column: groups 2^ratio apart around 1."""
    n = d // group
    return 2.0 ** (ratio * ((n - 1) / 2 - np.arange(d) // group))


@BOTH
@pytest.mark.parametrize("ratio", [8, 16, 24, 60])
def test_groups_of_unequal_size(dtype, ratio):
    """Every group of a head keeps its own bits."""
    for d, group, seed in ((64, 32, 20), (128, 64, 21), (128, 32, 22)):
        size = sized(ratio, d, group)
        case(seed, dtype, d, group, [1, 77, 200], lambda rng, b, t: rng.standard_normal(d) * size)
        case(seed + 10, dtype, d, group, [3, 150], lambda rng, b, t: rng.standard_normal(d) * size, new=[3, 5])


@BOTH
@pytest.mark.parametrize("ratio", [16, 40])
def test_groups_whose_sizes_change_from_token_to_token(dtype, ratio):
    """The large group is another one from token to token; and, once, far into the sequence."""
    def turns(rng, b, t):
        return rng.standard_normal(128) * np.where(np.arange(128) // 32 == t % 4, 2.0 ** ratio, 1.0)

    def once(rng, b, t):
        return rng.standard_normal(64) * np.where((np.arange(64) < 32) & (t == 130), 2.0 ** ratio, 1.0)
    case(40, dtype, 128, 32, [150], turns)
    case(41, dtype, 64, 32, [200, 131], once)
    case(42, dtype, 64, 32, [140], once, new=[15])  # rows that see it and rows that do not, in one item


@BOTH
def test_large_group_of_little_weight(dtype):
    """A token whose second group is large and whose weight is as much smaller: the others' bits stay in both groups."""
    def key(rng, b, t):
        return np.full(64, (-40.0 if t in (0, 70) else 0.02 * t) / 64 ** 0.5 / 1.4426950408889634)

    def value(rng, b, t):
        return rng.standard_normal(64) * np.where((np.arange(64) >= 32) & (t in (0, 70)), 2.0 ** 30, 1.0)
    # seen by its tolerance only where V is small: the first group's columns
    case(43, dtype, 64, 32, [100], value, key=key)
    case(44, dtype, 64, 32, [90], value, new=[4], key=key)


@BOTH
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 40, 2.0 ** 99])
@pytest.mark.parametrize("new", [None, 5])
def test_scores_far_below_zero(dtype, size, new):
    """Queries of up to 2^99 against keys whose every score is large and negative: the nearest key, or the mean of equal ones."""
    d, hq, page, group, n = 64, 4, 16, 32, 37
    rng = np.random.default_rng(60)
    pool = Pool4(rng, dtype, 1, d, page, group, [n, n])
    for b in range(2):
        for t in range(n):
            # flat keys, held exactly: all alike in the first sequence; in the second one nearer than the others from token 3 on
            pool.put(b, t, 0, 0, np.full(d, -4.0 if b == 0 else -2.0 if t == 3 else -4.0 - t))
            pool.put(b, t, 0, 1, rounded(rng.standard_normal(d), dtype))
    off = np.array([0, 1, 2] if new is None else [0, new, 2 * new], np.int32)
    got = run(pool, np.full((off[-1], hq, d), size), None if new is None else off, new is not None, hq)
    for b in range(2):
        _, step, low = Q.held(pool.bytes, pool.table[b], n, 0, page, d, group, 1)
        code = Q.held(pool.bytes, pool.table[b], n, 0, page, d, group, 1)[0]
        v = low + step * code
        for i in range(off[b + 1] - off[b]):
            seen = n if new is None else n - new + i + 1
            ref = v[:seen].mean(0) if b == 0 else v[3]
            s = step[:seen].mean(0) if b == 0 else step[3]
            # the output's rounding, weights' (equal: 2^-11 or 2^-22 of 8 steps) and fp32 sums of at most n values
            u, w = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -22)
            tol = u * np.abs(ref) + 8 * w * s + (8 * n ** 0.5 + 16) * 2.0 ** -24 * (15 * step + np.abs(low))[:seen].max(0)
            assert np.all(np.abs(got[off[b] + i] - ref) <= tol), (b, i, np.max(np.abs(got[off[b] + i] - ref) / tol))


@BOTH
def test_many_keys_of_the_largest_values(dtype):
    """160 sequences of 131,072 tokens whose values are one number near the type's largest; scores rise once, by 7.9 in log2,
    after each warp's first keys. All tokens lie in two pages, which every table row names again and again."""
    d, group, page, B, n = 64, 64, 64, 160, 1 << 17
    value = -1.5 * 2.0 ** 127
    pool = Pool4(np.random.default_rng(0), dtype, 1, d, page, group, [2 * page])
    high = rounded(np.full(1, 7.9 * 8 / 1.4426950408889634 / d), "bf16").item()
    for t in range(2 * page):
        pool.put(0, t, 0, 0, np.full(d, 0.0 if t < page else high))
        pool.put(0, t, 0, 1, np.full(d, value))
    first, rest = (int(x) for x in pool.table[0, :2])
    table = np.full((B, n // page), rest, np.int32)
    table[:, :24] = first
    pool.table, pool.seq_lens = table, np.full(B, n, np.int32)
    got = run(pool, np.ones((B, 4, d)), None, False, 4)
    # attention over one number: the output's rounding, and sums of n equal fp32 products as they grow
    assert np.all(np.abs(got / value - 1) <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24 * 8 * n ** 0.5)), got.ravel()[:4]
