"""GPU tests of art_append_kv, dense_extend and dense_decode_shared against the
fp64 oracle (oracle/cache_ops.py), through the Python binding of the C ABI.

Pools are NaN wherever no token is, so a read of a masked or unwritten row that
reached a result would show. Tolerances: cache_ops_harness.py."""
import ctypes

import numpy as np
import pytest

from cache_ops_harness import E24, U, Pool, attend_tol, rounded
from oracle import cache_ops as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv_cache_early_gb300 as K  # noqa: E402

SENTINEL = 7.75  # exact in bf16


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def host(t):
    return t.double().cpu().numpy()


def workspace(nbytes):
    return torch.full((max(64, nbytes),), 0xA5, dtype=torch.uint8, device="cuda")  # nothing in it may be relied on


# ----------------------------------------------------------------------------
# art_append_kv
# ----------------------------------------------------------------------------
def append_case(seed, dtype, hq, hkv, d, page, new, ctx, rot, interleaved, fused=False, scale=1.0, positions=False,
                with_q=True, in_place=False, base=10000.0, pad=(0, 0), offsets=True):
    rng = np.random.default_rng(seed)
    new, ctx = np.asarray(new), np.asarray(ctx)
    pool = Pool(rng, dtype, hkv, d, page, new + ctx, fill=False, poison=False)
    pool.k[:] = rounded(rng.standard_normal(pool.k.shape), dtype)
    pool.v[:] = rounded(rng.standard_normal(pool.v.shape), dtype)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + pad[0]
    T = int(off[-1]) + pad[1]
    q, k, v = (rounded(rng.standard_normal((T, h, d)), dtype) for h in (hq, hkv, hkv))
    inv = (base ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    pos = rng.integers(0, 1 << 20, T).astype(np.int32) if positions else None
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.art_append_workspace_bytes(shape))
    kc, vc = dev(pool.k, dtype), dev(pool.v, dtype)
    if fused:
        row = dev(np.concatenate([q, k, v], 1), dtype)
        tq, tk, tv = row[:, :hq], row[:, hq:hq + hkv], row[:, hq + hkv:]
    else:
        tq, tk, tv = dev(q, dtype), dev(k, dtype), dev(v, dtype)
    q_out = tq if in_place else torch.full((T, hq, d), SENTINEL, dtype=kc.dtype, device="cuda")
    K.art_append_kv(tq if with_q else None, tk, tv, dev(pool.table), dev(pool.seq_lens), dev(off) if offsets else None,
                    dev(inv) if rot else None, q_out if with_q else None, kc, vc, shape, ws, rot_dim=rot,
                    interleaved=interleaved, scale=scale, positions=None if pos is None else dev(pos))
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    rq, rk, rv = O.append(q, k, v, off, pos, pool.table, pool.seq_lens, inv, rot, interleaved, scale, pool.k, pool.v,
                          pool.num_pages)
    # |x| + |y| of a pair is at most twice the larger; every value here is below 6.5 in magnitude
    slack = 8.2 * E24 * 13.0 * scale
    for got, ref, name in ((host(kc), rk, "k_cache"), (host(vc), rv, "v_cache")):
        assert np.all(np.abs(got - ref) <= slack + U[dtype] * np.abs(ref)), (name, np.abs(got - ref).max())
    assert np.array_equal(host(vc), rv)  # values are copied
    if with_q:
        got = host(q_out)
        held = ~np.isnan(rq).all(axis=(1, 2))
        assert np.all(np.abs(got - rq)[held] <= slack + U[dtype] * np.abs(rq[held]))
        keep = q if in_place else np.full_like(q, SENTINEL)
        assert np.array_equal(got[~held], keep[~held])  # rows of no sequence stay


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (14, 2, 64), (8, 8, 64), (8, 1, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_heads(dtype, hq, hkv, d, interleaved):
    append_case(1, dtype, hq, hkv, d, 16, [1, 5, 0, 33], [0, 15, 100, 1], d, interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot", [0, 2, 6, 8, 16, 30, 32, 48, 64, 126])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_partial_rotation(dtype, rot, interleaved):
    append_case(2, dtype, 4, 2, 128, 8, [3, 9], [7, 0], rot, interleaved, fused=True, scale=1.25)


@pytest.mark.parametrize("page", [8, 64, 4096])
@pytest.mark.parametrize("fused", [False, True])
def test_append_pages_and_strides(page, fused):
    append_case(3, "bf16", 4, 4, 64, page, [1, 70, 2], [page - 1, 63, 0], 64, False, fused=fused, pad=(2, 3))


def test_append_one_token_each():
    append_case(4, "bf16", 8, 2, 128, 16, [1] * 37, np.arange(37) * 3, 128, False, offsets=False)
    append_case(4, "f32", 8, 2, 128, 16, [1], [0], 128, False, offsets=False)


def test_append_many_sequences():
    """More sequences than a block has threads, some without new tokens."""
    new = np.array([(b * 7) % 3 for b in range(600)])
    append_case(5, "bf16", 1, 1, 64, 8, new, np.arange(600) % 11, 64, True)


def test_append_far_positions():
    append_case(6, "f32", 2, 2, 64, 16, [5, 1], [3, 2], 64, False, positions=True, base=500000.0)


def test_append_without_queries_and_in_place():
    append_case(7, "bf16", 8, 2, 64, 16, [4, 1], [3, 30], 64, False, with_q=False)
    append_case(8, "bf16", 8, 2, 64, 16, [4, 1], [3, 30], 64, False, in_place=True)
    append_case(8, "f32", 8, 2, 64, 16, [4, 1], [3, 30], 22, True, in_place=True)


def test_append_nothing():
    append_case(9, "bf16", 8, 2, 64, 16, [0, 0], [3, 0], 64, False)


def test_append_bad_device_data():
    rng = np.random.default_rng(10)
    dtype, hq, hkv, d, page = "bf16", 4, 2, 64, 16
    new, ctx = np.array([2, 3, 2, 20]), np.array([4, 0, 40, 10])
    pool = Pool(rng, dtype, hkv, d, page, new + ctx, fill=False, poison=False)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q, k, v = (rounded(rng.standard_normal((off[-1], h, d)), dtype) for h in (hq, hkv, hkv))
    lens = pool.seq_lens.copy()
    lens[0] = 1                                   # fewer than its new tokens
    lens[2] = pool.table.shape[1] * page + 1      # beyond the table
    pool.table[3, 1] = pool.num_pages             # second page of the last sequence
    inv = np.ones(d // 2, np.float32)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(64)
    kc, vc = dev(pool.k, dtype), dev(pool.v, dtype)
    q_out = torch.full((int(off[-1]), hq, d), SENTINEL, dtype=kc.dtype, device="cuda")
    args = (dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(pool.table), dev(lens))
    K.art_append_kv(*args, dev(off), dev(inv), q_out, kc, vc, shape, ws, rot_dim=d)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 4 | 8
    rq, rk, rv = O.append(q, k, v, off, None, pool.table, lens, inv, d, False, 1.0, pool.k, pool.v, pool.num_pages)
    assert np.all(np.abs(host(kc) - rk) <= 8.2 * E24 * 13 + U[dtype] * np.abs(rk))
    assert np.array_equal(host(vc), rv)
    assert np.all(np.abs(host(q_out) - rq) <= 8.2 * E24 * 13 + U[dtype] * np.abs(rq))
    # offsets that fall, or pass the tokens: flagged, nothing outside the tensors is touched
    for bad in ([0, 2, 1, 7, int(off[-1])], [0, 2, 5, 7, int(off[-1]) + 9], [-3, 2, 5, 7, int(off[-1])]):
        K.art_append_kv(*args, dev(np.array(bad, np.int32)), dev(inv), q_out, kc, vc, shape, ws, rot_dim=d)
        torch.cuda.synchronize()
        assert K.art_read_device_status(ws) & 128


@pytest.mark.parametrize("offsets", [[-3, 2, 5, 9], [0, 2, 5, 12]])
def test_append_skips_the_sequence_with_bad_offsets(offsets):
    """Only the sequence whose own two offsets lie outside 0 .. num_tokens appends nothing, its q_out rows stay."""
    rng = np.random.default_rng(12)
    dtype, hq, hkv, d, page = "bf16", 4, 2, 64, 16
    T, off = 9, np.array(offsets, np.int32)
    pool = Pool(rng, dtype, hkv, d, page, [20, 30, 40], fill=False, poison=False)
    q, k, v = (rounded(rng.standard_normal((T, h, d)), dtype) for h in (hq, hkv, hkv))
    inv = np.ones(d // 2, np.float32)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(64)
    kc, vc = dev(pool.k, dtype), dev(pool.v, dtype)
    q_out = torch.full((T, hq, d), SENTINEL, dtype=kc.dtype, device="cuda")
    K.art_append_kv(dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(pool.table), dev(pool.seq_lens), dev(off),
                    dev(inv), q_out, kc, vc, shape, ws, rot_dim=d)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 128
    wrong = 0 if offsets[0] < 0 else 2
    lo, hi = max(0, offsets[wrong]), min(T, offsets[wrong + 1])
    kept = [b for b in range(3) if b != wrong]
    rq, rk, rv = q * np.nan, pool.k, pool.v
    for b in kept:  # one sequence at a time: the oracle knows no bad offsets
        one, rk, rv = O.append(q, k, v, off[b:b + 2], None, pool.table[b:b + 1], pool.seq_lens[b:b + 1], inv, d, False,
                               1.0, rk, rv, pool.num_pages)
        rq[off[b]:off[b + 1]] = one[off[b]:off[b + 1]]
    assert np.all(np.abs(host(kc) - rk) <= 8.2 * E24 * 13 + U[dtype] * np.abs(rk))
    assert np.array_equal(host(vc), rv)
    got, held = host(q_out), np.r_[0:lo, hi:T]
    assert np.all(np.abs(got - rq)[held] <= 8.2 * E24 * 13 + U[dtype] * np.abs(rq[held]))
    assert np.all(got[lo:hi] == SENTINEL)


@pytest.mark.parametrize("dtype,rot,interleaved", [("bf16", 64, False), ("f32", 64, True), ("bf16", 22, False)])
def test_append_many_tokens(dtype, rot, interleaved):
    """Many tokens: two to a CTA, whose tokens belong to several sequences, to none, or to one."""
    new = [1, 2, 3, 0, 5, 700, 1, 1, 350, 13]
    append_case(11, dtype, 2, 1, 64, 16, new, np.arange(10) * 7, rot, interleaved, fused=True, pad=(3, 5))


# ----------------------------------------------------------------------------
# dense_extend
# ----------------------------------------------------------------------------
def attend_close(got, q, rows_of, dtype, skip_nan=True):
    """rows_of(t, h) -> (k, v) of the keys that row sees, in fp64, or None."""
    T, hq, d = q.shape
    for t in range(T):
        for h in range(hq):
            kv = rows_of(t, h)
            if kv is None:
                continue
            k, v = kv
            if len(k) == 0:
                assert np.all(got[t, h] == 0), (t, h)
                continue
            qd = q[t, h].astype(np.float64)
            ref = O.attend(qd, k, v)
            tol = attend_tol(ref, O.attend(qd, k, np.abs(v)), (np.abs(k) @ np.abs(qd)).max() / np.sqrt(d), len(k), d,
                             np.abs(v).max(), dtype)
            err = np.abs(got[t, h] - ref)
            assert np.all(err <= tol), (t, h, len(k), float((err / tol).max()), float(err.max()))


def extend_case(seed, dtype, hq, hkv, d, page, new, seq, causal, pad=(0, 0), q_scale=1.0, check_rows=None):
    rng = np.random.default_rng(seed)
    pool = Pool(rng, dtype, hkv, d, page, seq)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + pad[0]
    T = int(off[-1]) + pad[1]
    q = rounded(q_scale * rng.standard_normal((T, hq, d)), dtype)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.dense_extend_workspace_bytes(shape, T))
    tq = dev(q, dtype)
    out = torch.full_like(tq, SENTINEL)
    K.dense_extend(tq, dev(pool.k, dtype), dev(pool.v, dtype), dev(pool.table), dev(pool.seq_lens), dev(off), out,
                   shape, ws, causal=causal)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    got = host(out)
    held = np.zeros(T, bool)
    of = np.full(T, -1)
    cache = {}
    for b in range(len(seq)):
        held[off[b]:off[b + 1]] = True
        of[off[b]:off[b + 1]] = b

    def rows_of(t, h):
        b = of[t]
        if b < 0 or (check_rows is not None and not check_rows(t - off[b], h)):
            return None
        g = h // (hq // hkv)
        if (b, g) not in cache:
            cache[b, g] = [O.gather(c, pool.table[b], int(seq[b]), g) for c in (pool.k, pool.v)]
        n = seq[b] - (off[b + 1] - off[b]) + (t - off[b]) + 1 if causal else seq[b]
        return [c[:n] for c in cache[b, g]]

    attend_close(got, q, rows_of, dtype)
    assert np.all(got[~held] == SENTINEL)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (14, 2, 64), (4, 4, 64), (8, 1, 128), (7, 1, 128), (4, 2, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_extend_heads(dtype, hq, hkv, d, causal):
    extend_case(20, dtype, hq, hkv, d, 16, [5, 1, 0, 17], [5, 200, 40, 130], causal, pad=(1, 2))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257])
@pytest.mark.parametrize("causal", [True, False])
def test_extend_lengths(n, causal):
    extend_case(21, "bf16", 4, 1, 64, 8, [n, 1], [n, n], causal)
    extend_case(22, "bf16", 2, 1, 128, 32, [1, 3], [n + 3, 3], causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 16, 128, 256, 4096])
def test_extend_pages(dtype, page):
    extend_case(23, dtype, 4, 2, 64, page, [3, 40, 2], [300, 41, 129], True)


@pytest.mark.parametrize("rows", [16, 17, 128, 129, 256, 257, 600])
def test_extend_row_tiles(rows):
    """Rows of one KV head around the tiles' borders, keys enough for several CTAs."""
    check = lambda i, h: i < 4 or i % 61 == 0 or i > rows - 4
    extend_case(24, "bf16", 1, 1, 128, 16, [rows], [rows + 700], True, check_rows=check)
    extend_case(25, "bf16", 7, 1, 64, 16, [rows // 7 + 1, 2], [rows // 7 + 500, 900], False, check_rows=check)


def test_extend_long_context_split():
    """Few rows, many keys: one item over many CTAs."""
    extend_case(26, "bf16", 4, 1, 128, 16, [3], [9001], True)
    extend_case(27, "f32", 2, 2, 64, 64, [2], [5003], True)


def test_extend_encoder_longer_and_shorter():
    extend_case(28, "bf16", 4, 4, 64, 64, [50, 3, 4], [7, 300, 0], False)


def test_extend_no_tokens():
    extend_case(29, "bf16", 4, 2, 64, 16, [0, 0], [7, 0], True)
    extend_case(29, "bf16", 4, 2, 64, 16, [0, 0], [7, 0], True, pad=(0, 3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extend_large_scores(dtype):
    """Scores of several hundred: weights of zero and one, maxima that rise late."""
    extend_case(30, dtype, 4, 2, 128, 16, [33], [700], True, q_scale=16.0)


def steep(pool, up):
    """Keys along one direction whose scores with q = unit * 8 climb (or fall) by hundreds in steps of 37 keys."""
    d = pool.d
    u = np.zeros(d, np.float32)
    u[::2] = 1.0
    for b, n in enumerate(pool.seq_lens):
        for t in range(int(n)):
            pg, r = pool.table[b, t // pool.page], t % pool.page
            level = float((t if up else int(n) - 1 - t) // 37 - 6)
            pool.k[pg, :, r] = rounded(u * level + 0.0, pool.dtype)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 1, 128), ("bf16", 4, 2, 64), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("new", [3, 20, 70])
@pytest.mark.parametrize("up", [True, False])
def test_extend_maxima_that_move_far(dtype, hq, hkv, d, new, up):
    """A row's maximum climbs by hundreds of powers of two between and inside key tiles, or is met first and everything
    after it underflows; the rows of a tile do so in opposite directions (the sign of q)."""
    rng = np.random.default_rng(33)
    seq = [new + 400]
    pool = Pool(rng, dtype, hkv, d, 16, seq)
    steep(pool, up)
    q = np.zeros((new, hq, d), np.float32)
    q[..., ::2] = 8.0
    q[::2] *= -1.0
    q[:, ::3] *= 0.125
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.dense_extend_workspace_bytes(shape, new))
    out = torch.full((new, hq, d), SENTINEL, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    K.dense_extend(dev(q, dtype), dev(pool.k, dtype), dev(pool.v, dtype), dev(pool.table), dev(pool.seq_lens),
                   dev(np.array([0, new], np.int32)), out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    rows = {g: [O.gather(c, pool.table[0], seq[0], g) for c in (pool.k, pool.v)] for g in range(hkv)}
    attend_close(host(out), q, lambda t, h: [c[:401 + t] for c in rows[h // (hq // hkv)]], dtype)


def test_extend_nan_and_infinity_in_seen_keys():
    """A NaN key makes the rows that see it NaN, of its KV head only; a score of +infinity likewise; keys that
    no row sees change nothing."""
    rng = np.random.default_rng(34)
    for new in (3, 40):
        pool = Pool(rng, "bf16", 2, 64, 16, [new + 300])
        n = new + 300
        pool.k[pool.table[0, 50 // 16], 0, 50 % 16, 3] = np.nan          # head 0: seen by all
        last = n - 2                                                     # head 1: seen by the last two rows
        pool.k[pool.table[0, last // 16], 1, last % 16, 5] = np.inf
        q = rounded(1 + np.abs(rng.standard_normal((new, 4, 64))), "bf16")  # q > 0: the score is +infinity
        shape = K.make_shape(**pool.shape(4))
        ws = workspace(K.dense_extend_workspace_bytes(shape, new))
        out = torch.zeros((new, 4, 64), dtype=torch.bfloat16, device="cuda")
        K.dense_extend(dev(q, "bf16"), dev(pool.k, "bf16"), dev(pool.v, "bf16"), dev(pool.table), dev(pool.seq_lens),
                       dev(np.array([0, new], np.int32)), out, shape, ws)
        torch.cuda.synchronize()
        got = host(out)
        assert np.isnan(got[:, :2]).all()
        assert np.isnan(got[-2:, 2:]).all()
        k, v = (O.gather(c, pool.table[0], n, 1) for c in (pool.k, pool.v))
        attend_close(got[:-2, 2:], q[:-2, 2:], lambda t, h: (k[:301 + t], v[:301 + t]), "bf16")


def test_extend_many_sequences():
    """More sequences than the plan takes in one round, some without tokens or keys, split over all CTAs."""
    rng = np.random.default_rng(35)
    new = [(b * 5) % 4 for b in range(700)]
    seq = [n + (b * 13) % 40 for b, n in enumerate(new)]
    for causal in (True, False):
        extend_case(35, "bf16", 2, 1, 64, 8, new, seq, causal, check_rows=lambda i, h: h == 0)
    extend_case(36, "f32", 1, 1, 64, 8, new[:300], seq[:300], True)


def test_extend_wide_table():
    """A table whose longest possible sequences would pass 31-bit cost units: plain tile counts are used."""
    rng = np.random.default_rng(37)
    new, seq = [3] * 40, [200] * 40
    pool = Pool(rng, "bf16", 1, 64, 4096, seq)
    cols = 1 << 18
    table = torch.full((40, cols), -1, dtype=torch.int32, device="cuda")
    table[:, : pool.table.shape[1]] = dev(pool.table)
    q = rounded(rng.standard_normal((120, 2, 64)), "bf16")
    shape = K.make_shape(**pool.shape(2, max_pages_per_seq=cols))
    n = K.dense_extend_workspace_bytes(shape, 120)
    assert n > 0
    ws = workspace(n)
    out = torch.zeros((120, 2, 64), dtype=torch.bfloat16, device="cuda")
    K.dense_extend(dev(q, "bf16"), dev(pool.k, "bf16"), dev(pool.v, "bf16"), table, dev(pool.seq_lens),
                   dev(np.arange(0, 121, 3).astype(np.int32)), out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    rows = [[O.gather(c, pool.table[b], 200, 0) for c in (pool.k, pool.v)] for b in range(40)]
    attend_close(host(out), q, lambda t, h: [r[:198 + t % 3] for r in rows[t // 3]], "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_past_32_bit_offsets(dtype):
    """A pool of more than 2^32 elements, whose last pages the tokens lie in: append, extend and shared decode."""
    hq, hkv, d, page = 4, 2, 64, 64
    pages = (1 << 32) // (hkv * page * d) + 40
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    kc = torch.empty((pages, hkv, page, d), dtype=dt, device="cuda")
    vc = torch.empty_like(kc)
    rng = np.random.default_rng(38)
    n = 150
    table = np.array([[pages - 1, pages - 7, pages - 3], [pages - 1, pages - 5, pages - 2]], np.int32)
    k, v = (rounded(rng.standard_normal((2 * n, hkv, d)), dtype) for _ in range(2))
    q = rounded(rng.standard_normal((2 * n, hq, d)), dtype)
    k[n:n + page], v[n:n + page] = k[:page], v[:page]  # the first page is the same for both
    shape = K.make_shape(batch=2, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page, block_size=64,
                         max_pages_per_seq=3, max_visit=1, num_probe=1, num_pages_total=pages,
                         dtype=0 if dtype == "bf16" else 1)
    off, lens = dev(np.array([0, n, 2 * n], np.int32)), dev(np.array([n, n], np.int32))
    tq, tt = dev(q, dtype), dev(table)
    ws = workspace(max(K.dense_extend_workspace_bytes(shape, 2 * n), K.dense_decode_shared_workspace_bytes(shape, 1)))
    q_out = torch.empty_like(tq)
    K.art_append_kv(tq, dev(k, dtype), dev(v, dtype), tt, lens, off, None, q_out, kc, vc, shape, ws, rot_dim=0)
    out = torch.empty_like(tq)
    K.dense_extend(q_out, kc, vc, tt, lens, off, out, shape, ws)
    dec = torch.empty((2, hq, d), dtype=dt, device="cuda")
    ql = q_out[[n - 1, 2 * n - 1]].contiguous()
    K.dense_decode_shared(ql, kc, vc, tt, lens, dev(np.array([0, 2], np.int32)), dev(np.array([page], np.int32)), dec,
                          shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    k64, v64 = k.astype(np.float64), v.astype(np.float64)
    seen = lambda t, h: [x[t // n * n:t + 1, h // 2] for x in (k64, v64)]
    some = [0, 1, 63, 64, 149, 150, 213, 214, 299]
    attend_close(host(out)[some], q[some], lambda i, h: seen(some[i], h), dtype)
    attend_close(host(dec), q[[n - 1, 2 * n - 1]], lambda i, h: seen((i + 1) * n - 1, h), dtype)


def test_bounded_wait_expires_and_next_call_is_clean(monkeypatch):
    """The consumer warps wait for what nothing completes (test hook): the call ends with the timeout bit, the
    context stays usable and the next call on the same buffers is right."""
    rng = np.random.default_rng(39)
    for new, seq in ([40, 3], [300, 150]), ([2], [5000]):
        pool = Pool(rng, "bf16", 2, 128, 16, seq)
        T = sum(new)
        q = rounded(rng.standard_normal((T, 8, 128)), "bf16")
        shape = K.make_shape(**pool.shape(8))
        ws = workspace(K.dense_extend_workspace_bytes(shape, T))
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        args = (dev(q, "bf16"), dev(pool.k, "bf16"), dev(pool.v, "bf16"), dev(pool.table), dev(pool.seq_lens), dev(off),
                torch.zeros((T, 8, 128), dtype=torch.bfloat16, device="cuda"), shape, ws)
        monkeypatch.setenv("ART_TEST_STALL_NS", "200000")
        K.dense_extend(*args)
        torch.cuda.synchronize()
        assert K.art_read_device_status(ws) & 32
        monkeypatch.delenv("ART_TEST_STALL_NS")
        K.dense_extend(*args)
        torch.cuda.synchronize()
        assert K.art_read_device_status(ws) == 0
        ref = O.extend(q, pool.k, pool.v, pool.table, seq, off, True)
        assert np.abs(host(args[6]) - ref).max() <= 8 * U["bf16"]  # |out| < 4 here: output and weight roundings


def test_extend_bad_device_data():
    rng = np.random.default_rng(31)
    dtype, hq, hkv, d, page = "bf16", 4, 2, 64, 16
    new, seq = [3, 2, 4, 2], [40, 30, 100, 20]
    pool = Pool(rng, dtype, hkv, d, page, seq)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    lens = pool.seq_lens.copy()
    lens[0] = 2                                   # fewer than its new tokens
    lens[3] = -1
    good = pool.table.copy()
    pool.table[2, 6] = -1                         # the page of its last tokens
    q = rounded(rng.standard_normal((off[-1], hq, d)), dtype)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.dense_extend_workspace_bytes(shape, int(off[-1])))
    tq, kc, vc = dev(q, dtype), dev(pool.k, dtype), dev(pool.v, dtype)
    out = torch.full_like(tq, SENTINEL)
    K.dense_extend(tq, kc, vc, dev(pool.table), dev(lens), dev(off), out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 4 | 8
    got = host(out)
    ref = O.extend(q, pool.k, pool.v, good, lens, off, True, skip=(0, 2, 3))
    assert np.all(got[off[0]:off[1]] == 0) and np.all(got[off[2]:] == 0)
    assert np.abs(got - ref).max() <= 4 * U[dtype]  # |out| < 2 here: output and weight roundings
    for bad in ([0, 3, 2, 9, 11], [0, 3, 5, 9, 12], [-1, 3, 5, 9, 11]):
        out.fill_(SENTINEL)
        K.dense_extend(tq, kc, vc, dev(good), dev(pool.seq_lens), dev(np.array(bad, np.int32)), out, shape, ws)
        torch.cuda.synchronize()
        assert K.art_read_device_status(ws) & 128
        assert torch.all(out == SENTINEL)


# ----------------------------------------------------------------------------
# dense_decode_shared
# ----------------------------------------------------------------------------
def shared_case(seed, dtype, hq, hkv, d, page, groups, singles, q_scale=1.0, before=0, empty_group=False):
    """groups: [(prefix, [own tokens of each member])]; singles: lengths; before: that many of them first."""
    rng = np.random.default_rng(seed)
    seq, of = [int(n) for n in singles[:before]], [-1] * before
    off, pre = [before], []
    for j, (p, own) in enumerate(groups):
        for o in own:
            seq.append(max(0, p + o))  # own < 0: shorter than the prefix
            of.append(j)
        off.append(len(seq))
        pre.append(p)
        if empty_group and j == 0:
            off.append(len(seq))
            pre.append(50)
            of = [x + 1 if x > 0 else x for x in of]
    if empty_group:
        of = []
        for b in range(len(seq)):
            of.append(next((j for j in range(len(pre)) if off[j] <= b < off[j + 1]), -1))
    seq += [int(n) for n in singles[before:]]
    of += [-1] * (len(seq) - len(of))
    if not groups:
        off = [0]
    lead = [b if of[b] < 0 else off[of[b]] for b in range(len(seq))]
    need = list(seq)
    for b in range(len(seq)):
        if of[b] >= 0 and lead[b] == b:
            need[b] = max(need[b], pre[of[b]])  # the leader's row holds the whole prefix
    pool = Pool(rng, dtype, hkv, d, page, need)
    for b in range(len(seq)):  # a member's own row is not read below the page of its first own token
        if of[b] >= 0 and lead[b] != b:
            pool.table[b, :pre[of[b]] // page] = -777
            if seq[b] <= pre[of[b]]:
                pool.table[b] = -777
    pool.seq_lens = np.asarray(seq, np.int32)
    q = rounded(q_scale * rng.standard_normal((len(seq), hq, d)), dtype)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.dense_decode_shared_workspace_bytes(shape, len(pre)))
    tq = dev(q, dtype)
    out = torch.full_like(tq, SENTINEL)
    K.dense_decode_shared(tq, dev(pool.k, dtype), dev(pool.v, dtype), dev(pool.table), dev(pool.seq_lens),
                          dev(np.array(off, np.int32)) if pre else None,
                          dev(np.array(pre, np.int32)) if pre else None, out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    cache = {}

    def rows_of(b, h):
        g = h // (hq // hkv)
        p = min(seq[b], pre[of[b]]) if of[b] >= 0 else 0
        if (lead[b], g) not in cache:
            cache[lead[b], g] = [O.gather(c, pool.table[lead[b]], max(p, pre[of[b]] if of[b] >= 0 else 0), g)
                                 for c in (pool.k, pool.v)]
        out = []
        for c, shared in zip((pool.k, pool.v), cache[lead[b], g]):
            own = np.zeros((seq[b] - p, d))
            for t in range(p, seq[b]):
                own[t - p] = c[int(pool.table[b, t // page]), g, t % page]
            out.append(np.concatenate([shared[:p], own]))
        return out

    attend_close(host(out), q, rows_of, dtype)
    return pool, out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (14, 2, 64), (4, 4, 64), (8, 1, 128), (4, 2, 128)])
def test_shared_heads(dtype, hq, hkv, d):
    shared_case(40, dtype, hq, hkv, d, 16, [(200, [1, 30, 0, 129]), (33, [7])], [50, 0])


@pytest.mark.parametrize("prefix", [1, 7, 8, 16, 63, 64, 65, 127, 128, 129, 1001])
def test_shared_prefix_lengths(prefix):
    shared_case(41, "bf16", 4, 1, 64, 8, [(prefix, [0, 1, 5, 64])], [])
    shared_case(42, "bf16", 4, 2, 128, 16, [(prefix, [2, 128, 3])], [9])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 64, 256, 1024])
def test_shared_pages(dtype, page):
    shared_case(43, dtype, 4, 2, 64, page, [(page + 3, [1, 40, 700]), (2 * page, [5, 0])], [3])


@pytest.mark.parametrize("members", [1, 2, 4, 5, 31, 33, 64, 70])
def test_shared_members(members):
    """Rows of a prefix around the tiles' borders (G = 4)."""
    shared_case(44, "bf16", 4, 1, 128, 16, [(300, [1 + i % 19 for i in range(members)])], [])


def test_shared_short_and_empty_members():
    """Members shorter than the prefix, of length 0, a leader shorter than it, an empty group, sequences before
    and behind the groups, a prefix of length 0."""
    shared_case(45, "bf16", 8, 2, 64, 16, [(100, [-100, 3, -99, -1, -50, 20]), (0, [5, 0]), (40, [-40, 6])],
                [17, 0, 33, 129], before=2)
    shared_case(46, "f32", 8, 2, 64, 16, [(100, [4, 3]), (30, [1])], [17], empty_group=True)


def test_shared_long_prefix_split():
    shared_case(47, "bf16", 4, 1, 128, 16, [(9001, [1, 200])], [])
    shared_case(48, "f32", 2, 2, 64, 64, [(5003, [1, 20])], [])


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 4, 64), ("f32", 32, 8, 64), ("bf16", 28, 4, 128)])
def test_shared_many_rows(dtype, hq, hkv, d):
    """More rows than one wave of the merge kernel's blocks, of prefixes cut into many pieces and of short ones."""
    rng = np.random.default_rng(47)
    own = lambda n: [int(x) for x in rng.integers(1, 20, n)]
    shared_case(47, dtype, hq, hkv, d, 16, [(2500, own(90)), (33, own(40)), (0, own(2))], own(8))


def test_shared_many_sequences_and_groups():
    """More groups and sequences than the plan takes in one round."""
    groups = [(10 + j % 60, [1 + (j + i) % 5 for i in range(j % 4)]) for j in range(300)]
    shared_case(52, "bf16", 2, 1, 64, 8, groups, [1 + b % 30 for b in range(50)], before=20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_large_scores(dtype):
    shared_case(49, dtype, 8, 2, 128, 16, [(500, [100, 1, 30])], [], q_scale=16.0)


def test_shared_without_groups_is_dense_decode():
    pool, out = shared_case(50, "bf16", 8, 2, 128, 16, [], [1, 64, 300, 1000])
    rng = np.random.default_rng(50)
    # the same call through dense_decode: both round once at the end and round the weights to bf16 or finer
    pool2 = Pool(rng, "bf16", 2, 128, 16, [1, 64, 300, 1000])
    q = rounded(rng.standard_normal((4, 8, 128)), "bf16")
    shape = K.make_shape(**pool2.shape(8))
    ws = torch.zeros(K.art_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    ref = torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    K.dense_decode(dev(q, "bf16"), dev(np.nan_to_num(pool2.k), "bf16"), dev(np.nan_to_num(pool2.v), "bf16"),
                   dev(pool2.table), dev(pool2.seq_lens), None, ref, shape, ws)
    torch.cuda.synchronize()
    assert np.array_equal(pool2.table, pool.table)
    vmax = np.nanmax(np.abs(pool.v))
    assert np.abs(host(out) - host(ref)).max() <= 4 * U["bf16"] * vmax


def test_shared_bad_device_data():
    rng = np.random.default_rng(51)
    dtype, hq, hkv, d, page = "bf16", 4, 2, 64, 16
    seq = [70, 80, 90, 60, 61, 40]
    pool = Pool(rng, dtype, hkv, d, page, seq)
    off, pre = np.array([0, 3, 5], np.int32), np.array([50, 48], np.int32)
    good = pool.table.copy()
    q = rounded(rng.standard_normal((6, hq, d)), dtype)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.dense_decode_shared_workspace_bytes(shape, 2))
    tq, kc, vc = dev(q, dtype), dev(pool.k, dtype), dev(pool.v, dtype)

    def run(table, lens, off, pre):
        out = torch.full_like(tq, SENTINEL)
        K.dense_decode_shared(tq, kc, vc, dev(table), dev(np.asarray(lens, np.int32)), dev(np.asarray(off, np.int32)),
                              dev(np.asarray(pre, np.int32)), out, shape, ws)
        torch.cuda.synchronize()
        return host(out), K.art_read_device_status(ws)

    def expect(got, lens, pre, skip):
        ref = O.decode_shared(q, pool.k, pool.v, good, lens, off, pre, skip)
        assert np.abs(got - ref).max() <= 4 * U[dtype]  # |out| < 2 here

    got, st = run(good, seq, off, pre)
    assert st == 0
    expect(got, seq, pre, ())
    bad = good.copy()
    bad[0, 1] = pool.num_pages          # a page of the first group's prefix
    got, st = run(bad, seq, off, pre)
    assert st == 4
    expect(got, seq, pre, (0, 1, 2))
    bad = good.copy()
    bad[4, 3] = -1                      # a member's own page
    got, st = run(bad, seq, off, pre)
    assert st == 4
    expect(got, seq, pre, (4,))
    lens = list(seq)
    lens[1], lens[5] = -5, pool.table.shape[1] * page + 1
    got, st = run(good, lens, off, pre)
    assert st == 8
    expect(got, [max(0, n) if n < 1000 else n for n in lens], pre, (1, 5))
    got, st = run(good, seq, off, [50, -1])
    assert st == 8
    expect(got, seq, [50, 0], (3, 4))
    for bad in ([0, 3, 2], [0, 3, 7], [-1, 3, 5]):
        got, st = run(good, seq, bad, pre)
        assert st & 128 and np.all(got == SENTINEL)


# ----------------------------------------------------------------------------
# together, streams, graphs
# ----------------------------------------------------------------------------
class Chain:
    """Two prompts appended in chunks, attended, then sampled: append -> extend -> append -> shared decode, and the
    framework's own dense_decode over the same cache."""

    def __init__(self, seed, dtype="bf16"):
        rng = np.random.default_rng(seed)
        self.dtype, hq, hkv, d, page = dtype, 8, 2, 64, 16
        self.hq, self.hkv, self.d, self.page = hq, hkv, d, page
        self.prompt, self.samples = 83, 3  # one prompt, three samples of it
        B = self.samples
        cols = -(-(self.prompt + 1) // page)
        self.num_pages = cols + B + 2
        order = rng.permutation(self.num_pages)
        table = np.full((B, cols), -1, np.int32)
        whole = self.prompt // page
        table[0, :cols] = order[:cols]
        for b in range(1, B):
            table[b, :whole] = table[0, :whole]
            table[b, whole:] = order[cols + b]
        self.table = table
        self.pk = rounded(rng.standard_normal((self.prompt, hq + 2 * hkv, d)), dtype)
        self.sk = rounded(rng.standard_normal((B, hq + 2 * hkv, d)), dtype)
        self.inv = (10000.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.t = {n: dev(a) for n, a in dict(table=table, inv=self.inv, off1=np.array([0, self.prompt], np.int32),
                                             len1=np.array([self.prompt], np.int32),
                                             len2=np.full(B, self.prompt + 1, np.int32),
                                             goff=np.array([0, B], np.int32),
                                             pre=np.array([whole * page], np.int32)).items()}
        self.t.update(prow=dev(self.pk, dtype), srow=dev(self.sk, dtype))
        pool = (self.num_pages, hkv, page, d)
        for n in ("kc", "vc"):
            self.t[n] = torch.full(pool, float("nan"), dtype=dt, device="cuda")
        for n, rows in (("pq", self.prompt), ("po", self.prompt), ("sq", B), ("so", B), ("dd", B)):
            self.t[n] = torch.zeros((rows, hq, d), dtype=dt, device="cuda")
        base = dict(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page, block_size=64,
                    max_pages_per_seq=cols, max_visit=1, num_probe=1, num_pages_total=self.num_pages,
                    dtype=0 if dtype == "bf16" else 1)
        self.s1, self.sB = K.make_shape(batch=1, **base), K.make_shape(batch=B, **base)
        self.copies = dev(np.stack([table[1:, whole], np.full(B - 1, table[0, whole])]).astype(np.int64))
        z = lambda n: torch.zeros(max(64, n), dtype=torch.uint8, device="cuda")
        self.ws = [z(64), z(K.dense_extend_workspace_bytes(self.s1, self.prompt)), z(64),
                   z(K.dense_decode_shared_workspace_bytes(self.sB, 1)), z(K.art_workspace_bytes(self.sB))]

    def run(self, stream=None):
        t, hq, hkv = self.t, self.hq, self.hkv
        cut = lambda r: (r[:, :hq], r[:, hq:hq + hkv], r[:, hq + hkv:])
        table1 = t["table"][:1]
        K.art_append_kv(*cut(t["prow"]), table1, t["len1"], t["off1"], t["inv"], t["pq"], t["kc"], t["vc"], self.s1,
                        self.ws[0], rot_dim=self.d, stream=stream)
        K.dense_extend(t["pq"], t["kc"], t["vc"], table1, t["len1"], t["off1"], t["po"], self.s1, self.ws[1],
                       stream=stream)
        for c in ("kc", "vc"):  # the prompt's last, partly filled page is copied for the other samples
            t[c][self.copies[0]] = t[c][self.copies[1]]
        K.art_append_kv(*cut(t["srow"]), t["table"], t["len2"], None, t["inv"], t["sq"], t["kc"], t["vc"], self.sB,
                        self.ws[2], rot_dim=self.d, stream=stream)
        K.dense_decode_shared(t["sq"], t["kc"], t["vc"], t["table"], t["len2"], t["goff"], t["pre"], t["so"], self.sB,
                              self.ws[3], stream=stream)
        K.dense_decode(t["sq"], t["kc"], t["vc"], t["table"], t["len2"], None, t["dd"], self.sB, self.ws[4],
                       stream=stream)

    def check(self):
        for w in self.ws:
            assert K.art_read_device_status(w) == 0
        t, hq, hkv, d = self.t, self.hq, self.hkv, self.d
        nan = np.full((self.num_pages, hkv, self.page, d), np.nan)
        n = self.prompt
        pq, kc, vc = O.append(self.pk[:, :hq], self.pk[:, hq:hq + hkv], self.pk[:, hq + hkv:], [0, n], None,
                              self.table[:1], [n], self.inv, d, False, 1.0, nan, nan, self.num_pages)
        for got, ref in ((host(t["pq"]), pq),):
            assert np.all(np.abs(got - ref) <= 8.2 * E24 * 13 + U[self.dtype] * np.abs(ref))
        # what the kernels read from here on are the rounded values on the device
        pq, sq, kc, vc = (host(t[x]) for x in ("pq", "sq", "kc", "vc"))
        rows = {}
        for b in range(self.samples):
            for g in range(hkv):
                rows[b, g] = [O.gather(c, self.table[b], n + 1, g) for c in (kc, vc)]
        first = {}
        for g in range(hkv):
            first[g] = [r[:n] for r in rows[0, g]]
        attend_close(host(t["po"]), pq, lambda i, h: [r[:i + 1] for r in first[h // (hq // hkv)]], self.dtype)
        attend_close(host(t["so"]), sq, lambda b, h: rows[b, h // (hq // hkv)], self.dtype)
        attend_close(host(t["dd"]), sq, lambda b, h: rows[b, h // (hq // hkv)], self.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_extend_decode_together(dtype):
    c = Chain(60, dtype)
    c.run()
    torch.cuda.synchronize()
    c.check()


def test_two_streams_at_once():
    a, b = Chain(61), Chain(62)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for c, s in ((a, sa), (b, sb)):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_captured_and_replayed():
    c = Chain(63)
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for n in ("kc", "vc"):
        c.t[n].fill_(float("nan"))
    for n in ("pq", "po", "sq", "so", "dd"):
        c.t[n].fill_(SENTINEL)
    other = Chain(64)  # new contents for the same buffers
    for n in ("prow", "srow"):
        c.t[n].copy_(other.t[n])
    c.pk, c.sk = other.pk, other.sk
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    c.check()


def test_two_graphs_share_their_workspaces():
    """Graphs of the same program captured twice and replayed in turn on one stream."""
    c = Chain(67)
    c.run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for n in ("pq", "po", "sq", "so", "dd"):
        c.t[n].fill_(SENTINEL)
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    c.check()


def test_captured_behind_a_copy_of_another_stream():
    """The first kernel of a call follows a memory copy and an event of another stream, in a capture and outside."""
    c = Chain(68)
    c.run()
    torch.cuda.synchronize()
    rows = c.t["prow"].clone()
    side = torch.cuda.Stream()

    def joined():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.t["prow"].copy_(rows)
        K.dense_extend(c.t["pq"], c.t["kc"], c.t["vc"], c.t["table"][:1], c.t["len1"], c.t["off1"], c.t["po"], c.s1,
                       c.ws[1])
        torch.cuda.current_stream().wait_stream(side)
        c.run()
        c.t["po"].zero_()
        K.dense_extend(c.t["pq"], c.t["kc"], c.t["vc"], c.t["table"][:1], c.t["len1"], c.t["off1"], c.t["po"], c.s1,
                       c.ws[1])

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        joined()
    for run in (g.replay, joined, g.replay):
        c.t["prow"].fill_(float("nan"))
        for n in ("pq", "po", "sq", "so", "dd"):
            c.t[n].fill_(SENTINEL)
        run()
        torch.cuda.synchronize()
        c.check()


def test_repeated_calls_give_the_same_bits():
    c = Chain(65)
    c.run()
    torch.cuda.synchronize()
    first = [c.t[n].clone() for n in ("pq", "po", "sq", "so")]
    for _ in range(20):
        c.run()
    torch.cuda.synchronize()
    for n, f in zip(("pq", "po", "sq", "so"), first):
        assert torch.equal(c.t[n], f), n


def test_binding_refuses_what_the_pointers_would_hide():
    c = Chain(66)
    t = c.t
    args = [t["sq"], t["kc"], t["vc"], t["table"], t["len2"], t["goff"], t["pre"], t["so"], c.sB, c.ws[3]]
    K.dense_decode_shared(*args)
    for i, wrong in ((0, t["sq"].float()), (1, t["kc"][1:]), (3, t["table"].long()), (4, t["len2"].cpu()),
                     (7, t["so"].transpose(0, 1)), (5, t["pre"]), (9, c.ws[3].cpu())):
        bad = list(args)
        bad[i] = wrong
        with pytest.raises(K.ArtError):
            K.dense_decode_shared(*bad)
    with pytest.raises(K.ArtError):  # the new tokens' offsets are not optional here
        K.dense_extend(t["pq"], t["kc"], t["vc"], t["table"][:1], t["len1"], None, t["po"], c.s1, c.ws[1])
    row = t["srow"]
    with pytest.raises(K.ArtError):  # heads not side by side
        K.art_append_kv(row[:, 0:16:2], row[:, 8:10], row[:, 10:12], t["table"], t["len2"], None, t["inv"], t["sq"],
                        t["kc"], t["vc"], c.sB, c.ws[2], rot_dim=c.d)
    with pytest.raises(K.ArtError):  # too few frequencies
        K.art_append_kv(None, row[:, 8:10], row[:, 10:12], t["table"], t["len2"], None, t["inv"][:3], None, t["kc"],
                        t["vc"], c.sB, c.ws[2], rot_dim=c.d)
    torch.cuda.synchronize()
