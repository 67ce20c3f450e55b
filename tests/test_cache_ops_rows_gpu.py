"""GPU tests that the rows of a call do not disturb each other: rows whose scores
climb by hundreds of powers of two beside rows that see no key of a tile, that see
none at all, or whose queries are not numbers; and of refused shapes. fp64 oracle: oracle/cache_ops.py;
tolerances: cache_ops_harness.py."""
import numpy as np
import pytest

from cache_ops_harness import E24, U, Pool, attend_tol, rounded
from oracle import cache_ops as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv_cache_early_gb300 as K  # noqa: E402
from test_cache_ops_gpu import SENTINEL, Chain, attend_close, dev, host, workspace  # noqa: E402


def climbing_pool(rng, dtype, hkv, d, lens, first, up):
    """A pool whose sequence b holds tokens first[b] .. lens[b] - 1 (elsewhere NaN). The keys lie along one direction:
    their scores with signed_queries climb (or fall) by hundreds of powers of two in steps of 37 keys, over and over,
    so that a segment of several key tiles meets a rise wherever it starts."""
    pool = Pool(rng, dtype, hkv, d, 16, lens, fill=False)
    u = np.zeros(d, np.float32)
    u[::2] = 1.0
    for b, n in enumerate(lens):
        t = np.arange(first[b], n)
        at = pool.table[b, t // 16], slice(None), t % 16
        level = (t if up else n - 1 - t) // 37 % 12 - 6
        pool.k[at] = (level[:, None] * u)[:, None]
        pool.v[at] = rounded(rng.standard_normal((len(t), hkv, d)), dtype)
    return pool


def signed_queries(n, hq, d):
    """Queries along the direction of climbing_pool's keys: rising and falling scores, of several sizes."""
    q = np.zeros((n, hq, d), np.float32)
    q[..., ::2] = 8.0
    q[1::2] *= -1.0
    q[:, ::3] *= 0.125
    return q


def shared_climb(dtype, hq, hkv, d, prefix, lens, up, heads, nan_rows=()):
    """One group behind a prefix whose scores climb; lens: whole lengths of its members (the first leads); heads:
    the query heads that are checked; nan_rows: (member, head) of queries that are NaN."""
    rng = np.random.default_rng(70)
    pool = climbing_pool(rng, dtype, hkv, d, [max(lens[0], prefix)] + lens[1:], [0] + [prefix] * (len(lens) - 1), up)
    pool.seq_lens = np.asarray(lens, np.int32)
    for b in range(1, len(lens)):
        pool.table[b, :prefix // 16] = -777  # read through the leader's row
        if lens[b] <= prefix:
            pool.table[b] = -777
    q = signed_queries(len(lens), hq, d)
    for b, h in nan_rows:
        q[b, h] = np.nan
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.dense_decode_shared_workspace_bytes(shape, 1))
    tq = dev(q, dtype)
    out = torch.full_like(tq, SENTINEL)
    K.dense_decode_shared(tq, dev(pool.k, dtype), dev(pool.v, dtype), dev(pool.table), dev(pool.seq_lens),
                          dev(np.array([0, len(lens)], np.int32)), dev(np.array([prefix], np.int32)), out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    got = host(out)
    lead = {g: [O.gather(c, pool.table[0], max(lens[0], prefix), g) for c in (pool.k, pool.v)]
            for g in {h // (hq // hkv) for h in heads}}

    def rows_of(b, h):
        if (b, h) in nan_rows or h not in heads:
            return None
        g, p, rows = h // (hq // hkv), min(prefix, lens[b]), []
        for c, shared in zip((pool.k, pool.v), lead[g]):
            own = [c[pool.table[b, t // 16], g, t % 16] for t in range(p, lens[b])]
            rows.append(np.concatenate([shared[:p], np.reshape(own, (-1, d)).astype(np.float64)]))
        return rows

    attend_close(got, q, rows_of, dtype)
    for b, h in nan_rows:  # no key seen: zero, whatever the query holds
        assert np.isnan(got[b, h]).all() if lens[b] > 0 else np.all(got[b, h] == 0), (b, h)


# Enough keys and KV heads that a CTA's share of the prefix is several key tiles.
LONG = 6000


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("bf16", 16, 8, 64), ("bf16", 28, 4, 128), ("f32", 16, 4, 64)])
@pytest.mark.parametrize("members", [6, 30, 70])
def test_shared_short_member_beside_climbing_scores(dtype, hq, hkv, d, members):
    """A member that sees the first 40 keys of the prefix (nothing of a tile's second half) among members whose
    scores climb over all of it: rows of one tile, and of more."""
    lens = [LONG + 1 + 3 * i % 50 for i in range(members)]
    lens[2] = 40
    lens[members - 1] = 1
    shared_climb(dtype, hq, hkv, d, LONG, lens, members != 30, (0, 1, hq - 1))


@pytest.mark.parametrize("members", [3, 6, 30, 70])
@pytest.mark.parametrize("length", [0, LONG + 30])
def test_shared_nan_query_beside_climbing_scores(members, length):
    """A query that is NaN, of a padded member without keys and of one with keys."""
    lens = [LONG + 1 + 3 * i % 50 for i in range(members)]
    lens[1] = length
    shared_climb("bf16", 32, 8, 128, LONG, lens, True, (0, 1, 30, 31),
                 nan_rows=[(1, h) for h in range(0, 32, 3)])


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 4, 128), ("bf16", 8, 4, 64), ("f32", 8, 4, 64)])
@pytest.mark.parametrize("new", [3, 20, 70])
@pytest.mark.parametrize("up", [True, False])
def test_extend_nan_query_beside_climbing_scores(dtype, hq, hkv, d, new, up):
    rng = np.random.default_rng(71)
    n = new + LONG
    pool = climbing_pool(rng, dtype, hkv, d, [n], [0], up)
    q = signed_queries(new, hq, d)
    bad = [(t, h) for t in (1, new // 2, new - 1) for h in range(t % 2, hq, 3)]
    for t, h in bad:
        q[t, h] = np.nan
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.dense_extend_workspace_bytes(shape, new))
    tq = dev(q, dtype)
    out = torch.full_like(tq, SENTINEL)
    K.dense_extend(tq, dev(pool.k, dtype), dev(pool.v, dtype), dev(pool.table), dev(pool.seq_lens),
                   dev(np.array([0, new], np.int32)), out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    got = host(out)
    group, heads = hq // hkv, (0, 1, hq - 2, hq - 1)
    rows = {g: [O.gather(c, pool.table[0], n, g) for c in (pool.k, pool.v)] for g in {h // group for h in heads}}
    attend_close(got, q, lambda t, h: [c[:LONG + 1 + t] for c in rows[h // group]]
                 if h in heads and (t, h) not in bad else None, dtype)
    for t, h in bad:
        assert np.isnan(got[t, h]).all(), (t, h)


@pytest.mark.parametrize("new,hq,hkv,d", [(5, 32, 8, 128), (32, 8, 2, 64), (16, 8, 1, 128)])
def test_one_row_tile_joins_both_halves_every_time(new, hq, hkv, d):
    """17 to 128 rows: the two halves of every key tile are summed apart and each is read by the warps of both.
    Many calls of many items (whole ones and cut ones), the same bits every time, and right."""
    rng = np.random.default_rng(72)
    seq = [200 + 64 * (b % 5) + 37 * b for b in range(24)]
    pool = Pool(rng, "bf16", hkv, d, 16, seq)
    off = np.arange(len(seq) + 1, dtype=np.int32) * new
    q = rounded(rng.standard_normal((int(off[-1]), hq, d)), "bf16")
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.dense_extend_workspace_bytes(shape, int(off[-1])))
    tq = dev(q, "bf16")
    args = dev(pool.k, "bf16"), dev(pool.v, "bf16"), dev(pool.table), dev(pool.seq_lens), dev(off)
    outs = torch.full((40,) + tuple(tq.shape), SENTINEL, dtype=tq.dtype, device="cuda")
    for o in outs:
        K.dense_extend(tq, *args, o, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    assert bool((outs == outs[:1]).all())
    got, heads = host(outs[0]), (0, hq - 1)
    rows = {(b, g): [O.gather(c, pool.table[b], seq[b], g) for c in (pool.k, pool.v)]
            for b in range(0, len(seq), 5) for g in {h // (hq // hkv) for h in heads}}
    attend_close(got, q, lambda t, h: [c[:seq[t // new] - new + t % new + 1] for c in rows[t // new, h // (hq // hkv)]]
                 if h in heads and t // new % 5 == 0 else None, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot", [64, 22])
@pytest.mark.parametrize("new", [[1, 2, 0, 3], [301, 1, 499]])
def test_append_rows_of_no_sequence_may_hold_anything(dtype, rot, new):
    """A batch padded in front and behind with rows that are no numbers: nothing of them is kept, their rows of
    q_out stay as they were. (Vector and scalar form; one token a CTA and two.)"""
    rng = np.random.default_rng(73)
    hq, hkv, d, page = 4, 2, 64, 16
    pool = Pool(rng, dtype, hkv, d, page, [n + 7 for n in new], fill=False)
    off = (np.concatenate([[0], np.cumsum(new)]) + 5).astype(np.int32)
    T = int(off[-1]) + 3
    q, k, v = (rounded(rng.standard_normal((T, h, d)), dtype) for h in (hq, hkv, hkv))
    for x in (q, k, v):
        x[:5], x[off[-1]:] = np.nan, np.inf
    inv = (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.art_append_workspace_bytes(shape))
    kc, vc = dev(pool.k, dtype), dev(pool.v, dtype)
    q_out = torch.full((T, hq, d), SENTINEL, dtype=kc.dtype, device="cuda")
    K.art_append_kv(dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(pool.table), dev(pool.seq_lens), dev(off),
                    dev(inv), q_out, kc, vc, shape, ws, rot_dim=rot)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    rq, rk, rv = O.append(q, k, v, off, None, pool.table, pool.seq_lens, inv, rot, False, 1.0, pool.k, pool.v,
                          pool.num_pages)
    for got, ref in ((host(kc), rk), (host(vc), rv), (host(q_out)[5:off[-1]], rq[5:off[-1]])):
        held = ~np.isnan(ref)
        assert np.array_equal(np.isnan(got), ~held)
        assert np.all(np.abs(got - ref)[held] <= 8.2 * E24 * 13 + U[dtype] * np.abs(ref[held]))
    assert np.all(host(q_out)[:5] == SENTINEL) and np.all(host(q_out)[off[-1]:] == SENTINEL)


def test_append_angles_of_both_reductions():
    """Positions and products on both sides of 2^24, negative ones too, fp32 results: beyond 2^24 the 64-bit
    product, the turns and 2 pi are each off by 2^-53 of 2^27 at most, 3 2^-26 radians in all."""
    rng = np.random.default_rng(74)
    d, T = 64, 24
    pos = np.array([0, 1, -1, 5, -4097, 99991, (1 << 20) + 1, -(1 << 20) - 3, (1 << 22) - 1, 3 - (1 << 22), 1 << 23,
                    8388607, (1 << 24) - 1, 1 - (1 << 24), 1 << 24, -(1 << 24), (1 << 24) + 1, (1 << 24) + 7,
                    -(1 << 24) - 5, 11863283, 2670176, 2670177, 3, 4], np.int32)
    inv = (10000.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)
    inv[1], inv[2], inv[3] = 0.0, 1.0, np.float32(2.0 * np.pi)  # 2 pi: whole turns, products past 2^24 below pos 2^24
    pool = Pool(rng, "f32", 1, d, 16, [T], fill=False)
    k, v = (rounded(rng.standard_normal((T, 1, d)), "f32") for _ in range(2))
    shape = K.make_shape(**pool.shape(1))
    ws = workspace(K.art_append_workspace_bytes(shape))
    kc, vc = dev(pool.k, "f32"), dev(pool.v, "f32")
    K.art_append_kv(None, dev(k, "f32"), dev(v, "f32"), dev(pool.table), dev(pool.seq_lens),
                    dev(np.array([0, T], np.int32)), dev(inv), None, kc, vc, shape, ws, rot_dim=d, positions=dev(pos))
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    _, rk, _ = O.append(np.zeros((T, 1, d)), k, v, [0, T], pos, pool.table, [T], inv, d, False, 1.0, pool.k, pool.v,
                        pool.num_pages)
    got, held = host(kc), ~np.isnan(rk)
    tol = (8.2 * E24 + 3 * 2.0 ** -26) * 2 * np.abs(k).max() + U["f32"] * np.abs(rk[held])
    assert np.all(np.abs(got[held] - rk[held]) <= tol), np.abs(got[held] - rk[held]).max()


def test_binding_refuses_as_many_elements_in_another_order():
    """A tensor with the right number of elements and another shape is other data: [pages, page_size, heads, d]
    caches, transposed tables, heads behind columns, flat rows."""
    c = Chain(75)
    t, row, hq, hkv, d = c.t, c.t["srow"], c.hq, c.hkv, c.d
    z = lambda *n: torch.zeros(*n, dtype=torch.bfloat16, device="cuda")
    swapped = z(c.num_pages, c.page, hkv, d)
    table = t["table"].t().contiguous()
    shared = [t["sq"], t["kc"], t["vc"], t["table"], t["len2"], t["goff"], t["pre"], t["so"], c.sB, c.ws[3]]
    extend = [t["pq"], t["kc"], t["vc"], t["table"][:1], t["len1"], t["off1"], t["po"], c.s1, c.ws[1]]
    append = [row[:, :hq], row[:, hq:hq + hkv], row[:, hq + hkv:], t["table"], t["len2"], None, t["inv"], t["sq"],
              t["kc"], t["vc"], c.sB, c.ws[2]]
    for call, good, wrongs in (
            (K.dense_decode_shared, shared, [(0, z(3, d, hq)), (0, z(3, hq * d)), (1, swapped), (2, swapped), (3, table),
                                             (4, t["len2"][:, None]), (5, t["goff"][None]), (6, t["pre"][:, None]),
                                             (7, z(3, d, hq))]),
            (K.dense_extend, extend, [(0, z(c.prompt, d, hq)), (1, swapped), (2, swapped), (3, table[:, :1]),
                                      (5, t["off1"][None]), (6, z(c.prompt, hq * d))]),
            (lambda *a: K.art_append_kv(*a, rot_dim=d), append,
             [(3, table), (4, t["len2"][None]), (6, t["inv"][None]), (7, z(3, d, hq)), (8, swapped), (9, swapped)])):
        call(*good)
        for i, wrong in wrongs:
            assert wrong.numel() == good[i].numel()
            bad = list(good)
            bad[i] = wrong
            with pytest.raises(K.ArtError):
                call(*bad)
    torch.cuda.synchronize()


def test_weights_are_rounded_once():
    """bf16, more than 128 rows: the maximum of the second half of a key tile moves the reference of weights that are
    rounded already. Their scaling must not round them again. Weights against an integer reference (in log2) have the
    same bits whatever it is, so the oracle rounds its own: out = bf16(p_a2) v / (p_a1 + p_a2 + p_b), to the output's
    rounding and the fp32 scores' 2^-15. Rows whose p_a2 lies within 2^-13 of a tie are left out."""
    rng = np.random.default_rng(76)
    d, rows, n, a1, a2, b = 64, 160, 128, 5, 40, 100
    pool = Pool(rng, "bf16", 1, d, 16, [n], fill=False)
    k, v = np.zeros((n, d), np.float32), np.zeros((n, d), np.float32)
    k[:, 0] = -4.0  # weights below 2^-60 of the others
    k[a1, 0], k[a2, 0], k[b, 0] = 1.0, 1.0, 2.0
    k[a2, 1:8] = rounded(rng.standard_normal(7), "bf16")
    v[a2] = 2.0 ** 17 * rounded(1.0 + rng.random(d), "bf16")
    at = pool.table[0, np.arange(n) // 16], 0, np.arange(n) % 16
    pool.k[at], pool.v[at] = k, v
    q = np.zeros((rows, 1, d), np.float32)
    q[:, 0, 0] = 100.0 + rng.integers(0, 32, rows)  # b leads a1 by 18 to 24 powers of two
    q[:, 0, 1:8] = rounded(rng.standard_normal((rows, 7)) - 1.5 * np.sign(k[a2, 1:8]), "bf16")  # a2 stays below a1
    shape = K.make_shape(**pool.shape(1))
    ws = workspace(K.dense_extend_workspace_bytes(shape, rows))
    tq = dev(q, "bf16")
    out = torch.full_like(tq, SENTINEL)
    K.dense_extend(tq, dev(pool.k, "bf16"), dev(pool.v, "bf16"), dev(pool.table), dev(pool.seq_lens),
                   dev(np.array([0, rows], np.int32)), out, shape, ws, causal=False)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    s = q[:, 0].astype(np.float64) @ k.astype(np.float64).T / np.sqrt(d) / np.log(2.0)
    p = 2.0 ** (s - np.ceil(s[:, b:b + 1]))
    frac, _ = np.frexp(p[:, a2])          # bf16 keeps 8 bits: steps of 2^-8 of frac in [0.5, 1)
    near = np.abs(frac * 256 - np.floor(frac * 256) - 0.5) < 256 * 2.0 ** -13
    once = rounded(p[:, a2], "bf16").astype(np.float64)
    ref = (once / p.sum(1))[:, None] * v[a2].astype(np.float64)
    err = np.abs(host(out)[:, 0] - ref) / ref
    assert (~near).sum() > rows / 2 and np.all(err[~near] <= U["bf16"] + 2.0 ** -15), err[~near].max() / U["bf16"]


def close_to_two_parts(got, q, rows_of):
    """bf16 with the weights in two bf16 parts: the rounding of the second leaves u^2 of a weight (u = 2^-8)."""
    for t in range(q.shape[0]):
        for h in range(q.shape[1]):
            k, v = rows_of(t, h)
            qd = q[t, h].astype(np.float64)
            ref, ref_abs = O.attend(qd, k, v), O.attend(qd, k, np.abs(v))
            tol = attend_tol(ref, ref_abs, (np.abs(k) @ np.abs(qd)).max() / np.sqrt(q.shape[2]), len(k), q.shape[2],
                             np.abs(v).max(), "bf16") - U["bf16"] * (1 - U["bf16"]) * ref_abs
            assert np.all(np.abs(got[t, h] - ref) <= tol), (t, h, len(k))


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 8, 64), (14, 2, 64), (8, 1, 128)])
def test_few_rows_keep_the_weights_of_dense_decode(hq, hkv, d):
    """Eight rows or fewer: sequences without groups, few samples of one prompt, few drafted tokens."""
    rng = np.random.default_rng(77)
    g = hq // hkv
    seq = [1, 17, 130, 700, 701, 702]
    pool = Pool(rng, "bf16", hkv, d, 16, seq)
    shape = K.make_shape(**pool.shape(hq))
    kc, vc, lens = dev(pool.k, "bf16"), dev(pool.v, "bf16"), dev(pool.seq_lens)
    rows = {(b, x): [O.gather(c, pool.table[b], seq[b], x) for c in (pool.k, pool.v)]
            for b in range(len(seq)) for x in range(hkv)}
    q = rounded(rng.standard_normal((len(seq), hq, d)), "bf16")
    tq = dev(q, "bf16")
    ws = workspace(K.dense_decode_shared_workspace_bytes(shape, 1))
    out = torch.full_like(tq, SENTINEL)
    K.dense_decode_shared(tq, kc, vc, dev(pool.table), lens, None, None, out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    close_to_two_parts(host(out), q, lambda b, h: rows[b, h // g])
    # the last members as samples of one prompt: their first 640 tokens are sequence `lead`'s
    members, pre = min(3, 8 // g), 640
    lead = len(seq) - members
    K.dense_decode_shared(tq, kc, vc, dev(pool.table), lens, dev(np.array([lead, len(seq)], np.int32)),
                          dev(np.array([pre], np.int32)), out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    close_to_two_parts(host(out), q, lambda b, h: rows[b, h // g] if b < lead else
                       [np.concatenate([s[:pre], o[pre:]]) for s, o in zip(rows[lead, h // g], rows[b, h // g])])
    n = 8 // g
    off = np.array([0, 1, 2, 2 + n, 2 + 2 * n, 3 + 2 * n, 3 + 3 * n], np.int32)
    q = rounded(rng.standard_normal((int(off[-1]), hq, d)), "bf16")
    ws = workspace(K.dense_extend_workspace_bytes(shape, int(off[-1])))
    tq = dev(q, "bf16")
    out = torch.full_like(tq, SENTINEL)
    K.dense_extend(tq, kc, vc, dev(pool.table), lens, dev(off), out, shape, ws)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    of = np.searchsorted(off, np.arange(off[-1]), side="right") - 1
    close_to_two_parts(host(out), q, lambda t, h: [c[:seq[of[t]] - (off[of[t] + 1] - t) + 1] for c in rows[of[t], h // g]])


# ----------------------------------------------------------------------------
# calls that the documentation allows
# ----------------------------------------------------------------------------
def test_stream_given_as_object_and_as_handle():
    c = Chain(78)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # the copies between the calls go there too
        c.run(stream=side)
    torch.cuda.synchronize()
    c.check()
    for n in ("pq", "po", "sq", "so", "dd"):
        c.t[n].fill_(SENTINEL)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        c.run(stream=side.cuda_stream)
    side.synchronize()
    c.check()


def test_return_codes_without_check():
    c = Chain(79)
    t = c.t
    small = c.ws[1][:32]
    args = (t["pq"], t["kc"], t["vc"], t["table"][:1], t["len1"], t["off1"], t["po"], c.s1)
    assert K.dense_extend(*args, small, check=False) == K.ART_ERR_WORKSPACE
    with pytest.raises(K.ArtError):
        K.dense_extend(*args, small)
    assert K.dense_decode_shared(t["sq"], t["kc"], t["vc"], t["table"], t["len2"], t["goff"], t["pre"], t["so"], c.sB,
                                 c.ws[3][8:], check=False) == K.ART_ERR_INVALID_ARG  # not 16-byte aligned
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_results_in_place_of_the_queries(dtype):
    """out may be q: whole items and cut ones, rows of one tile, of several, and few."""
    rng = np.random.default_rng(80)
    hq, hkv, d = 8, 2, 64
    new, seq = [1, 40, 0, 150, 3], [3000, 90, 10, 2150, 700]
    pool = Pool(rng, dtype, hkv, d, 16, seq)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    shape = K.make_shape(**pool.shape(hq))
    q = rounded(rng.standard_normal((int(off[-1]), hq, d)), dtype)
    q1 = rounded(rng.standard_normal((len(seq), hq, d)), dtype)
    cache = dev(pool.k, dtype), dev(pool.v, dtype), dev(pool.table), dev(pool.seq_lens)
    we = workspace(K.dense_extend_workspace_bytes(shape, int(off[-1])))
    wd = workspace(K.dense_decode_shared_workspace_bytes(shape, 0))
    for causal in (True, False):
        a, b = dev(q, dtype), torch.full((len(q), hq, d), SENTINEL, device="cuda").to(dev(q[:1], dtype).dtype)
        K.dense_extend(a, *cache, dev(off), b, shape, we, causal=causal)
        K.dense_extend(a, *cache, dev(off), a, shape, we, causal=causal)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    a = dev(q1, dtype)
    b = torch.empty_like(a)
    K.dense_decode_shared(a, *cache, None, None, b, shape, wd)
    K.dense_decode_shared(a, *cache, None, None, a, shape, wd)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_replay_with_other_lengths_offsets_and_tables():
    """A captured call reads its lengths, offsets, prefixes and tables at the replay."""
    rng = np.random.default_rng(81)
    hq, hkv, d, T, B, cols = 8, 2, 64, 64, 4, 80
    one = dict(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=16, block_size=64, max_pages_per_seq=cols,
               max_visit=1, num_probe=1, num_pages_total=B * cols, dtype=0, batch=B)
    shape = K.make_shape(**one)
    kv = [rounded(np.clip(rng.standard_normal((B * cols, hkv, 16, d)), -3.9, 3.9), "bf16") for _ in range(2)]
    q, q1 = (rounded(rng.standard_normal((n, hq, d)), "bf16") for n in (T, B))
    kc, vc, tq, tq1 = (dev(x, "bf16") for x in (*kv, q, q1))
    table, lens, off, goff, pre = (torch.zeros(n, dtype=torch.int32, device="cuda")
                                   for n in ((B, cols), B, B + 1, 3, 2))
    out, dec = torch.empty_like(tq), torch.empty_like(tq1)
    we, wd = (workspace(n) for n in (K.dense_extend_workspace_bytes(shape, T),
                                     K.dense_decode_shared_workspace_bytes(shape, 2)))

    def run():
        K.dense_extend(tq, kc, vc, table, lens, off, out, shape, we)
        K.dense_decode_shared(tq1, kc, vc, table, lens, goff, pre, dec, shape, wd)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for hlens, hoff, hgoff, hpre in (([64, 1200, 7, 300], [0, 1, 40, 40, 64], [0, 2, 4], [50, 7]),
                                     ([0, 0, 0, 0], [5, 5, 5, 5, 5], [0, 0, 0], [0, 0]),
                                     ([1280, 33, 1280, 1], [0, 30, 63, 64, 64], [1, 1, 4], [9, 33])):
        htable = rng.permutation(B * cols).reshape(B, cols).astype(np.int32)
        for x, h in ((table, htable), (lens, hlens), (off, hoff), (goff, hgoff), (pre, hpre)):
            x.copy_(dev(np.asarray(h, np.int32)))
        out.fill_(SENTINEL)
        dec.fill_(SENTINEL)
        g.replay()
        torch.cuda.synchronize()
        assert K.art_read_device_status(we) == 0 and K.art_read_device_status(wd) == 0
        ref = O.extend(q, kv[0], kv[1], htable, hlens, hoff, True)
        got, held = host(out), ~np.isnan(ref)
        assert np.all(got[~held] == SENTINEL)
        assert np.all(np.abs(got - ref)[held] <= 8 * U["bf16"])  # |v| < 4: u |out| + u sum(p |v|)
        ref = O.decode_shared(q1, kv[0], kv[1], htable, hlens, hgoff, hpre)
        assert np.abs(host(dec) - ref).max() <= 8 * U["bf16"]
