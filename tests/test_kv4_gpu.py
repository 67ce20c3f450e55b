"""GPU tests of art_append_kv4, art_read_kv4 and dense_extend_kv4 against the fp64 oracle (oracle/kv4.py), through
the Python binding of the C ABI. The caches' bytes are random wherever no token is, so scales there are
anything, NaN included. Tolerances: kv4_harness.py."""
import numpy as np
import pytest

from cache_ops_harness import E24, U, rounded
from kv4_harness import Pool4, attend_tol, cuts
from oracle import cache_ops as O
from oracle import kv4 as Q

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


def offsets_of(new, lead=0):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + lead


# ----------------------------------------------------------------------------
# art_append_kv4
# ----------------------------------------------------------------------------
def append_case(seed, dtype, heads, page, group, new, ctx, rot, interleaved, fused=False, scale=1.0, positions=None,
                with_q=True, in_place=False, base=10000.0, pad=(0, 0), offsets=True, values=None):
    rng = np.random.default_rng(seed)
    hq, hkv, d = heads
    new, ctx = np.asarray(new), np.asarray(ctx)
    pool = Pool4(rng, dtype, hkv, d, page, group, new + ctx)
    off = offsets_of(new, pad[0])
    T = int(off[-1]) + pad[1]
    q, k, v = (rounded(rng.standard_normal((T, h, d)), dtype) for h in (hq, hkv, hkv))
    if values is not None:
        k, v = rounded(values(rng, k), dtype), rounded(values(rng, v), dtype)
    inv = (base ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    pos = None if positions is None else rng.integers(0, positions, T).astype(np.int32)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(K.art_append_kv4_workspace_bytes(shape))
    cache = dev(pool.bytes)
    if fused:
        row = dev(np.concatenate([q, k, v], 1), dtype)
        tq, tk, tv = row[:, :hq], row[:, hq:hq + hkv], row[:, hq + hkv:]
    else:
        tq, tk, tv = dev(q, dtype), dev(k, dtype), dev(v, dtype)
    q_out = tq if in_place else torch.full((T, hq, d), SENTINEL, dtype=tq.dtype, device="cuda")
    K.art_append_kv4(tq if with_q else None, tk, tv, dev(pool.table), dev(pool.seq_lens), dev(off) if offsets else None,
                     dev(inv) if rot else None, q_out if with_q else None, cache, shape, ws, group=group, rot_dim=rot,
                     interleaved=interleaved, scale=scale, positions=None if pos is None else dev(pos))
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    ref = Q.append(k, v, off, pos, pool.table, pool.seq_lens, inv, rot, interleaved, scale, pool.bytes, page, group, dtype)
    got = cache.cpu().numpy()
    assert np.array_equal(got, ref), np.argwhere(got != ref)[:5]
    if with_q:
        rq = O.append(q, k, v, off, pos, pool.table, pool.seq_lens, inv, rot, interleaved, scale,
                      np.zeros((1, hkv, page, d)), np.zeros((1, hkv, page, d)), 0)[0]
        got = host(q_out)
        held = ~np.isnan(rq).all(axis=(1, 2))
        assert np.all(np.abs(got - rq)[held] <= 8.2 * E24 * 13.0 * scale + U[dtype] * np.abs(rq[held]))
        keep = q if in_place else np.full_like(q, SENTINEL)
        assert np.array_equal(got[~held], keep[~held])  # rows of no sequence stay


HEADS = [(8, 2, 128), (14, 2, 64), (8, 8, 64), (8, 1, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_heads_and_groups(dtype, heads, group, interleaved):
    if group > heads[2]:
        pytest.skip("a group is no wider than a head")
    append_case(1, dtype, heads, 16, group, [1, 5, 0, 33], [0, 15, 100, 1], heads[2], interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot", [0, 2, 6, 8, 16, 30, 32, 48, 64, 126])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_partial_rotation(dtype, rot, interleaved):
    append_case(2, dtype, (4, 2, 128), 8, 32, [3, 9], [7, 0], rot, interleaved, fused=True, scale=1.25)


@pytest.mark.parametrize("page", [8, 32, 64, 128, 4096])
@pytest.mark.parametrize("fused", [False, True])
def test_append_pages_and_strides(page, fused):
    append_case(3, "bf16", (4, 4, 64), page, 64, [1, 70, 2], [page - 1, 63, 0], 64, False, fused=fused, pad=(2, 3))


def test_append_one_token_each():
    append_case(4, "bf16", (8, 2, 128), 16, 64, [1] * 37, np.arange(37) * 3, 128, False, offsets=False)
    append_case(4, "f32", (8, 2, 128), 16, 128, [1], [0], 128, False, offsets=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_many_tokens(dtype):
    """Beyond the size at which a CTA takes a tile of tokens; tiles that begin and end inside units of eight."""
    append_case(5, dtype, (4, 2, 64), 32, 32, [301, 7, 450, 1, 33], [3, 0, 13, 9, 100], 64, False, fused=True)
    append_case(5, dtype, (1, 1, 128), 16, 128, [611], [5], 24, True, with_q=False)
    append_case(5, dtype, (2, 2, 128), 16, 64, [611], [5], 20, False)


def test_append_many_sequences():
    new = np.array([(b * 7) % 3 for b in range(600)])
    append_case(6, "bf16", (1, 1, 64), 8, 32, new, np.arange(600) % 11, 64, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_far_positions(dtype):
    append_case(7, dtype, (2, 2, 128), 16, 64, [200, 1], [3, 2], 128, False, positions=1 << 20, base=500000.0)
    append_case(7, dtype, (2, 2, 64), 16, 64, [50], [3], 64, True, positions=1 << 23, base=10.0)


def test_append_without_queries_and_in_place():
    append_case(8, "bf16", (8, 2, 64), 16, 64, [4, 1], [3, 30], 64, False, with_q=False)
    append_case(8, "bf16", (8, 2, 64), 16, 64, [4, 1], [3, 30], 64, False, in_place=True)
    append_case(8, "f32", (8, 2, 64), 16, 32, [4, 1], [3, 30], 22, True, in_place=True)
    append_case(8, "bf16", (8, 2, 64), 16, 64, [0, 0], [3, 0], 64, False)


def _ties(rng, x):  # steps and values on coarse grids: quotients at and around the borders
    return np.round(x * 4) / 4 + np.where(rng.random(x.shape) < 0.1, 2.0 ** -6, 0)


def _flat(rng, x):  # groups of one value, of two, of zeros of both signs
    y = np.where(np.arange(x.shape[-1]) // 32 % 2, 1.5, np.where(rng.random(x.shape) < 0.5, -0.0, 0.0))
    y[::2] = np.where(rng.random(y[::2].shape) < 0.5, -3.25, 8.0)
    return y


def _wide(rng, x):  # values of all sizes, beside and far from the group's lowest
    return x * np.exp(rng.standard_normal(x.shape) * 5)


def _far(rng, x):  # small differences of large numbers
    return 1000.0 + x * 1e-2


def _not_finite(rng, x):
    y = x.copy()
    y[rng.random(x.shape) < 0.01] = np.inf
    y[rng.random(x.shape) < 0.01] = -np.inf
    y[rng.random(x.shape) < 0.01] = np.nan
    y[0] = x[0] * 2.0 ** 99
    y[1] = x[1] * 2.0 ** 110
    y[2] = x[2] * 2.0 ** -97
    y[3] = x[3] * 2.0 ** -120
    y[4] = np.where(x[4] > 0, 3e38, -3e38)
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("values", [_ties, _flat, _wide, _far, _not_finite])
def test_append_values(dtype, group, values):
    append_case(9, dtype, (2, 2, 128), 16, group, [40], [3], 0, False, values=values)


@pytest.mark.parametrize("few", [True, False])
def test_append_bad_device_data(few):
    rng = np.random.default_rng(10)
    dtype, hq, hkv, d, page, group = "bf16", 4, 2, 64, 16, 32
    new, ctx = np.array([2, 3, 2, 20 if few else 700]), np.array([4, 0, 40, 10])
    pool = Pool4(rng, dtype, hkv, d, page, group, new + ctx)
    off = offsets_of(new)
    q, k, v = (rounded(rng.standard_normal((off[-1], h, d)), dtype) for h in (hq, hkv, hkv))
    lens = pool.seq_lens.copy()
    lens[0] = 1                                   # fewer than its new tokens
    lens[2] = pool.table.shape[1] * page + 1      # beyond the table
    pool.table[3, 1] = pool.num_pages             # second page of the last sequence
    inv = np.ones(d // 2, np.float32)
    shape = K.make_shape(**pool.shape(hq))
    ws = workspace(64)
    cache = dev(pool.bytes)
    q_out = torch.full((int(off[-1]), hq, d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    args = (dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(pool.table), dev(lens))
    K.art_append_kv4(*args, dev(off), dev(inv), q_out, cache, shape, ws, group=group, rot_dim=d)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 4 | 8
    ref = Q.append(k, v, off, None, pool.table, lens, inv, d, False, 1.0, pool.bytes, page, group, dtype)
    assert np.array_equal(cache.cpu().numpy(), ref)
    got = host(q_out)
    assert not got[:2].any() and not got[5:7].any() and (got[2:5] != SENTINEL).all()
    for bad in ([0, 2, 1, 7, int(off[-1])], [0, 2, 5, 7, int(off[-1]) + 9], [-3, 2, 5, 7, int(off[-1])]):
        K.art_append_kv4(*args, dev(np.array(bad, np.int32)), dev(inv), q_out, cache, shape, ws, group=group, rot_dim=d)
        torch.cuda.synchronize()
        assert K.art_read_device_status(ws) & 128


# ----------------------------------------------------------------------------
# art_read_kv4
# ----------------------------------------------------------------------------
def stood_for(pool, b, t, kv, dtype):
    """[heads, d] as the call gives it: one fp32 rounding, then the type's."""
    out = []
    for g in range(pool.hkv):
        c, s, z = Q.get(pool.bytes, pool.page, pool.d, pool.group, int(pool.table[b, t // pool.page]), g, t % pool.page, kv)
        with np.errstate(all="ignore"):
            out.append(rounded((z + s * c).astype(np.float32), dtype))
    return np.array(out)


def same(got, ref):
    return np.array_equal(got, ref, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,d,group", [(2, 128, 32), (2, 128, 64), (1, 128, 128), (3, 64, 32), (8, 64, 64)])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_read_rows(dtype, hkv, d, group, page):
    rng = np.random.default_rng(20)
    lens, new = [1, 130, 0, 9, 70], [1, 77, 0, 3, 70]
    pool = Pool4(rng, dtype, hkv, d, page, group, lens).fill(rng)
    off = offsets_of(new, 2)
    T = int(off[-1]) + 3
    shape = K.make_shape(**pool.shape(hkv))
    ws = workspace(K.art_read_kv4_workspace_bytes(shape))
    outs = [torch.full((T, hkv, d), SENTINEL, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
            for _ in range(2)]
    K.art_read_kv4(dev(pool.bytes), dev(pool.table), dev(pool.seq_lens), dev(off), *outs, shape, ws, group=group)
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    for kv, o in enumerate(outs):
        ref = np.full((T, hkv, d), SENTINEL)
        for b, (n, m) in enumerate(zip(lens, new)):
            for i in range(m):
                ref[off[b] + i] = stood_for(pool, b, n - m + i, kv, dtype)
        assert same(host(o), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,d,group,page", [(2, 128, 64, 16), (1, 64, 32, 8), (2, 64, 64, 128)])
def test_read_pages(dtype, hkv, d, group, page):
    rng = np.random.default_rng(21)
    lens = [300, 1, 0, 65, 8]
    pool = Pool4(rng, dtype, hkv, d, page, group, lens).fill(rng)
    n_out = pool.num_pages + 5
    table = np.full(pool.table.shape, 999999, np.int32)
    order, at = rng.permutation(n_out), 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = order[at:at + m]
        at += m
    shape = K.make_shape(**pool.shape(hkv))
    ws = workspace(64)
    outs = [torch.full((n_out, hkv, page, d), SENTINEL, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32,
                       device="cuda") for _ in range(2)]
    K.art_read_kv4(dev(pool.bytes), dev(pool.table), dev(pool.seq_lens), None, *outs, shape, ws, group=group,
                   out_table=dev(table))
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    for kv, o in enumerate(outs):
        ref = np.full((n_out, hkv, page, d), SENTINEL)
        for b, n in enumerate(lens):
            for t in range(n):
                ref[table[b, t // page], :, t % page] = stood_for(pool, b, t, kv, dtype)
        assert same(host(o), ref)  # places beyond a sequence's end stay


def test_read_one_token_each_and_many_sequences():
    rng = np.random.default_rng(22)
    lens = 1 + np.arange(700) % 13  # more sequences than a block has threads
    pool = Pool4(rng, "f32", 1, 64, 8, 32, lens).fill(rng)
    shape = K.make_shape(**pool.shape(1))
    ws = workspace(64)
    outs = [torch.full((700, 1, 64), SENTINEL, device="cuda") for _ in range(2)]
    K.art_read_kv4(dev(pool.bytes), dev(pool.table), dev(pool.seq_lens), None, *outs, shape, ws, group=32)
    for kv, o in enumerate(outs):
        assert same(host(o), np.array([stood_for(pool, b, n - 1, kv, "f32") for b, n in enumerate(lens)]))
    off = offsets_of(lens)
    outs = [torch.full((int(off[-1]), 1, 64), SENTINEL, device="cuda") for _ in range(2)]
    K.art_read_kv4(dev(pool.bytes), dev(pool.table), dev(pool.seq_lens), dev(off), *outs, shape, ws, group=32)
    for kv, o in enumerate(outs):
        assert same(host(o), np.array([stood_for(pool, b, t, kv, "f32") for b, n in enumerate(lens) for t in range(n)]))


def test_read_bad_device_data():
    rng = np.random.default_rng(23)
    page, group = 16, 64
    lens = [20, 5, 40]
    pool = Pool4(rng, "bf16", 2, 64, page, group, lens).fill(rng)
    shape = K.make_shape(**pool.shape(2))
    ws = workspace(64)
    good = pool.table.copy()
    pool.table[0, 1] = -1
    bad_lens = np.array([20, 3, pool.table.shape[1] * page + 1], np.int32)
    off = offsets_of([20, 4, 2])
    outs = [torch.full((int(off[-1]), 2, 64), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    K.art_read_kv4(dev(pool.bytes), dev(pool.table), dev(bad_lens), dev(off), *outs, shape, ws, group=group)
    assert K.art_read_device_status(ws) == 4 | 8
    for kv, o in enumerate(outs):
        got = host(o)
        assert same(got[:16], np.array([stood_for(pool, 0, t, kv, "bf16") for t in range(16)]))
        assert not got[16:].any()  # the bad page's tokens, and the sequences with bad lengths
    for wrong in ([0, 2, 1, 3], [0, 20, 24, 27], [-1, 20, 24, 26]):
        outs = [torch.full((26, 2, 64), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        K.art_read_kv4(dev(pool.bytes), dev(good), dev(pool.seq_lens), dev(np.array(wrong, np.int32)), *outs, shape, ws,
                       group=group)
        assert K.art_read_device_status(ws) & 128
        assert all((host(o) == SENTINEL).all() for o in outs)
    # pages: a bad id of the output is skipped, one of the cache reads as zero, a bad length writes nothing
    to = np.arange(9, dtype=np.int32).reshape(3, 3)[:, :pool.table.shape[1]]
    to = np.concatenate([to, np.full((3, pool.table.shape[1] - to.shape[1]), -5, np.int32)], 1)
    to[2, 1] = 9
    outs = [torch.full((9, 2, page, 64), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lens2 = np.array([20, -1, 40], np.int32)
    K.art_read_kv4(dev(pool.bytes), dev(pool.table), dev(lens2), None, *outs, shape, ws, group=group, out_table=dev(to))
    assert K.art_read_device_status(ws) == 4 | 8
    for kv, o in enumerate(outs):
        ref = np.full((9, 2, page, 64), SENTINEL)
        for t in range(20):
            ref[t // page, :, t % page] = 0 if t >= 16 else stood_for(pool, 0, t, kv, "bf16")
        for t in list(range(16)) + list(range(32, 40)):
            ref[6 + t // page, :, t % page] = stood_for(pool, 2, t, kv, "bf16")
        assert same(host(o), ref)


# ----------------------------------------------------------------------------
# dense_extend_kv4
# ----------------------------------------------------------------------------
def run_extend(pool, q, off, causal, hq, offsets=True, table=None, lens=None, in_place=False, path=0):
    """path 0: a workspace that keeps every call on the codes."""
    dtype = pool.dtype
    shape = K.make_shape(**pool.shape(hq))
    T = q.shape[0]
    size = K.dense_extend_kv4_workspace_bytes if path else K.dense_extend_kv4_min_workspace_bytes
    ws = workspace(size(shape, T, pool.group))
    tq = dev(q, dtype)
    out = tq if in_place else torch.full(q.shape, SENTINEL, dtype=tq.dtype, device="cuda")
    K.dense_extend_kv4(tq, dev(pool.bytes), dev(pool.table if table is None else table),
                       dev(pool.seq_lens if lens is None else lens), dev(off) if offsets else None, out, shape, ws,
                       group=pool.group, causal=causal)
    torch.cuda.synchronize()
    return host(out), K.art_read_device_status(ws)


def check(got, ref, terms, d, dtype, keep=None):
    held = ~np.isnan(ref).all(axis=(1, 2)) if keep is None else keep
    tol = attend_tol(ref, terms, d, dtype)
    err = np.abs(got - ref)[held]
    assert np.all(err <= tol[held]), (np.nanmax(err / tol[held]), np.argwhere(~(err <= tol[held]))[:4])
    assert np.all(got[~held] == SENTINEL)


def extend_case(seed, dtype, heads, page, group, new, lens, causal=True, pad=(0, 0), scale=1.0, kscale=1.0, qscale=1.0,
                in_place=False):
    rng = np.random.default_rng(seed)
    hq, hkv, d = heads
    pool = Pool4(rng, dtype, hkv, d, page, group, lens).fill(rng, scale, kscale)
    off = offsets_of(new, pad[0])
    T = int(off[-1]) + pad[1]
    q = rounded(rng.standard_normal((T, hq, d)) * qscale, dtype)
    got, status = run_extend(pool, q, off, causal, hq, in_place=in_place)
    assert status == 0
    ref, terms = Q.extend(q, pool.bytes, pool.table, pool.seq_lens, off, causal, page, group)
    check(got, ref, terms, d, dtype)


def decode_case(seed, dtype, heads, page, group, lens, scale=1.0, kscale=1.0, qscale=1.0):
    rng = np.random.default_rng(seed)
    hq, hkv, d = heads
    pool = Pool4(rng, dtype, hkv, d, page, group, lens).fill(rng, scale, kscale)
    B = len(lens)
    q = rounded(rng.standard_normal((B, hq, d)) * qscale, dtype)
    got, status = run_extend(pool, q, None, True, hq, offsets=False)
    assert status == 0
    ref, terms = Q.extend(q, pool.bytes, pool.table, pool.seq_lens, np.arange(B + 1), False, page, group)
    check(got, ref, terms, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (2, 2, 64), (8, 1, 128), (2, 1, 128)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_decode(dtype, heads, group):
    if group > heads[2]:
        pytest.skip("a group is no wider than a head")
    decode_case(30, dtype, heads, 16, group, [1, 0, 7, 16, 33, 127, 128, 129, 300])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 4096])
def test_decode_pages(dtype, page):
    decode_case(31, dtype, (4, 1, 64), page, 32, [5, 63, 64, 65, 200, 513])


def test_decode_long():
    """Sequences that many CTAs share, and more items than CTAs."""
    decode_case(32, "bf16", (4, 1, 128), 64, 64, [9000, 1])
    decode_case(33, "f32", (2, 1, 64), 64, 64, [5001])
    decode_case(34, "bf16", (4, 4, 64), 16, 64, list(range(1, 60)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (4, 4, 64), (8, 1, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_extend_heads(dtype, heads, causal):
    new = [1, 3, 0, 17, 5, 2]
    lens = [1, 3, 4, 150, 260, 0 if not causal else 2]
    extend_case(40, dtype, heads, 16, 32, new, lens, causal, pad=(1, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 40])
def test_extend_row_counts(dtype, n):
    """Rows of an item from one to several tiles: 4 heads a key head."""
    extend_case(41, dtype, (4, 1, 64), 8, 64, [n, n], [n, 200 + n])
    extend_case(42, dtype, (4, 1, 128), 64, 64, [n], [130 + n], in_place=True)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_extend_whole_prompts(group):
    extend_case(43, "bf16", (4, 2, 128), 16, group, [150, 1, 33], [150, 1, 33])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_peaked_and_climbing_scores(dtype):
    """References that move, far and often; weights of one key only."""
    decode_case(50, dtype, (8, 1, 64), 16, 32, [300, 600], qscale=6.0)
    decode_case(51, dtype, (8, 1, 64), 16, 64, [500], kscale=lambda b, t: 0.02 * (t + 1))
    extend_case(52, dtype, (4, 1, 64), 16, 64, [8], [400], kscale=lambda b, t: 0.02 * (400 - t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** -80, 2.0 ** -30, 2.0 ** 30, 2.0 ** 80])
def test_values_of_any_size(dtype, size):
    decode_case(53, dtype, (4, 1, 64), 16, 32, [40, 300], scale=size)
    extend_case(54, dtype, (4, 1, 64), 16, 64, [5], [200], scale=lambda b, t: size if t % 7 == 0 else 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes_of_queries_and_keys(dtype):
    """Scores of ordinary size from large queries and small keys, and the other way round."""
    for e in (-60, -20, 20, 60):
        decode_case(55, dtype, (4, 1, 128), 16, 64, [200], qscale=2.0 ** e, kscale=2.0 ** -e)
    # rows of very different size beside each other; a row of zeros
    rng = np.random.default_rng(56)
    pool = Pool4(rng, dtype, 1, 64, 16, 32, [150]).fill(rng)
    q = rounded(rng.standard_normal((1, 8, 64)) * 2.0 ** np.arange(-30, 2, 4)[None, :, None], dtype)
    q[0, 3] = 0
    got, status = run_extend(pool, q, None, True, 8, offsets=False)
    ref, terms = Q.extend(q, pool.bytes, pool.table, pool.seq_lens, [0, 1], False, 16, 32)
    check(got, ref, terms, 64, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_with_large_columns(dtype, d):
    """Columns of a query 64 times larger than the others, whose keys are small there: scores stay ordinary."""
    rng = np.random.default_rng(64)
    hq, page, group = 4, 16, 32
    pool = Pool4(rng, dtype, 1, d, page, group, [500, 77])
    small = np.where(np.arange(d) % 32 == 5, 1 / 64, 1.0)
    for b, n in enumerate(pool.seq_lens):
        for t in range(int(n)):
            pool.put(b, t, 0, 0, rounded(rng.standard_normal(d) * small, dtype))
            pool.put(b, t, 0, 1, rounded(rng.standard_normal(d), dtype))
    q = rounded(rng.standard_normal((2, hq, d)) / small, dtype)
    got, status = run_extend(pool, q, None, True, hq, offsets=False)
    assert status == 0
    ref, terms = Q.extend(q, pool.bytes, pool.table, pool.seq_lens, [0, 1, 2], False, page, group)
    steps = max(Q.held(pool.bytes, pool.table[b], int(n), 0, page, d, group, 0)[1].max() for b, n in enumerate(pool.seq_lens))
    tol = attend_tol(ref, terms, d, dtype)
    if dtype == "bf16":
        tol = tol + cuts(np.abs(q).max(-1)[..., None], steps, terms[..., 2][..., None], d)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


def test_flat_groups():
    """Groups without a step: codes mean nothing there."""
    rng = np.random.default_rng(57)
    pool = Pool4(rng, "f32", 1, 64, 16, 32, [100]).fill(rng)
    for t in range(100):
        pool.put(0, t, 0, 1, np.full(64, float(t % 5)))
    q = rng.standard_normal((1, 4, 64)).astype(np.float32)
    got, _ = run_extend(pool, q, None, True, 4, offsets=False)
    ref, terms = Q.extend(q, pool.bytes, pool.table, pool.seq_lens, [0, 1], False, 16, 32)
    check(got, ref, terms, 64, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups_of_nan_stay_with_the_rows_that_see_them(dtype):
    """A key or value that is no number reaches the rows that see it and no other (4 heads, causal)."""
    rng = np.random.default_rng(58)
    n, ctx = 6, 100
    pool = Pool4(rng, dtype, 1, 64, 16, 32, [ctx + n, 70]).fill(rng)
    x = np.full(64, np.nan)
    x[:32] = 1.0
    pool.put(0, ctx + 3, 0, 1, x)   # its values' second group: tokens 3 .. of the new ones
    pool.put(0, ctx + 5, 0, 0, x)   # a key: the last token
    q = rounded(rng.standard_normal((n + 1, 4, 64)), dtype)
    off = offsets_of([n, 1])
    got, status = run_extend(pool, q, off, True, 4)
    assert status == 0
    ref, terms = Q.extend(q, pool.bytes, pool.table, pool.seq_lens, off, True, 16, 32)
    assert np.isnan(got[5]).all() and np.isnan(got[3:5, :, 32:]).all()
    for rows, cols in (([0, 1, 2, 6], slice(0, 64)),):
        check(got[rows], ref[rows], terms[rows], 64, dtype)
    # the columns of the other group: attention over a cache whose NaN are zeros there
    clean = Pool4(np.random.default_rng(58), dtype, 1, 64, 16, 32, [ctx + n, 70])
    clean.bytes, clean.table = pool.bytes.copy(), pool.table
    clean.put(0, ctx + 3, 0, 1, np.where(np.isnan(x), 0.0, x))
    ref, terms = Q.extend(q, clean.bytes, pool.table, pool.seq_lens, off, True, 16, 32)
    assert np.all(np.abs(got - ref)[3:5, :, :32] <= attend_tol(ref, terms, 64, dtype)[3:5, :, :32])


def test_query_of_nan_stays_in_its_row():
    rng = np.random.default_rng(59)
    for n in (1, 3, 6):
        pool = Pool4(rng, "bf16", 1, 64, 16, 64, [200]).fill(rng)
        q = rounded(rng.standard_normal((n, 4, 64)), "bf16")
        q[0, 1, 5] = np.nan
        off = offsets_of([n])
        got, _ = run_extend(pool, q, off, True, 4)
        assert np.isnan(got[0, 1]).all()
        q2 = np.where(np.isnan(q), 0.0, q)
        ref, terms = Q.extend(q2, pool.bytes, pool.table, pool.seq_lens, off, True, 16, 64)
        ok = np.ones((n, 4), bool)
        ok[0, 1] = False
        assert np.all((np.abs(got - ref) <= attend_tol(ref, terms, 64, "bf16"))[ok])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [[2, 3, 1, 30, 4], [1, 1, 1, 1, 1]])
def test_extend_bad_device_data(dtype, new):
    rng = np.random.default_rng(60)
    page, group = 16, 32
    lens = [40, 50, 30, 300, 20]
    pool = Pool4(rng, dtype, 2, 64, page, group, lens).fill(rng)
    off = offsets_of(new)
    q = rounded(rng.standard_normal((int(off[-1]), 8, 64)), dtype)
    bad_lens = pool.seq_lens.copy()
    bad_lens[0] = -1
    bad_lens[2] = pool.table.shape[1] * page + 1
    table = pool.table.copy()
    table[3, 7] = pool.num_pages
    for offsets in (True, False):
        if not offsets and new[1] != 1:
            continue
        got, status = run_extend(pool, q, off, True, 8, offsets=offsets, table=table, lens=bad_lens)
        assert status == 4 | 8
        ref, terms = Q.extend(q, pool.bytes, pool.table, pool.seq_lens, off, True, page, group, skip=(0, 2, 3))
        check(got, ref, terms, 64, dtype)
    for wrong in ([0, 2, 1, 3, 4, 5], [0, 1, 2, 3, 4, int(off[-1]) + 1], [-1, 1, 2, 3, 4, 5]):
        got, status = run_extend(pool, q, np.array(wrong, np.int32), True, 8)
        assert status & 128 and (got == SENTINEL).all()


def test_no_tokens():
    rng = np.random.default_rng(61)
    pool = Pool4(rng, "bf16", 2, 64, 16, 32, [10, 0]).fill(rng)
    got, status = run_extend(pool, np.zeros((0, 4, 64), np.float32), np.zeros(3, np.int32), True, 4)
    assert got.size == 0 and status == 0
    got, status = run_extend(pool, np.ones((3, 4, 64), np.float32), np.zeros(3, np.int32), True, 4)
    assert (got == SENTINEL).all() and status == 0


# ----------------------------------------------------------------------------
# prompt chunks: the cache read back in the workspace
# ----------------------------------------------------------------------------
def plain_rows(pool, b, kv):
    """What art_read_kv4 gives of a sequence, [heads, tokens, d]."""
    n = int(pool.seq_lens[b])
    out = []
    for g in range(pool.hkv):
        c, s, z = Q.held(pool.bytes, pool.table[b], n, g, pool.page, pool.d, pool.group, kv)
        out.append(rounded((z + s * c).astype(np.float32), "bf16").astype(np.float64))
    return out


@pytest.mark.parametrize("heads,page,group", [((8, 2, 128), 16, 64), ((8, 1, 64), 8, 32), ((14, 2, 128), 256, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_chunks(heads, page, group, causal):
    """Against attention over the values rounded to bf16, with dense_extend's tolerances (cache_ops_harness)."""
    import cache_ops_harness as H
    rng = np.random.default_rng(80)
    hq, hkv, d = heads
    new, lens = [200, 0, 90, 3], [200, 40, 240, 131]
    pool = Pool4(rng, "bf16", hkv, d, page, group, lens).fill(rng)
    pool.table[1] = -7  # a sequence without new tokens is not read
    off = offsets_of(new, 1)
    T = int(off[-1]) + 2
    q = rounded(rng.standard_normal((T, hq, d)), "bf16")
    shape = K.make_shape(**pool.shape(hq))
    n = K.dense_extend_kv4_workspace_bytes(shape, T, group)
    assert K.dense_extend_kv4_path(shape, T, group, n) == 1 and K.dense_extend_kv4_path(shape, T, group, n - 1) == 0
    got, status = run_extend(pool, q, off, causal, hq, path=1)
    assert status == 0
    for b, (m, s) in enumerate(zip(new, lens)):
        if m == 0:
            continue
        k, v = plain_rows(pool, b, 0), plain_rows(pool, b, 1)
        for h in range(hq):
            g = h // (hq // hkv)
            for i in range(m):
                seen = s - m + i + 1 if causal else s
                x, kk, vv = q[off[b] + i, h], k[g][:seen], v[g][:seen]
                ref, ref_abs = O.attend(x, kk, vv), O.attend(x, kk, np.abs(vv))
                score = (np.abs(kk) @ np.abs(x)).max() / np.sqrt(d)
                tol = H.attend_tol(ref, ref_abs, score, seen, d, np.abs(vv).max(), "bf16")
                assert np.all(np.abs(got[off[b] + i, h] - ref) <= tol), (b, h, i)
    assert (got[:1] == SENTINEL).all() and (got[T - 2:] == SENTINEL).all()


def test_prompt_chunks_bad_device_data():
    rng = np.random.default_rng(81)
    new, lens = [90, 100, 80, 130], [90, 100, 150, 300]
    pool = Pool4(rng, "bf16", 2, 64, 16, 32, lens).fill(rng)
    off = offsets_of(new)
    q = rounded(rng.standard_normal((int(off[-1]), 8, 64)), "bf16")
    good, status = run_extend(pool, q, off, True, 8, path=1)
    assert status == 0 and np.isfinite(good).all()
    bad_lens, table = pool.seq_lens.copy(), pool.table.copy()
    bad_lens[0] = 89                    # fewer than its new tokens
    bad_lens[2] = pool.table.shape[1] * 16 + 1
    table[3, 7] = pool.num_pages
    got, status = run_extend(pool, q, off, True, 8, table=table, lens=bad_lens, path=1)
    assert status == 4 | 8
    assert not got[:90].any() and not got[190:].any() and np.array_equal(got[90:190], good[90:190])
    got, status = run_extend(pool, q, np.array([0, 90, 80, 270, 400], np.int32), True, 8, path=1)
    assert status & 128 and (got == SENTINEL).all()


# ----------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_run(dtype):
    """Prompts, then decode steps, through all three calls on one cache, replayed from a graph as the lengths grow;
    against attention over what is read back, and dense_extend over the pages that are read back."""
    torch.manual_seed(0)
    hq, hkv, d, page, group, B, cap = 8, 2, 128, 16, 64, 3, 20
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    shape = K.make_shape(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page, block_size=64,
                         max_pages_per_seq=cap, max_visit=1, num_probe=1, num_pages_total=B * cap,
                         dtype=0 if dtype == "bf16" else 1)
    table = torch.randperm(B * cap, device="cuda").to(torch.int32).reshape(B, cap)
    cache = torch.randint(0, 256, (B * cap, hkv, K.art_kv4_page_bytes(shape, group)), dtype=torch.uint8, device="cuda")
    inv = (10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)).float()
    lens = torch.tensor([37, 1, 230], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 37, 38, 268], dtype=torch.int32, device="cuda")
    ws = [workspace(K.art_append_kv4_workspace_bytes(shape)), workspace(K.art_read_kv4_workspace_bytes(shape))]
    T = 268
    ws_e = workspace(K.dense_extend_kv4_min_workspace_bytes(shape, T, group))  # over the codes
    qkv = torch.randn(T, hq + 2 * hkv, d, device="cuda").to(dt)
    q_rot, out = torch.empty(T, hq, d, dtype=dt, device="cuda"), torch.empty(T, hq, d, dtype=dt, device="cuda")
    K.art_append_kv4(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], table, lens, off, inv, q_rot, cache, shape, ws[0],
                     group=group, rot_dim=d)
    K.dense_extend_kv4(q_rot, cache, table, lens, off, out, shape, ws_e, group=group)

    def reference(q, new):
        """fp64 attention over the fp32 values of the cache (an fp32 shape reads them unrounded)."""
        s32 = K.make_shape(**{n: getattr(shape, n) for n, _ in K.ArtShape._fields_ if n != "dtype"}, dtype=1)
        outs, at = [], 0
        total = int(lens.sum())
        o = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), lens.cumsum(0).to(torch.int32)])
        k, v = (torch.empty(total, hkv, d, device="cuda") for _ in range(2))
        K.art_read_kv4(cache, table, lens, o, k, v, s32, ws[1], group=group)
        for b in range(B):
            n, m = int(lens[b]), new[b]
            kk, vv = (x[int(o[b]):int(o[b + 1])].double() for x in (k, v))
            for i in range(m):
                seen = n - m + i + 1
                qq = q[at + i].double().reshape(hkv, hq // hkv, d)
                s = torch.einsum("hgd,lhd->hgl", qq, kk[:seen]) / d ** 0.5
                outs.append(torch.einsum("hgl,lhd->hgd", torch.softmax(s, -1), vv[:seen]).reshape(hq, d))
            at += m
        return torch.stack(outs)

    # bf16: output 2^-8 |ref| and weights 2^-12 of values of at most 16 steps, |v| < 6; fp32: far below
    def near(got, ref):
        tol = (2.0 ** -8 * ref.abs() + 2.0 ** -12 * 12) if dtype == "bf16" else 2.0 ** -24 * (8 * 12 * 40 + 8 * 15 + 16) * 12 + 0 * ref
        assert (((got.double() - ref).abs() <= tol)).all(), float((got.double() - ref).abs().max())

    near(out, reference(q_rot, [37, 1, 230]))
    # the same cache through the plain calls: pages read back, dense_extend over them
    kc, vc = (torch.full((B * cap, hkv, page, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    K.art_read_kv4(cache, table, lens, None, kc, vc, shape, ws[1], group=group, out_table=table)
    plain = torch.empty_like(out)
    ws_p = workspace(K.dense_extend_workspace_bytes(shape, T))
    K.dense_extend(q_rot, kc, vc, table, lens, off, plain, shape, ws_p)
    # ... as dense_extend_kv4 does by itself where the workspace holds the pages: the same bits
    if dtype == "bf16":
        n = K.dense_extend_kv4_workspace_bytes(shape, T, group)
        assert K.dense_extend_kv4_path(shape, T, group, n) == 1
        back, ws_b = torch.empty_like(out), workspace(n)
        K.dense_extend_kv4(q_rot, cache, table, lens, off, back, shape, ws_b, group=group)
        assert torch.equal(back, plain) and K.art_read_device_status(ws_b) == 0
    # there keys and values are rounded to bf16: 2^-8 of scores (|q . k| / sqrt(d) < 40) and of values, on both sides
    tol = 2.0 ** -8 * (2 * 40 + 2) * 6 if dtype == "bf16" else 1e-3
    assert float((plain.double() - out.double()).abs().max()) <= tol
    # decode steps from one graph
    step = torch.empty(B, hq + 2 * hkv, d, dtype=dt, device="cuda")
    q1, o1 = torch.empty(B, hq, d, dtype=dt, device="cuda"), torch.empty(B, hq, d, dtype=dt, device="cuda")
    ws_d = workspace(K.dense_extend_kv4_workspace_bytes(shape, B, group))

    def decode():
        lens.add_(1)
        K.art_append_kv4(step[:, :hq], step[:, hq:hq + hkv], step[:, hq + hkv:], table, lens, None, inv, q1, cache, shape,
                         ws[0], group=group, rot_dim=d)
        K.dense_extend_kv4(q1, cache, table, lens, None, o1, shape, ws_d, group=group)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step.copy_(torch.randn(step.shape, device="cuda"))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a stream of the caller's
        decode()
    torch.cuda.current_stream().wait_stream(side)
    near(o1, reference(q1, [1] * B))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode()
    for i in range(40):
        step.copy_(torch.randn(step.shape, device="cuda"))
        graph.replay()
        if i % 8 == 0:
            near(o1, reference(q1, [1] * B))
    torch.cuda.synchronize()
    assert all(K.art_read_device_status(w) == 0 for w in ws + [ws_d, ws_e])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_sequences(dtype):
    """More sequences than a block has threads, some empty: decode, and one to three new tokens of some."""
    lens = [(b * 37) % 50 for b in range(600)]
    decode_case(62, dtype, (2, 1, 64), 8, 32, lens)
    new = [min(n, b % 4) for b, n in enumerate(lens)]
    extend_case(63, dtype, (4, 1, 64), 8, 64, new, lens)


def test_cache_beyond_32_bits():
    """Pages that lie more than 4 GiB into the cache and into the plain pool: the same results as in the first pages."""
    torch.manual_seed(1)
    hq, hkv, d, page, group, B = 8, 8, 128, 64, 128, 2
    pages = 64000
    shape = K.make_shape(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page, block_size=64,
                         max_pages_per_seq=4, max_visit=1, num_probe=1, num_pages_total=pages, dtype=0)
    cache = torch.zeros(pages, hkv, K.art_kv4_page_bytes(shape, group), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    lens = torch.tensor([200, 130], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 200, 330], dtype=torch.int32, device="cuda")
    rows = torch.randn(330, hq + 2 * hkv, d, device="cuda").bfloat16()
    inv = (10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)).float()
    ws = workspace(max(K.dense_extend_kv4_workspace_bytes(shape, 330, group), 64))
    small = K.make_shape(**{n: getattr(shape, n) for n, _ in K.ArtShape._fields_ if n != "num_pages_total"}, num_pages_total=8)
    results = []
    for first in (0, pages - 8):
        table = (first + torch.arange(8, device="cuda")).int().reshape(B, 4)
        q = torch.empty(330, hq, d, dtype=torch.bfloat16, device="cuda")
        K.art_append_kv4(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], table, lens, off, inv, q, cache, shape, ws,
                         group=group, rot_dim=d)
        out, one = torch.empty_like(q), torch.empty(B, hq, d, dtype=torch.bfloat16, device="cuda")
        K.dense_extend_kv4(q, cache, table, lens, off, out, shape, ws, group=group)
        K.dense_extend_kv4(q[:2], cache, table, lens, None, one, shape, ws, group=group)
        k, v = (torch.empty(330, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        K.art_read_kv4(cache, table, lens, off, k, v, shape, ws, group=group)
        assert K.art_read_device_status(ws) == 0
        results.append((q, out, one, k, v, cache[first:first + 8].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*results)) and results[0][5].any()
    n = (1 << 32) // (hkv * page * d * 2) + 16  # pages of a plain pool beyond 4 GiB
    kc, vc = (torch.zeros(n, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    to = (n - 8 + torch.arange(8, device="cuda")).int().reshape(B, 4)
    K.art_read_kv4(results[0][5], torch.arange(8, device="cuda").int().reshape(B, 4), lens, None, kc, vc, small, ws,
                   group=group, out_table=to)
    assert K.art_read_device_status(ws) == 0
    for b in range(B):
        for c in range(4):
            m = max(0, min(64, int(lens[b]) - 64 * c))
            for pool, x in ((kc, results[0][3]), (vc, results[0][4])):
                lo = int(off[b]) + 64 * c
                assert torch.equal(pool[int(to[b, c]), :, :m].transpose(0, 1), x[lo:lo + m])
                assert not pool[int(to[b, c]), :, m:].any()


def test_calls_repeat_and_overlap():
    """The same call gives the same bits; two calls on two streams with workspaces of their own do not disturb
    each other."""
    rng = np.random.default_rng(70)
    pool = Pool4(rng, "bf16", 2, 128, 16, 64, [700, 33, 250]).fill(rng)
    shape = K.make_shape(**pool.shape(8))
    qs = [dev(rng.standard_normal((3, 8, 128)), "bf16") for _ in range(2)]
    args = [dev(x) for x in (pool.bytes, pool.table, pool.seq_lens)]
    n = K.dense_extend_kv4_workspace_bytes(shape, 3, 64)
    ws = [workspace(n) for _ in range(2)]
    first = []
    for q, w in zip(qs, ws):
        out = torch.empty_like(q)
        K.dense_extend_kv4(q, args[0], args[1], args[2], None, out, shape, w, group=64)
        first.append(out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    for i in range(20):
        for q, w, s, o in zip(qs, ws, streams, outs):
            K.dense_extend_kv4(q, args[0], args[1], args[2], None, o[i], shape, w, group=64,
                               stream=s if i % 2 else s.cuda_stream)
    torch.cuda.synchronize()
    for f, o in zip(first, outs):
        assert all(torch.equal(f, x) for x in o)


def test_bounded_wait_expires_and_next_call_is_clean(monkeypatch):
    rng = np.random.default_rng(71)
    pool = Pool4(rng, "bf16", 2, 64, 16, 32, [300, 20]).fill(rng)
    q = rounded(rng.standard_normal((2, 8, 64)), "bf16")
    monkeypatch.setenv("ART_TEST_STALL_NS", "200000")
    _, status = run_extend(pool, q, None, True, 8, offsets=False)
    assert status & 32
    monkeypatch.delenv("ART_TEST_STALL_NS")
    got, status = run_extend(pool, q, None, True, 8, offsets=False)
    assert status == 0
    ref, terms = Q.extend(q, pool.bytes, pool.table, pool.seq_lens, [0, 1, 2], False, 16, 32)
    check(got, ref, terms, 64, "bf16")


def test_binding_refusals():
    rng = np.random.default_rng(72)
    pool = Pool4(rng, "bf16", 2, 64, 16, 32, [30, 20])
    shape = K.make_shape(**pool.shape(4))
    cache, table, lens = (dev(x) for x in (pool.bytes, pool.table, pool.seq_lens))
    q, out = (torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = workspace(K.dense_extend_kv4_workspace_bytes(shape, 2, 32))
    off = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    inv = torch.ones(32, device="cuda")

    def calls(**kw):
        a = dict(q=q, out=out, k=k, v=v, cache=cache, table=table, lens=lens, off=off, ws=ws, group=32, inv=inv)
        a.update(kw)
        return (lambda: K.dense_extend_kv4(a["q"], a["cache"], a["table"], a["lens"], a["off"], a["out"], shape, a["ws"],
                                           group=a["group"]),
                lambda: K.art_read_kv4(a["cache"], a["table"], a["lens"], a["off"], a["k"], a["v"], shape, a["ws"],
                                       group=a["group"]),
                lambda: K.art_append_kv4(a["q"], a["k"], a["v"], a["table"], a["lens"], a["off"], a["inv"], a["out"],
                                         a["cache"], shape, a["ws"], group=a["group"], rot_dim=64))

    for c in calls():
        assert c() == K.ART_OK
    bad_all = [dict(cache=cache[:-1]), dict(cache=cache.transpose(0, 1).contiguous().transpose(0, 1)), dict(cache=cache.float()),
               dict(group=64), dict(table=table[:, :-1].contiguous()), dict(lens=lens.long()), dict(off=off[:-1]),
               dict(ws=ws.cpu()), dict(ws=ws[::2])]
    for kw in bad_all:
        for c in calls(**kw):
            with pytest.raises(K.ArtError):
                c()
    ext, rd, app = range(3)
    for which, kw in ((ext, dict(q=q.float())), (ext, dict(out=out[:1])), (ext, dict(q=q.transpose(1, 2))),
                      (rd, dict(k=k.float())), (rd, dict(v=v[:1])), (app, dict(k=k.float())), (app, dict(v=v[:, :1])),
                      (app, dict(inv=inv[:-1])), (app, dict(out=out[:1])), (app, dict(q=q.float()))):
        with pytest.raises(K.ArtError):
            calls(**kw)[which]()
    with pytest.raises(K.ArtError):  # one token of each sequence: as many rows as sequences
        K.dense_extend_kv4(torch.cat([q, q]), cache, table, lens, None, torch.cat([out, out]), shape, ws, group=32)
    small = torch.zeros(8, dtype=torch.uint8, device="cuda")
    for c in calls(ws=small):
        with pytest.raises(K.ArtError):
            c()
