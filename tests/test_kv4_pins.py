"""CPU tests around the cache in 4 bits: pins of the oracle (oracle/kv4.py) by closed forms, the host-side refusals
of the C ABI and the binding's own checks. Nothing here needs a GPU."""
import ctypes

import numpy as np
import pytest

import kv_cache_early_gb300 as K
from kv4_harness import Pool4
from kv_cache_early_gb300 import build as B
from oracle import kv4 as Q
from test_abi import FAKE, good_shape

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.lib()


# ----------------------------------------------------------------------------
# the oracle
# ----------------------------------------------------------------------------
def test_quantise_closed_forms():
    c, s, z = Q.quantise(np.arange(16.0).repeat(2), 32)                  # 0 .. 15: step 1
    assert s == [1.0] and z == [0.0] and np.array_equal(c, np.arange(16).repeat(2))
    c, s, z = Q.quantise(np.full(32, -2.5), 32)                          # one value: no step
    assert s == [0.0] and z == [-2.5] and not c.any()
    x = np.zeros(64)
    x[32:] = np.nan
    c, s, z = Q.quantise(x, 32)                                          # a NaN takes its own group
    assert z[0] == 0.0 and np.isnan(z[1]) and s[1] == 0.0
    # ties go to even: 0.5 -> 0, 1.5 -> 2, 2.5 -> 2 with step 1
    x = np.array([0.0, 15.0, 0.5, 1.5, 2.5, 3.5] + [7.0] * 26)
    assert list(Q.quantise(x, 32)[0][:6]) == [0, 15, 0, 2, 2, 4]
    assert list(Q.quantise(-x, 32)[0][:6]) == [15, 0, 14, 14, 12, 12]
    # the lowest value is rounded down, never up
    for v in (1.0 + 2.0 ** -9, -1.0 - 2.0 ** -9, -1.0 + 2.0 ** -10):
        assert Q.floor_bf16(v) <= v < Q.floor_bf16(v) + 2.0 ** -7
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 128))
    for row in x:
        for group in (32, 64, 128):
            c, s, z = Q.quantise(row, group)
            back = (z[:, None] + s[:, None] * c.reshape(-1, group)).ravel()
            assert np.all(np.abs(back - row) <= 0.5 * s.repeat(group) * (1 + 15 * 2.0 ** -8))


@pytest.mark.parametrize("page,d,group", [(8, 64, 32), (8, 128, 128), (16, 128, 64), (64, 64, 64), (256, 128, 32)])
def test_layout_is_a_partition(page, d, group):
    """Every byte of a page belongs to one token's codes or scales, two columns to a code's byte."""
    seen = np.zeros(Q.page_bytes(page, d, group), int)
    for t in range(page):
        codes, scales = Q.addresses(page, d, group, t)
        for kv in (0, 1):
            seen[codes[kv][0::2]] += 1
            assert np.array_equal(codes[kv][0::2], codes[kv][1::2])
            for k in range(4):
                seen[scales[kv] + k] += 1
    assert np.all(seen == 1)


def test_put_and_get():
    rng = np.random.default_rng(1)
    pool = Pool4(rng, "f32", 2, 64, 16, 32, [20])
    before = pool.bytes.copy()
    x, y = rng.standard_normal(64), rng.standard_normal(64)
    pool.put(0, 17, 1, 0, x)
    pool.put(0, 17, 1, 1, y)
    for kv, row in ((0, x), (1, y)):
        c, s, z = Q.quantise(row, 32)
        code, step, low = Q.get(pool.bytes, 16, 64, 32, int(pool.table[0, 1]), 1, 1, kv)
        assert np.array_equal(code, c) and np.array_equal(step, s.repeat(32)) and np.array_equal(low, z.repeat(32))
    assert (pool.bytes != before).sum() <= 64 + 16


# ----------------------------------------------------------------------------
# refusals
# ----------------------------------------------------------------------------
def append(lib, shape, group=64, q=FAKE, k=FAKE, qs=None, off=FAKE, T=4, table=FAKE, inv=FAKE, rope=K.ArtRope(64, 0, 1.0),
           q_out=FAKE + 4096, cache=FAKE, ws=FAKE, ws_bytes=64):
    w = 1024 if qs is None else qs
    return lib.art_append_kv4(P(q), P(k), P(FAKE), w, w, w, P(off), T, None, P(table), P(FAKE), P(inv),
                              ctypes.byref(rope), P(q_out), P(cache), group, ctypes.byref(shape), P(ws), ws_bytes, None)


def read(lib, shape, group=64, cache=FAKE, table=FAKE, off=FAKE, T=4, out_table=0, out_pages=0, k=FAKE, ws=FAKE, ws_bytes=64):
    return lib.art_read_kv4(P(cache), group, P(table), P(FAKE), P(off), T, P(out_table), out_pages, P(k), P(FAKE),
                            ctypes.byref(shape), P(ws), ws_bytes, None)


def extend(lib, shape, group=64, q=FAKE, cache=FAKE, table=FAKE, off=FAKE, T=4, causal=1, out=FAKE, ws=FAKE, ws_bytes=64):
    return lib.dense_extend_kv4(P(q), P(cache), group, P(table), P(FAKE), P(off), T, causal, P(out), ctypes.byref(shape),
                                P(ws), ws_bytes, None)


INV, UNS, WS = K.ART_ERR_INVALID_ARG, K.ART_ERR_UNSUPPORTED, K.ART_ERR_WORKSPACE


@pytest.mark.parametrize("kw,expect", [
    (dict(ws_bytes=8), WS), (dict(group=16), UNS), (dict(group=96), UNS), (dict(group=0), UNS), (dict(group=256), UNS),
    (dict(shape=good_shape(head_dim=64), group=128), UNS), (dict(shape=good_shape(head_dim=96)), UNS),
    (dict(shape=good_shape(dtype=7)), INV), (dict(k=0), INV), (dict(q=0), INV), (dict(q_out=0), INV), (dict(cache=0), INV),
    (dict(cache=FAKE + 8), INV), (dict(table=0), INV), (dict(inv=0), INV), (dict(qs=1000), INV), (dict(qs=1028), INV),
    (dict(off=0, T=3), INV), (dict(T=-1), INV), (dict(T=1 << 30), UNS), (dict(rope=K.ArtRope(63, 0, 1.0)), INV),
    (dict(rope=K.ArtRope(130, 0, 1.0)), INV), (dict(rope=K.ArtRope(64, 2, 1.0)), INV), (dict(ws=0), INV),
])
def test_append_refusals(lib, kw, expect):
    kw = dict(kw)
    assert append(lib, kw.pop("shape", good_shape()), **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(ws_bytes=8), WS), (dict(group=48), UNS), (dict(shape=good_shape(page_size=4)), UNS), (dict(cache=0), INV),
    (dict(cache=FAKE + 4), INV), (dict(k=0), INV), (dict(k=FAKE + 8), INV), (dict(table=0), INV), (dict(off=0), INV),
    (dict(off=0, T=2, ws_bytes=0), WS), (dict(out_pages=3), INV), (dict(out_table=FAKE, out_pages=3), INV),
    (dict(out_table=FAKE, out_pages=3, off=0), INV), (dict(out_table=FAKE, out_pages=0, off=0, T=0), INV),
    (dict(out_table=FAKE, out_pages=3, off=0, T=0, ws_bytes=0), WS), (dict(out_table=FAKE, out_pages=3, off=0, T=0, k=0), INV),
    (dict(T=-1), INV), (dict(shape=good_shape(page_size=4096, max_pages_per_seq=1 << 19)), UNS), (dict(ws=0), INV),
    (dict(shape=good_shape(batch=33, page_size=4096, max_pages_per_seq=1 << 16), out_table=FAKE, out_pages=3, off=0, T=0), UNS),
    (dict(shape=good_shape(batch=32, page_size=4096, max_pages_per_seq=1 << 16), out_table=FAKE, out_pages=3, off=0, T=0,
          ws_bytes=0), WS),
])
def test_read_refusals(lib, kw, expect):
    kw = dict(kw)
    assert read(lib, kw.pop("shape", good_shape()), **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(ws_bytes=8), WS), (dict(group=24), UNS), (dict(shape=good_shape(num_q_heads=6)), UNS), (dict(cache=0), INV),
    (dict(q=0), INV), (dict(out=0), INV), (dict(q=FAKE + 2), INV), (dict(cache=FAKE + 8), INV), (dict(out=FAKE + 4), INV),
    (dict(table=0), INV), (dict(off=0), INV), (dict(off=0, T=2), WS), (dict(causal=2), INV), (dict(T=-1), INV),
    (dict(ws=0), INV), (dict(shape=good_shape(page_size=4096, max_pages_per_seq=1 << 19)), UNS),
])
def test_extend_refusals(lib, kw, expect):
    kw = dict(kw)
    assert extend(lib, kw.pop("shape", good_shape()), **kw) == expect


def test_sizes(lib):
    s = good_shape()
    for page, d, group in ((16, 128, 64), (8, 64, 32), (256, 128, 128)):
        t = good_shape(page_size=page, head_dim=d)
        assert K.art_kv4_page_bytes(t, group) == Q.page_bytes(page, d, group)
    for bad in (0, 16, 96, 256):
        with pytest.raises(K.ArtError):
            K.art_kv4_page_bytes(s, bad)
    assert lib.art_kv4_page_bytes(None, 64) == 0
    assert K.art_append_kv4_workspace_bytes(s) == K.art_read_kv4_workspace_bytes(s) == 64
    assert lib.art_append_kv4_workspace_bytes(None) == lib.art_read_kv4_workspace_bytes(None) == 0
    assert K.dense_extend_kv4_workspace_bytes(s, 4, 64) > 0
    # with as many tokens as sequences a call may go without offsets: room for either
    assert K.dense_extend_kv4_workspace_bytes(s, s.batch, 64) >= K.dense_extend_kv4_workspace_bytes(s, 3, 64)
    assert K.dense_extend_kv4_workspace_bytes(s, -1, 64) == K.dense_extend_kv4_workspace_bytes(s, 4, 5) == 0
    assert lib.dense_extend_kv4_workspace_bytes(None, 4, 64) == 0


def test_paths(lib):
    """Path 1, in bf16 from 96 rows a sequence and 2048 rows in all on, where the pages fit 4 GiB and the workspace has room for them."""
    s = good_shape(batch=2)  # 4 heads a key head
    assert K.dense_extend_kv4_path(good_shape(batch=40), 959, 64, 1 << 40) == 0
    assert K.dense_extend_kv4_path(good_shape(batch=40), 960, 64, 1 << 40) == 1
    for tokens, path in ((255, 0), (256, 1), (1000, 1)):
        full, least = (f(s, tokens, 64) for f in (K.dense_extend_kv4_workspace_bytes, K.dense_extend_kv4_min_workspace_bytes))
        assert K.dense_extend_kv4_path(s, tokens, 64, full) == path and (full > least) == (path == 1)
        assert K.dense_extend_kv4_path(s, tokens, 64, full - 1) == 0
    assert full - least > 2 * 2 * 8 * 16 * 2 * 128 * 2  # keys and values of every page of the table
    assert K.dense_extend_kv4_path(good_shape(batch=2, dtype=1), 1000, 64, 1 << 40) == 0
    # 2 * 1 << 20 pages of 16 tokens x 2 heads x 128 columns x 2 bytes, keys and values: 32 GiB
    assert K.dense_extend_kv4_path(good_shape(batch=2, max_pages_per_seq=1 << 20), 1000, 64, 1 << 40) == 0
    assert K.dense_extend_kv4_path(s, -1, 64, 1 << 40) == K.dense_extend_kv4_path(s, 1000, 7, 1 << 40) == 0


def test_binding_refuses_tensors_on_the_host():
    torch = pytest.importorskip("torch")
    s = good_shape()
    cache = torch.zeros(16, 2, K.art_kv4_page_bytes(s, 64), dtype=torch.uint8)
    with pytest.raises(K.ArtError, match="not on a CUDA device"):
        K.dense_extend_kv4(torch.zeros(2, 8, 128), cache, None, None, None, None, s, cache, group=64)
    with pytest.raises(K.ArtError, match="4 bits"):
        K.art_read_kv4(cache, None, None, None, None, None, s, cache, group=40)


@pytest.mark.parametrize("size", [K.dense_extend_kv4_workspace_bytes, K.dense_extend_kv4_min_workspace_bytes])
@pytest.mark.parametrize("batch", [1, 7, 128])
@pytest.mark.parametrize("dtype", [0, 1])
def test_a_workspace_serves_calls_with_fewer_tokens(lib, size, batch, dtype):
    """Its bytes never fall as the tokens rise, the call without offsets (a decode step of the batch) among them."""
    for heads in ((32, 8), (8, 1)):
        s = good_shape(batch=batch, num_q_heads=heads[0], num_kv_heads=heads[1], dtype=dtype)
        sizes = [size(s, t, 64) for t in [*range(2 * batch + 3), 5 * batch, 64 * batch, 96 * batch, 1000 * batch]]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_read_refuses_tokens_times_heads_beyond_2_40(lib):
    """2^33 tokens of a table's rows times 128 heads, at the limit and above it."""
    def at(heads):
        s = good_shape(batch=32, num_q_heads=heads, num_kv_heads=heads, page_size=4096, max_pages_per_seq=1 << 16)
        return read(lib, s, out_table=FAKE, out_pages=3, off=0, T=0, ws_bytes=0)  # refused for its workspace at the latest
    assert at(128) == WS and at(129) == UNS
    s = good_shape(num_q_heads=1024, num_kv_heads=1024)
    assert read(lib, s, T=1 << 30, ws_bytes=0) == WS and read(lib, s, T=(1 << 30) + 1, ws_bytes=0) == UNS


def test_the_least_workspace_keeps_path_0(lib):
    """... where a decode step's part is larger than the pages of a small table, too (cross attention of many sequences)."""
    for batch in (16, 4096):
        for pages in (1, 2, 16):
            s = good_shape(batch=batch, num_q_heads=64, num_kv_heads=8, page_size=8, max_pages_per_seq=pages)
            for t in (12 * batch, 40 * batch):
                least, full = (f(s, t, 64) for f in (K.dense_extend_kv4_min_workspace_bytes, K.dense_extend_kv4_workspace_bytes))
                assert K.dense_extend_kv4_path(s, t, 64, least) == 0 and least < full
                assert K.dense_extend_kv4_path(s, t, 64, full) == 1
