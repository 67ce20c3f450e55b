"""CPU tests around art_append_kv, dense_extend and dense_decode_shared: pins of
the oracle (oracle/cache_ops.py) by closed forms, the host-side refusals of the
C ABI, and the binding's own checks. Nothing here needs a GPU."""
import ctypes

import numpy as np
import pytest

import kv_cache_early_gb300 as K
from cache_ops_harness import Pool
from kv_cache_early_gb300 import build as B
from oracle import cache_ops as O
from test_abi import FAKE, good_shape

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.lib()


# ----------------------------------------------------------------------------
# the oracle
# ----------------------------------------------------------------------------
def test_rotation_closed_forms():
    x = np.arange(1.0, 9.0)
    inv = np.array([1.0, 0.5, 0.25, 0.0])
    assert np.array_equal(O.rotate(x, 0, inv, 8, False), x)                       # position 0
    y = O.rotate(x, 3, inv, 8, False)
    assert np.allclose(y[0:8:4] @ y[0:8:4], x[0:8:4] @ x[0:8:4])                  # lengths of pairs stay
    assert y[3] == x[3] and y[7] == x[7]                                          # frequency 0
    quarter = np.array([np.pi / 2])
    assert np.allclose(O.rotate(x, 1, quarter, 2, True)[:2], [-2.0, 1.0])         # a quarter turn
    assert np.allclose(O.rotate(x, 1, quarter, 2, False, 2.0)[:3], [-4.0, 2.0, 3.0])
    # q . k depends on the distance of the positions only
    a, b = np.linspace(-1, 1, 8), np.linspace(2, -3, 8)
    for inter in (False, True):
        d1 = O.rotate(a, 9, inv, 8, inter) @ O.rotate(b, 4, inv, 8, inter)
        d2 = O.rotate(a, 105, inv, 8, inter) @ O.rotate(b, 100, inv, 8, inter)
        assert abs(d1 - d2) < 1e-12


def test_append_places():
    rng = np.random.default_rng(0)
    pool = Pool(rng, "f32", 1, 4, 2, [5, 3], fill=False)
    k, v = np.arange(12.0).reshape(3, 1, 4), -np.arange(12.0).reshape(3, 1, 4)
    q = np.zeros((3, 1, 4))
    _, kc, vc = O.append(q, k, v, [0, 2, 3], None, pool.table, [5, 3], [], 0, False, 1.0, pool.k, pool.v,
                         pool.num_pages)
    t = pool.table
    assert np.array_equal(kc[t[0, 1], 0, 1], k[0, 0]) and np.array_equal(kc[t[0, 2], 0, 0], k[1, 0])
    assert np.array_equal(vc[t[1, 1], 0, 0], v[2, 0])
    assert np.isnan(kc).sum() == kc.size - 12


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    pool = Pool(rng, "f32", 2, 8, 8, [9, 20])
    q = rng.standard_normal((5, 4, 8))
    off = [0, 2, 5]
    # equal keys: the mean of the visible values
    pool.k[:] = 0.5
    out = O.extend(q, pool.k, pool.v, pool.table, [9, 20], off, True)
    v = O.gather(pool.v, pool.table[1], 20, 1)
    assert np.allclose(out[2, 2], v[:18].mean(0)) and np.allclose(out[4, 3], v.mean(0))
    full = O.extend(q, pool.k, pool.v, pool.table, [9, 20], off, False)
    assert np.allclose(full[2, 2], v.mean(0))
    # a shared prefix read through the leader equals the leader's own rows
    pool.k[:] = rng.standard_normal(pool.k.shape)
    one = O.decode_shared(q[:2], pool.k, pool.v, pool.table, [9, 20], [0, 2], [8])
    table = pool.table.copy()
    table[1, 0] = table[0, 0]
    two = O.decode_shared(q[:2], pool.k, pool.v, table, [9, 20], [0], [])
    assert np.allclose(one, two)
    assert np.array_equal(O.decode_shared(q[:2], pool.k, pool.v, table, [0, 20], [0, 2], [8])[0], np.zeros((4, 8)))


# ----------------------------------------------------------------------------
# refusals of the C ABI (host checks only: no device pointer is touched)
# ----------------------------------------------------------------------------
def call_append(lib, shape=None, q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, qs=1024, ks=256, vs=256, off=FAKE, T=4,
                inv=FAKE, rot=128, inter=0, ws=FAKE, ws_bytes=64, reserved=0, rope=True, kc=FAKE):
    r = K.ArtRope(rot_dim=rot, interleaved=inter, scale=1.0)
    r.reserved[2] = reserved
    s = good_shape() if shape is None else shape
    return lib.art_append_kv(P(q), P(k), P(v), qs, ks, vs, P(off), T, None, P(FAKE), P(FAKE), P(inv),
                             ctypes.byref(r) if rope else None, P(q_out), P(kc), P(FAKE), ctypes.byref(s), P(ws),
                             ws_bytes, None)


BAD, UNS, WS = K.ART_ERR_INVALID_ARG, K.ART_ERR_UNSUPPORTED, K.ART_ERR_WORKSPACE


@pytest.mark.parametrize("case,expect", [
    (dict(shape=good_shape(head_dim=96)), UNS),
    (dict(shape=good_shape(page_size=12)), UNS),
    (dict(shape=good_shape(num_pages_total=0)), BAD),
    (dict(k=0), BAD), (dict(v=0), BAD), (dict(kc=0), BAD), (dict(ws=0), BAD), (dict(rope=False), BAD),
    (dict(q=0), BAD), (dict(q_out=0), BAD),                 # queries in and out go together
    (dict(k=FAKE + 8), BAD), (dict(q_out=FAKE + 2), BAD),   # 16-byte rows
    (dict(qs=1020), BAD), (dict(qs=1000), BAD),             # a stride off the 16-byte chunks; shorter than a row
    (dict(ks=248), BAD), (dict(vs=260), BAD),
    (dict(T=-1), BAD), (dict(off=0, T=4), BAD),             # without offsets: one token for each of 2 sequences
    (dict(rot=3), BAD), (dict(rot=-2), BAD), (dict(rot=130), BAD), (dict(inter=2), BAD), (dict(inv=0), BAD),
    (dict(reserved=1), BAD),
    (dict(T=0x7fffffff), UNS),
    (dict(ws_bytes=63), WS),
    (dict(q=FAKE, q_out=FAKE, qs=1536), BAD),               # in place, but the rows of q are further apart
    (dict(shape=good_shape(batch=1, num_q_heads=1 << 22, num_kv_heads=1 << 22), off=0, T=1, qs=1 << 29, ks=1 << 29,
          vs=1 << 29), UNS),
])
def test_append_refusals(lib, case, expect):
    assert call_append(lib, **case) == expect


def call_extend(lib, shape=None, q=FAKE, kc=FAKE, off=FAKE, T=4, causal=1, out=FAKE, ws=FAKE, ws_bytes=8):
    s = good_shape() if shape is None else shape
    return lib.dense_extend(P(q), P(kc), P(FAKE), P(FAKE), P(FAKE), P(off), T, causal, P(out), ctypes.byref(s), P(ws),
                            ws_bytes, None)


@pytest.mark.parametrize("case,expect", [
    (dict(shape=good_shape(num_q_heads=6)), UNS), (dict(shape=good_shape(dtype=3)), BAD),
    (dict(q=0), BAD), (dict(out=0), BAD), (dict(kc=0), BAD), (dict(off=0), BAD), (dict(ws=0), BAD),
    (dict(q=FAKE + 8), BAD), (dict(out=FAKE + 4), BAD), (dict(ws=FAKE + 8), BAD),
    (dict(T=-1), BAD), (dict(causal=2), BAD),
    (dict(T=1 << 30), UNS),                                  # rows beyond 32-bit counts
    (dict(shape=good_shape(max_pages_per_seq=1 << 27)), UNS),
    (dict(), WS),
])
def test_extend_refusals(lib, case, expect):
    assert call_extend(lib, **case) == expect


def call_shared(lib, shape=None, q=FAKE, off=FAKE, pre=FAKE, groups=1, out=FAKE, ws=FAKE, ws_bytes=8):
    s = good_shape() if shape is None else shape
    return lib.dense_decode_shared(P(q), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(off), P(pre), groups, P(out),
                                   ctypes.byref(s), P(ws), ws_bytes, None)


@pytest.mark.parametrize("case,expect", [
    (dict(shape=good_shape(block_size=32)), UNS),
    (dict(q=0), BAD), (dict(out=0), BAD), (dict(off=0), BAD), (dict(pre=0), BAD), (dict(groups=-1), BAD),
    (dict(groups=8193), UNS), (dict(shape=good_shape(batch=1 << 20, max_pages_per_seq=1 << 20)), UNS),
    (dict(q=FAKE + 8), BAD), (dict(ws=FAKE + 4), BAD),
    (dict(off=0, pre=0, groups=0), WS),                      # no groups need neither array
    (dict(), WS),
])
def test_shared_refusals(lib, case, expect):
    assert call_shared(lib, **case) == expect


def test_workspace_sizes(lib):
    s = good_shape()
    assert K.art_append_workspace_bytes(s) == 64
    a, b = K.dense_extend_workspace_bytes(s, 1), K.dense_extend_workspace_bytes(s, 100000)
    assert 64 < a < b
    assert K.dense_extend_workspace_bytes(s, -1) == 0 and K.dense_extend_workspace_bytes(s, 1 << 30) == 0
    assert K.dense_extend_workspace_bytes(good_shape(head_dim=96), 1) == 0
    assert 64 < K.dense_decode_shared_workspace_bytes(s, 0) <= K.dense_decode_shared_workspace_bytes(s, 500)
    assert lib.art_append_workspace_bytes(None) == 0
    assert lib.dense_extend_workspace_bytes(None, 1) == 0
    assert lib.dense_decode_shared_workspace_bytes(None, 1) == 0


def test_rope_struct_matches_header():
    assert ctypes.sizeof(K.ArtRope) == 32


def test_binding_refuses_host_tensors(lib):
    torch = pytest.importorskip("torch")
    s = good_shape()
    z = lambda *n, dt=torch.bfloat16: torch.zeros(*n, dtype=dt)
    pool = z(16, 2, 16, 128)
    i32 = lambda *n: z(*n, dt=torch.int32)
    with pytest.raises(K.ArtError):
        K.dense_extend(z(4, 8, 128), pool, pool, i32(2, 8), i32(2), i32(3), z(4, 8, 128), s, z(1 << 20, dt=torch.uint8))
    with pytest.raises(K.ArtError):
        K.dense_decode_shared(z(2, 8, 128, dt=torch.float32), pool, pool, i32(2, 8), i32(2), None, None, z(2, 8, 128), s,
                              z(1 << 20, dt=torch.uint8))
    with pytest.raises(K.ArtError):
        K.art_append_kv(None, z(4, 2, 128), z(4, 2, 128), i32(2, 8), i32(2), i32(3), z(64, dt=torch.float32), None,
                        pool, pool, s, z(64, dt=torch.uint8), rot_dim=128)
