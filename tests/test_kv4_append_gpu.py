"""GPU tests of art_append_kv4 at the ends of its ranges, against the fp64 oracle (oracle/kv4.py), byte by byte."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv_cache_early_gb300 as K  # noqa: E402
from cache_ops_harness import E24, U, rounded  # noqa: E402
from kv4_harness import Pool4  # noqa: E402
from oracle import cache_ops as O  # noqa: E402
from oracle import kv4 as Q  # noqa: E402
from test_kv4_gpu import append_case, dev, host, workspace  # noqa: E402

BOTH = pytest.mark.parametrize("dtype", ["bf16", "f32"])


@BOTH
@pytest.mark.parametrize("few", [True, False])
def test_spans_at_the_limit(dtype, few):
    """Groups that span just below 15 * 2^100, which keep their codes, that much, and just above, which become NaN."""
    def values(rng, x):
        y = np.round(rng.uniform(1, 29, x.shape)) / 2 * 2.0 ** 100  # at and between the borders of codes
        lowest = np.array([2.0 ** 60, 0.0, -2.0 ** 60, 2.0 ** 90, 2.0 ** 70])
        y[..., 0::32] = 15 * 2.0 ** 100
        y[..., 1::32] = lowest[(np.arange(x.shape[0])[:, None] + np.arange(x.shape[1])) % 5][..., None]
        return y
    append_case(30, dtype, (2, 2, 128), 16, 32, [40] if few else [640], [3], 0, False, values=values)
    append_case(31, dtype, (2, 2, 64), 16, 64, [12], [3], 0, False, values=values)


def far_case(seed, dtype, pos, inv, interleaved, exact):
    """One token a position of `pos`, heads of 64 columns that turn whole, each a sequence of one token."""
    rng = np.random.default_rng(seed)
    pos, inv, d, hq, hkv, page, group = np.asarray(pos, np.int32), np.asarray(inv, np.float32), 64, 2, 2, 8, 32
    T = len(pos)
    pool = Pool4(rng, dtype, hkv, d, page, group, [1] * T)
    q, k, v = (rounded(rng.standard_normal((T, h, d)), dtype) for h in (hq, hkv, hkv))
    shape = K.make_shape(**pool.shape(hq))
    ws, cache, dt = workspace(64), dev(pool.bytes), torch.bfloat16 if dtype == "bf16" else torch.float32
    q_out = torch.zeros(T, hq, d, dtype=dt, device="cuda")
    K.art_append_kv4(dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(pool.table), dev(pool.seq_lens), None, dev(inv), q_out,
                     cache, shape, ws, group=group, rot_dim=d, interleaved=interleaved, positions=dev(pos))
    torch.cuda.synchronize()
    assert K.art_read_device_status(ws) == 0
    got = cache.cpu().numpy()
    if exact:
        ref = Q.append(k, v, np.arange(T + 1), pos, pool.table, pool.seq_lens, inv, d, interleaved, 1.0, pool.bytes, page, group,
                       dtype)
        assert np.array_equal(got, ref), np.argwhere(got != ref)[:5]
    # In 64 bits the product rounds alike here and in the oracle. What is left after the turns are taken off differs by
    # the turns times the rounding of 2 pi (2.5e-16 each), the rounding of their product where it is not fused
    # (2^-53 of the angle) and, of the kernel's sines, 1e-11 (keys) or 2^-23 (queries).
    away = np.abs(pos.astype(np.float64))[:, None] * np.abs(inv.astype(np.float64))  # [T, d / 2]
    away = np.repeat(away, 2, 1) if interleaved else np.concatenate([away, away], 1)
    away = away * (2.0 ** -53 + 2.5e-16 / 6.28)
    for t in range(T):
        for g in range(hkv):
            code, step, low = Q.get(got, page, d, group, int(pool.table[t, 0]), g, 0, 0)
            x = O.rotate(k[t, g], int(pos[t]), inv, d, interleaved)
            # half a step from the key as rounded to the type; the step itself is rounded to 8 bits: 15 * 2^-9 of one at the top
            tol = 0.5 * step + 2 * U[dtype] * np.abs(x) + 2 * np.abs(k[t, g]).max() * (away[t] + 1e-11)
            assert np.all(np.abs(low + step * code - x) <= tol), (t, g)
        for h in range(hq):
            x = O.rotate(q[t, h], int(pos[t]), inv, d, interleaved)
            top = 2 * np.abs(q[t, h]).max()
            assert np.all(np.abs(host(q_out[t, h]) - x) <= U[dtype] * np.abs(x) + top * (8.2 * E24 + away[t])), (t, h)


@BOTH
@pytest.mark.parametrize("interleaved", [False, True])
def test_negative_and_far_positions(dtype, interleaved):
    """Positions of both signs; angles below 2^24, exact; and those beyond, by position or by frequency, from 64 bits."""
    inv = 10000.0 ** (-np.arange(32) / 32)
    far_case(40, dtype, [-1, 0, 1, -77, 12345, -(1 << 20), (1 << 24) - 1, 1 - (1 << 24)], inv, interleaved, exact=True)
    far_case(41, dtype, [1 << 24, -(1 << 24), (1 << 27) + 1, -(1 << 30) - 3, (1 << 31) - 1, -(1 << 31)], inv, interleaved,
             exact=False)
    far_case(42, dtype, [3, -5, 100000, -2000000, 1 << 25], 3.0 ** np.linspace(4, -4, 32), interleaved, exact=False)
