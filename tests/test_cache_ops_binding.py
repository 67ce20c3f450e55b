"""CPU tests of the binding of art_append_kv, dense_extend and dense_decode_shared, and of their host checks
beside the decode path's."""
import ctypes

import numpy as np
import pytest

import kv_cache_early_gb300 as K
from kv_cache_early_gb300 import build as B
from test_abi import FAKE, good_shape


def test_rope_goes_by_values():
    """The rotation's options are kept by their values: a scale that is changed in place is not found as it was."""
    torch = pytest.importorskip("torch")
    for scale in (torch.tensor(0.5), np.array(0.5)):
        a = K._rope(64, False, scale)
        assert (a.rot_dim, a.interleaved, a.scale) == (64, 0, 0.5) and not any(a.reserved)
        scale.fill_(2.0) if hasattr(scale, "fill_") else scale.fill(2.0)
        assert K._rope(64, False, scale).scale == 2.0
        assert K._rope(64, False, 0.5).scale == 0.5
    assert K._rope(64, True, 1).interleaved == 1 and K._rope(64, False, 1).interleaved == 0
    for i in range(200):
        assert K._rope(2, False, float(i)).scale == float(i)
    assert len(K._ropes) <= 64


SIZES = dict(batch=(0, -1, 1, 1 << 29), num_q_heads=(0, 2, 4, 6, 7, 8, 10, 12, 14, 16, 32), num_kv_heads=(0, 1, 2, 3, 4, 8),
             head_dim=(0, 32, 64, 96, 128, 256), page_size=(0, 4, 8, 12, 16, 4096, 8192), block_size=(0, 32, 64, 128),
             max_pages_per_seq=(0, 1, 100), num_pages_total=(0, 1, 1 << 20), dtype=(-1, 0, 1, 2))


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.lib()


def test_shape_rules_are_those_of_the_decode_path(lib):
    """The calls around the cache take the shapes that dense_decode takes, with the same answer for the others.
    (Host checks only: a workspace of 8 bytes ends every call whose shape passes.)"""
    P = ctypes.c_void_p
    shapes = [good_shape(**{n: x}) for n, xs in SIZES.items() for x in xs]
    shapes += [good_shape(num_q_heads=a, num_kv_heads=b) for a in SIZES["num_q_heads"] for b in SIZES["num_kv_heads"]]
    rng = np.random.default_rng(0)
    shapes += [good_shape(**{n: int(rng.choice(SIZES[n])) for n in rng.choice(list(SIZES), 2, replace=False)})
               for _ in range(300)]
    seen = set()
    for s in shapes:
        sp = ctypes.byref(s)
        expect = lib.dense_decode(P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, P(FAKE), sp, P(FAKE), 8, None)
        seen.add(expect)
        rope = K.ArtRope(0, 0, 1.0)
        wide = 1 << 12  # a stride that is long enough for every shape here
        got = (lib.art_append_kv(P(FAKE), P(FAKE), P(FAKE), wide, wide, wide, P(FAKE), 4, None, P(FAKE), P(FAKE), None,
                                 ctypes.byref(rope), P(FAKE + 4096), P(FAKE), P(FAKE), sp, P(FAKE), 8, None),
               lib.dense_extend(P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), 4, 1, P(FAKE), sp, P(FAKE), 8, None),
               lib.dense_decode_shared(P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), None, None, 0, P(FAKE), sp, P(FAKE),
                                       8, None))
        sizes = [getattr(s, f) for f, _ in K.ArtShape._fields_]
        if s.batch == 1 << 29 and expect == K.ART_ERR_WORKSPACE:  # taken by the shape's rules, too large for a work list
            assert got[0] == expect and set(got[1:]) <= {expect, K.ART_ERR_UNSUPPORTED}, sizes
        else:
            assert got == (expect,) * 3, (sizes, expect, got)
    assert seen == {K.ART_ERR_INVALID_ARG, K.ART_ERR_UNSUPPORTED, K.ART_ERR_WORKSPACE}
    # what only the decode path needs
    assert lib.dense_extend_workspace_bytes(ctypes.byref(good_shape(max_visit=0, num_probe=0)), 4) > 0
