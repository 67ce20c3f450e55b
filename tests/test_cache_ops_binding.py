"""CPU tests of the binding of art_append_kv, dense_extend and dense_decode_shared."""
import numpy as np
import pytest

import kv_cache_early_gb300 as K


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
