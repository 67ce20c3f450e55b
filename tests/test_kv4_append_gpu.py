"""GPU tests of art_append_kv4 at the ends of its ranges, against the fp64 oracle (oracle/kv4.py), byte by byte."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_kv4_gpu import append_case  # noqa: E402

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
